"""Depthwise-convolution path for AMD Instinct MI355X (gfx950).

A thin ctypes binding over ``libdwconv.so``, whose C ABI is declared in
``include/dwconv.h``.  Every step of every operation runs in the library's
HIP kernels; this module only checks tensor dtypes, devices and layouts,
allocates outputs with torch when the caller gives none, and passes raw
device pointers plus torch's current HIP stream.  It fails loudly when the
library has not been built: there is no other implementation to fall back on.

Layouts are channel-last and contiguous: x [B,T,C] (1-D), [B,T,F,C] (2-D),
[B,T,F] (mel); weights tap-major w [K,C] / [3,3,C]; lengths int32 [B] on the
same device (or None for full length).
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct

import torch

__all__ = [
    "LIB_PATH", "DwconvError", "abi_version",
    "dwconv1d_fwd", "dwconv1d_stream_fwd", "dwconv1d_bwd", "dwconv1d_bwd_workspace_bytes", "dwsub_fused_fwd", "dwsub_fused_bwd", "dwsub_fused_bwd_workspace_bytes",
    "dwconv2d_fwd", "dwconv2d_bwd", "dwconv2d_bwd_workspace_bytes", "dwconv2d_bwd_noalloc",
    "dwattn_fwd", "dwattn_fwd_workspace_bytes", "dwattn_bwd", "dwattn_bwd_workspace_bytes", "rel_buckets",
    "dwnorm_fwd", "dwnorm_bwd", "dwnorm_bwd_workspace_bytes", "dwdrop_fwd", "dwdrop_bwd",
    "conv2d_out_shape", "CAUSAL_PADS_2D", "front_out_shape", "out_len",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libdwconv.so")

DW_OK, DW_ERR_INVALID_ARG, DW_ERR_UNSUPPORTED, DW_ERR_WORKSPACE, DW_ERR_HIP = 0, -1, -2, -3, -4
DW_F32, DW_BF16 = 0, 1
DW_PAD_SYMMETRIC, DW_PAD_CAUSAL = 0, 1


class DwconvError(RuntimeError):
    """A call into libdwconv.so returned a non-OK status."""

    def __init__(self, status: int, message: str):
        super().__init__(f"[status {status}] {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build the HIP library first "
        "(python conv_subsampling_amd/build.py, or __graft_entry__.build())")

_vp, _i64, _sz, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
_f32, _f64 = ctypes.c_float, ctypes.c_double


# struct dw_attn: 6 sizes, the strides of q, k, v, dq, dk and dv, buckets, reach,
# left, right; scale, dtype.
_attn_struct = struct.Struct("=28qfi")


def _bind(path: str) -> ctypes.CDLL:
    """Load a build of the library and declare its C signatures."""
    lib = ctypes.CDLL(path)
    lib.dw_abi_version.restype = _int
    lib.dw_abi_version.argtypes = []
    lib.dw_last_error.restype = ctypes.c_char_p
    lib.dw_last_error.argtypes = []
    lib.dwconv1d_fwd.restype = _int
    lib.dwconv1d_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _vp]
    lib.dwconv1d_stream_fwd.restype = _int
    lib.dwconv1d_stream_fwd.argtypes = [_vp] * 7 + [_i64] * 4 + [_int, _vp]
    lib.dwconv1d_bwd_workspace_bytes.restype = _sz
    lib.dwconv1d_bwd_workspace_bytes.argtypes = [_i64] * 4
    lib.dwconv1d_bwd.restype = _int
    lib.dwconv1d_bwd.argtypes = [_vp] * 8 + [_sz] + [_i64] * 4 + [_int, _int, _vp]
    lib.dwsub_fused_fwd_ex.restype = _int
    lib.dwsub_fused_fwd_ex.argtypes = [_vp] * 7 + [_i64] * 4 + [_int, _int, _vp]
    lib.dwsub_fused_bwd_workspace_bytes_ex.restype = _sz
    lib.dwsub_fused_bwd_workspace_bytes_ex.argtypes = [_i64] * 4 + [_int]
    lib.dwsub_fused_bwd_ex.restype = _int
    lib.dwsub_fused_bwd_ex.argtypes = [_vp] * 11 + [_sz] + [_i64] * 4 + [_int, _int, _vp]
    lib.dwsub_fused_fwd.restype = _int
    lib.dwsub_fused_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp]
    lib.dwsub_fused_bwd_workspace_bytes.restype = _sz
    lib.dwsub_fused_bwd_workspace_bytes.argtypes = [_i64] * 4
    lib.dwsub_fused_bwd.restype = _int
    lib.dwsub_fused_bwd.argtypes = [_vp] * 11 + [_sz] + [_i64] * 4 + [_vp]
    lib.dwconv2d_fwd.restype = _int
    lib.dwconv2d_fwd.argtypes = [_vp, _vp, _vp, _vp, _vp] + [_i64] * 8 + [_vp]
    lib.dwconv2d_bwd_workspace_bytes.restype = _sz
    lib.dwconv2d_bwd_workspace_bytes.argtypes = [_i64] * 8
    lib.dwconv2d_bwd.restype = _int
    lib.dwconv2d_bwd.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz] + [_i64] * 8 + [_vp]
    lib.dwconv2d_fwd_ex.restype = _int
    lib.dwconv2d_fwd_ex.argtypes = [_vp] * 5 + [_i64] * 11 + [_int, _vp]
    lib.dwconv2d_bwd_workspace_bytes_ex.restype = _sz
    lib.dwconv2d_bwd_workspace_bytes_ex.argtypes = [_i64] * 11
    lib.dwconv2d_bwd_ex.restype = _int
    lib.dwconv2d_bwd_ex.argtypes = [_vp] * 8 + [_sz] + [_i64] * 11 + [_int, _vp]
    lib.dwconv2d_bwd_noalloc.restype = _int
    lib.dwconv2d_bwd_noalloc.argtypes = [_vp] * 7 + [_i64] * 11 + [_int, _vp]
    lib.dwdrop_fwd.restype = _int
    lib.dwdrop_fwd.argtypes = [_vp] * 4 + [_i64] * 2 + [_f64, _f32, _int, _vp]
    lib.dwdrop_bwd.restype = _int
    lib.dwdrop_bwd.argtypes = [_vp] * 3 + [_i64] * 2 + [_f64, _f32, _int, _vp]
    lib.dwnorm_fwd.restype = _int
    lib.dwnorm_fwd.argtypes = [_vp] * 10 + [_i64] * 3 + [_f32, _f32, _f64, _int, _vp]
    lib.dwnorm_bwd_workspace_bytes.restype = _sz
    lib.dwnorm_bwd_workspace_bytes.argtypes = [_i64] * 3
    lib.dwnorm_bwd.restype = _int
    lib.dwnorm_bwd.argtypes = [_vp] * 13 + [_sz] + [_i64] * 3 + [_f32, _f64, _int, _vp]
    attn = ctypes.c_char_p  # a packed dw_attn
    lib.dwattn_rel_buckets.restype = _int
    lib.dwattn_rel_buckets.argtypes = [_vp, _i64, _i64, _int]
    lib.dwattn_fwd_workspace_bytes.restype = _sz
    lib.dwattn_fwd_workspace_bytes.argtypes = [attn]
    lib.dwattn_fwd.restype = _int
    lib.dwattn_fwd.argtypes = [attn] + [_vp] * 11 + [_sz, _vp]
    lib.dwattn_bwd_workspace_bytes.restype = _sz
    lib.dwattn_bwd_workspace_bytes.argtypes = [attn]
    lib.dwattn_bwd.restype = _int
    lib.dwattn_bwd.argtypes = [attn] + [_vp] * 16 + [_sz, _vp]
    return lib


_lib = _bind(LIB_PATH)


def abi_version() -> int:
    return _lib.dw_abi_version()


def _check(status: int) -> None:
    if status != DW_OK:
        raise DwconvError(status, _lib.dw_last_error().decode(errors="replace"))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _dev_tensor(name, t, dtype, device, shape=None, allow_none=False):
    if (type(t) is torch.Tensor and t.dtype is dtype and t.device == device and t.is_contiguous()
            and (shape is None or t.shape == shape)):
        return t  # the usual case, in one test: small calls are bound by the host
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


# The stream's handle without a torch.cuda.Stream object around it, which costs
# as much as a small kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def out_len(n: int) -> int:
    """Output length of a 3x3 / stride 2 / pad 1 convolution along one axis."""
    return (n + 1) // 2


def dwconv1d_fwd(x, w, bias=None, lengths=None, y=None, causal: bool = False):
    """Depthwise Conv1d in SSM_CONV form; x [B,T,C], w [K,C] (float32 or bfloat16)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    dev, dt = x.device, x.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError("dwconv1d_fwd takes float32 or bfloat16 tensors")
    B, T, C = x.shape
    _dev_tensor("x", x, dt, dev)
    if w.dim() != 2 or w.shape[1] != C:
        raise ValueError("w must be [K, C]")
    _dev_tensor("w", w, dt, dev)
    K = w.shape[0]
    _dev_tensor("bias", bias, dt, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    if y is None:
        y = torch.empty_like(x)
    _dev_tensor("y", y, dt, dev, (B, T, C))
    _check(_lib.dwconv1d_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(lengths), _ptr(y), B, T, C, K,
                             DW_PAD_CAUSAL if causal else DW_PAD_SYMMETRIC,
                             DW_BF16 if dt == torch.bfloat16 else DW_F32, _stream(dev)))
    return y


def dwconv1d_stream_fwd(x, w, bias, lengths, cache_in, cache_out=None, y=None):
    """One chunk x [B,Tc,C] of a causal 1-D depthwise conv after the cached
    K-1 frames cache_in [B,K-1,C]; returns (y, cache_out).  cache_out must be
    a different tensor from cache_in (it is allocated when not given)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, Tc, C]")
    dev, dt = x.device, x.dtype
    if dt not in (torch.float32, torch.bfloat16):
        raise TypeError(f"x must be float32 or bfloat16, not {dt}")
    B, Tc, C = x.shape
    _dev_tensor("x", x, dt, dev)
    if w.dim() != 2 or w.shape[1] != C:
        raise ValueError("w must be [K, C]")
    _dev_tensor("w", w, dt, dev)
    K = w.shape[0]
    _dev_tensor("bias", bias, dt, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    _dev_tensor("cache_in", cache_in, dt, dev, (B, K - 1, C))
    if cache_out is None:
        cache_out = torch.empty_like(cache_in)
    _dev_tensor("cache_out", cache_out, dt, dev, (B, K - 1, C))
    if y is None:
        y = torch.empty_like(x)
    _dev_tensor("y", y, dt, dev, (B, Tc, C))
    _check(_lib.dwconv1d_stream_fwd(_ptr(x), _ptr(w), _ptr(bias), _ptr(lengths), _ptr(cache_in), _ptr(y),
                                    _ptr(cache_out), B, Tc, C, K, DW_BF16 if dt == torch.bfloat16 else DW_F32,
                                    _stream(dev)))
    return y, cache_out


def dwconv1d_bwd_workspace_bytes(B, T, C, K) -> int:
    return int(_lib.dwconv1d_bwd_workspace_bytes(B, T, C, K))


def dwconv1d_bwd(x, w, lengths, dy, dx=None, dw=None, db=None, workspace=None, causal: bool = False,
                 need=("dx", "dw", "db")):
    """Gradients (dx, dw, db) of dwconv1d_fwd given dy [B,T,C].  x, w, dy and
    dx share one storage type (float32 or bfloat16); dw and db are float32."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    dev, f32 = x.device, torch.float32
    st, code = _storage(x)
    B, T, C = x.shape
    _dev_tensor("x", x, st, dev)
    if w.dim() != 2 or w.shape[1] != C:
        raise ValueError("w must be [K, C]")
    _dev_tensor("w", w, st, dev)
    K = w.shape[0]
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    _dev_tensor("dy", dy, st, dev, (B, T, C))
    if dx is None and "dx" in need:
        dx = torch.empty_like(x)
    if dw is None and "dw" in need:
        dw = torch.empty((K, C), dtype=f32, device=dev)
    if db is None and "db" in need:
        db = torch.empty((C,), dtype=f32, device=dev)
    _dev_tensor("dx", dx, st, dev, (B, T, C), allow_none=True)
    _dev_tensor("dw", dw, f32, dev, (K, C), allow_none=True)
    _dev_tensor("db", db, f32, dev, (C,), allow_none=True)
    ws_bytes = 0
    if dw is not None or db is not None:
        need_ws = dwconv1d_bwd_workspace_bytes(B, T, C, K)
        if workspace is None:
            workspace = torch.empty((max(need_ws, 1),), dtype=torch.uint8, device=dev)
        _dev_tensor("workspace", workspace, torch.uint8, dev)
        ws_bytes = workspace.numel()
    _check(_lib.dwconv1d_bwd(_ptr(x), _ptr(w), _ptr(lengths), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(db),
                             _ptr(workspace), ws_bytes, B, T, C, K,
                             DW_PAD_CAUSAL if causal else DW_PAD_SYMMETRIC, code, _stream(dev)))
    return dx, dw, db


def front_out_shape(T, F, causal: bool = False):
    """(T2, F2) of the fused front: two stride-2 stages, each padding 1 before
    and after (symmetric) or 2 before and 1 after (causal)."""
    d = 1 if causal else 0
    half = lambda n: (n - 1 + d) // 2 + 1 if n > 0 else d
    return half(half(T)), half(half(F))


def dwsub_fused_fwd(x, w0, b0, w1, b1, lengths=None, y=None, causal: bool = False):
    """Fused subsampler front; x [B,T,F] mel -> y [B,T2,F2,C].  x, the
    parameters and y share one storage type (float32 or bfloat16)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, F]")
    dev = x.device
    st, code = _storage(x)
    B, T, F = x.shape
    _dev_tensor("x", x, st, dev)
    if w0.dim() != 3 or w0.shape[:2] != (3, 3):
        raise ValueError("w0 must be [3, 3, C]")
    C = w0.shape[2]
    _dev_tensor("w0", w0, st, dev)
    _dev_tensor("b0", b0, st, dev, (C,), allow_none=True)
    _dev_tensor("w1", w1, st, dev, (3, 3, C))
    _dev_tensor("b1", b1, st, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    T2, F2 = front_out_shape(T, F, causal)
    if y is None:
        y = torch.empty((B, T2, F2, C), dtype=st, device=dev)
    _dev_tensor("y", y, st, dev, (B, T2, F2, C))
    _check(_lib.dwsub_fused_fwd_ex(_ptr(x), _ptr(w0), _ptr(b0), _ptr(w1), _ptr(b1), _ptr(lengths), _ptr(y),
                                   B, T, F, C, DW_PAD_CAUSAL if causal else DW_PAD_SYMMETRIC, code, _stream(dev)))
    return y


def dwsub_fused_bwd_workspace_bytes(B, T, F, C, causal: bool = False) -> int:
    return int(_lib.dwsub_fused_bwd_workspace_bytes_ex(B, T, F, C, DW_PAD_CAUSAL if causal else DW_PAD_SYMMETRIC))


def dwsub_fused_bwd(x, w0, b0, w1, lengths, dy, dw0=None, db0=None, dw1=None, db1=None, workspace=None,
                    need=("dw0", "db0", "dw1", "db1"), causal: bool = False):
    """Parameter gradients (dw0, db0, dw1, db1) of dwsub_fused_fwd given dy
    [B,T2,F2,C].  x, w0, b0, w1 and dy share one storage type; the gradients
    are float32."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, F]")
    dev, f32 = x.device, torch.float32
    st, code = _storage(x)
    B, T, F = x.shape
    _dev_tensor("x", x, st, dev)
    if w0.dim() != 3 or w0.shape[:2] != (3, 3):
        raise ValueError("w0 must be [3, 3, C]")
    C = w0.shape[2]
    _dev_tensor("w0", w0, st, dev)
    _dev_tensor("b0", b0, st, dev, (C,), allow_none=True)
    _dev_tensor("w1", w1, st, dev, (3, 3, C))
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    T2, F2 = front_out_shape(T, F, causal)
    _dev_tensor("dy", dy, st, dev, (B, T2, F2, C))
    outs = {}
    for name, t, shape in (("dw0", dw0, (3, 3, C)), ("db0", db0, (C,)), ("dw1", dw1, (3, 3, C)), ("db1", db1, (C,))):
        if t is None and name in need:
            t = torch.empty(shape, dtype=f32, device=dev)
        outs[name] = _dev_tensor(name, t, f32, dev, shape, allow_none=True)
    need_ws = dwsub_fused_bwd_workspace_bytes(B, T, F, C, causal)
    if workspace is None:
        workspace = torch.empty((max(need_ws, 1),), dtype=torch.uint8, device=dev)
    _dev_tensor("workspace", workspace, torch.uint8, dev)
    _check(_lib.dwsub_fused_bwd_ex(_ptr(x), _ptr(w0), _ptr(b0), _ptr(w1), _ptr(lengths), _ptr(dy),
                                   _ptr(outs["dw0"]), _ptr(outs["db0"]), _ptr(outs["dw1"]), _ptr(outs["db1"]),
                                   _ptr(workspace), workspace.numel(), B, T, F, C,
                                   DW_PAD_CAUSAL if causal else DW_PAD_SYMMETRIC, code, _stream(dev)))
    return outs["dw0"], outs["db0"], outs["dw1"], outs["db1"]


def _conv2d_dims(x, w):
    if x.dim() != 4:
        raise ValueError("x must be [B, T, F, C]")
    B, T, F, C = x.shape
    if w.dim() != 3 or w.shape[2] != C:
        raise ValueError("w must be [KH, KW, C]")
    return B, T, F, C, w.shape[0], w.shape[1]


CAUSAL_PADS_2D = (2, 1, 2, 1)   # kernel - 1 before, stride - 1 after, on each axis (3x3, stride 2)


def _pads(pad, pads):
    if pads is None:
        return (pad, pad, pad, pad)
    pads = tuple(int(v) for v in pads)
    if len(pads) != 4:
        raise ValueError("pads must be (time before, time after, freq before, freq after)")
    return pads


def conv2d_out_shape(T, F, KH=3, KW=3, stride=2, pad=1, pads=None):
    """(T', F') of the conv2d for these sizes and pads."""
    pt0, pt1, pf0, pf1 = _pads(pad, pads)
    return max(0, (T + pt0 + pt1 - KH) // stride + 1), max(0, (F + pf0 + pf1 - KW) // stride + 1)


def _storage(x):
    if x.dtype == torch.float32:
        return torch.float32, DW_F32
    if x.dtype == torch.bfloat16:
        return torch.bfloat16, DW_BF16
    raise TypeError(f"x must be float32 or bfloat16, not {x.dtype}")


def dwconv2d_fwd(x, w, bias=None, lengths=None, y=None, stride: int = 2, pad: int = 1, pads=None):
    """Masked depthwise conv2d; x [B,T,F,C], w [3,3,C] -> y [B,T',F',C].
    x, w, bias and y share one storage type (float32 or bfloat16); pads =
    (time before, time after, freq before, freq after) overrides pad
    (CAUSAL_PADS_2D is the causal padding)."""
    dev = x.device
    st, code = _storage(x)
    B, T, F, C, KH, KW = _conv2d_dims(x, w)
    _dev_tensor("x", x, st, dev)
    _dev_tensor("w", w, st, dev)
    _dev_tensor("bias", bias, st, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    pt0, pt1, pf0, pf1 = _pads(pad, pads)
    To, Fo = conv2d_out_shape(T, F, KH, KW, stride, pads=(pt0, pt1, pf0, pf1))
    if y is None:
        y = torch.empty((B, To, Fo, C), dtype=st, device=dev)
    _dev_tensor("y", y, st, dev, (B, To, Fo, C))
    _check(_lib.dwconv2d_fwd_ex(_ptr(x), _ptr(w), _ptr(bias), _ptr(lengths), _ptr(y),
                                B, T, F, C, KH, KW, stride, pt0, pt1, pf0, pf1, code, _stream(dev)))
    return y


def dwconv2d_bwd_workspace_bytes(B, T, F, C, KH=3, KW=3, stride=2, pad=1, pads=None) -> int:
    pt0, pt1, pf0, pf1 = _pads(pad, pads)
    return int(_lib.dwconv2d_bwd_workspace_bytes_ex(B, T, F, C, KH, KW, stride, pt0, pt1, pf0, pf1))


def dwconv2d_bwd(x, w, lengths, dy, dx=None, dw=None, db=None, workspace=None,
                 need=("dx", "dw", "db"), stride: int = 2, pad: int = 1, pads=None):
    """Gradients (dx, dw, db) of dwconv2d_fwd given dy; outputs not in `need`
    are skipped (None).  x, w, dy and dx share one storage type; dw and db
    are float32."""
    dev, f32 = x.device, torch.float32
    st, code = _storage(x)
    B, T, F, C, KH, KW = _conv2d_dims(x, w)
    _dev_tensor("x", x, st, dev)
    _dev_tensor("w", w, st, dev)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    pt0, pt1, pf0, pf1 = _pads(pad, pads)
    To, Fo = conv2d_out_shape(T, F, KH, KW, stride, pads=(pt0, pt1, pf0, pf1))
    _dev_tensor("dy", dy, st, dev, (B, To, Fo, C))
    if dx is None and "dx" in need:
        dx = torch.empty_like(x)
    if dw is None and "dw" in need:
        dw = torch.empty((KH, KW, C), dtype=f32, device=dev)
    if db is None and "db" in need:
        db = torch.empty((C,), dtype=f32, device=dev)
    _dev_tensor("dx", dx, st, dev, (B, T, F, C), allow_none=True)
    _dev_tensor("dw", dw, f32, dev, (KH, KW, C), allow_none=True)
    _dev_tensor("db", db, f32, dev, (C,), allow_none=True)
    ws_bytes = 0
    if dw is not None or db is not None:
        need_ws = dwconv2d_bwd_workspace_bytes(B, T, F, C, KH, KW, stride, pads=(pt0, pt1, pf0, pf1))
        if workspace is None:
            workspace = torch.empty((max(need_ws, 1),), dtype=torch.uint8, device=dev)
        _dev_tensor("workspace", workspace, torch.uint8, dev)
        ws_bytes = workspace.numel()
    _check(_lib.dwconv2d_bwd_ex(_ptr(x), _ptr(w), _ptr(lengths), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(db),
                                _ptr(workspace), ws_bytes, B, T, F, C, KH, KW, stride, pt0, pt1, pf0, pf1, code,
                                _stream(dev)))
    return dx, dw, db


def dwconv2d_bwd_noalloc(x, w, lengths, dy, dx=None, dw=None, db=None, stride: int = 2, pad: int = 1, pads=None):
    """dwconv2d_bwd through the allocation-free entry point: the caller gives
    every output it wants (None skips it) and no workspace; the library keeps
    the partial sums in its own per-device scratch array.  Nothing here
    allocates device memory.  Calls that overlap in time on one GPU race."""
    dev, f32 = x.device, torch.float32
    st, code = _storage(x)
    B, T, F, C, KH, KW = _conv2d_dims(x, w)
    _dev_tensor("x", x, st, dev)
    _dev_tensor("w", w, st, dev)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    pt0, pt1, pf0, pf1 = _pads(pad, pads)
    To, Fo = conv2d_out_shape(T, F, KH, KW, stride, pads=(pt0, pt1, pf0, pf1))
    _dev_tensor("dy", dy, st, dev, (B, To, Fo, C))
    _dev_tensor("dx", dx, st, dev, (B, T, F, C), allow_none=True)
    _dev_tensor("dw", dw, f32, dev, (KH, KW, C), allow_none=True)
    _dev_tensor("db", db, f32, dev, (C,), allow_none=True)
    _check(_lib.dwconv2d_bwd_noalloc(_ptr(x), _ptr(w), _ptr(lengths), _ptr(dy), _ptr(dx), _ptr(dw), _ptr(db),
                                     B, T, F, C, KH, KW, stride, pt0, pt1, pf0, pf1, code, _stream(dev)))
    return dx, dw, db


def _rng(rng, p, device):
    """The dropout generator's state: int64 [2] (seed, stream) on the device."""
    return _dev_tensor("rng", rng, torch.int64, device, (2,), allow_none=p == 0)


def _rows(t):
    """[rows, C] of a tensor whose last axis is the channels."""
    if t.dim() < 1:
        raise ValueError("dropout takes a tensor with a channel axis")
    C = t.shape[-1]
    rows = 1
    for n in t.shape[:-1]:
        rows *= n
    return rows, C


def dwdrop_fwd(x, rng, p: float, residual=None, alpha: float = 1.0, y=None):
    """residual + alpha * dropout(x); x [..., C] (float32 or bfloat16).  rng is
    an int64 tensor [2] on the device, (seed, stream), from which the mask
    follows; it is never stored."""
    dev = x.device
    st, code = _storage(x)
    _dev_tensor("x", x, st, dev)
    _dev_tensor("residual", residual, st, dev, x.shape, allow_none=True)
    y = torch.empty_like(x) if y is None else _dev_tensor("y", y, st, dev, x.shape)
    rows, C = _rows(x)
    _check(_lib.dwdrop_fwd(_ptr(x), _ptr(residual), _ptr(y), _ptr(_rng(rng, p, dev)), rows, C, p, alpha, code,
                           _stream(dev)))
    return y


def dwdrop_bwd(dy, rng, p: float, alpha: float = 1.0, dx=None):
    """dx of dwdrop_fwd given dy, with the forward's rng, p and alpha."""
    dev = dy.device
    st, code = _storage(dy)
    _dev_tensor("dy", dy, st, dev)
    dx = torch.empty_like(dy) if dx is None else _dev_tensor("dx", dx, st, dev, dy.shape)
    rows, C = _rows(dy)
    _check(_lib.dwdrop_bwd(_ptr(dy), _ptr(dx), _ptr(_rng(rng, p, dev)), rows, C, p, alpha, code, _stream(dev)))
    return dx


def dwnorm_fwd(x, gamma=None, beta=None, lengths=None, residual=None, rng=None, p: float = 0.0, alpha: float = 1.0,
               eps: float = 1e-5, y=None, sum=None, mean=None, rstd=None, need=("y", "sum", "mean", "rstd")):
    """Layer norm of s = residual + alpha * dropout(x) over the channels; x
    [B,T,C].  Returns (y, s, mean, rstd): s in x's storage type (x itself where
    there is neither a residual, a scale nor a dropout, no `sum` is given and y
    is not written over x), mean and rstd float32 [B,T].  s, mean and rstd not in `need` are skipped
    (None)."""
    if x.dim() != 3:
        raise ValueError("x must be [B, T, C]")
    dev, f32 = x.device, torch.float32
    st, code = _storage(x)
    B, T, C = x.shape
    _dev_tensor("x", x, st, dev)
    _dev_tensor("gamma", gamma, st, dev, (C,), allow_none=True)
    _dev_tensor("beta", beta, st, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    _dev_tensor("residual", residual, st, dev, (B, T, C), allow_none=True)
    _rng(rng, p, dev)
    y = torch.empty_like(x) if y is None else _dev_tensor("y", y, st, dev, (B, T, C))
    plain = residual is None and p == 0 and alpha == 1.0 and sum is None and y.data_ptr() != x.data_ptr()
    if sum is not None:
        _dev_tensor("sum", sum, st, dev, (B, T, C))
    elif "sum" in need and not plain:
        sum = torch.empty_like(x)
    if mean is not None:
        _dev_tensor("mean", mean, f32, dev, (B, T))
    elif "mean" in need:
        mean = torch.empty((B, T), dtype=f32, device=dev)
    if rstd is not None:
        _dev_tensor("rstd", rstd, f32, dev, (B, T))
    elif "rstd" in need:
        rstd = torch.empty((B, T), dtype=f32, device=dev) if mean is None else torch.empty_like(mean)
    _check(_lib.dwnorm_fwd(_ptr(x), _ptr(residual), _ptr(gamma), _ptr(beta), _ptr(lengths), _ptr(rng), _ptr(y),
                           _ptr(sum), _ptr(mean), _ptr(rstd), B, T, C, eps, alpha, p, code, _stream(dev)))
    return y, x if plain and "sum" in need else sum, mean, rstd


def dwnorm_bwd_workspace_bytes(B, T, C) -> int:
    return int(_lib.dwnorm_bwd_workspace_bytes(B, T, C))


def dwnorm_bwd(sum, gamma, lengths, mean, rstd, dy, dsum=None, rng=None, p: float = 0.0, alpha: float = 1.0, dx=None,
               dres=None, dgamma=None, dbeta=None, workspace=None, need=("dx", "dres", "dgamma", "dbeta")):
    """Gradients (dx, dres, dgamma, dbeta) of dwnorm_fwd given dy and, along
    the residual, dsum; sum, mean and rstd are the forward's.  dx and dres are
    in the storage type, dgamma and dbeta float32; those not in `need` are
    skipped (None)."""
    if sum.dim() != 3:
        raise ValueError("sum must be [B, T, C]")
    dev, f32 = sum.device, torch.float32
    st, code = _storage(sum)
    B, T, C = sum.shape
    _dev_tensor("sum", sum, st, dev)
    _dev_tensor("gamma", gamma, st, dev, (C,), allow_none=True)
    _dev_tensor("lengths", lengths, torch.int32, dev, (B,), allow_none=True)
    _dev_tensor("mean", mean, f32, dev, (B, T))
    _dev_tensor("rstd", rstd, f32, dev, (B, T))
    _dev_tensor("dy", dy, st, dev, (B, T, C))
    _dev_tensor("dsum", dsum, st, dev, (B, T, C), allow_none=True)
    _rng(rng, p, dev)
    if dx is not None:
        _dev_tensor("dx", dx, st, dev, (B, T, C))
    elif "dx" in need:
        dx = torch.empty_like(sum)
    if dres is not None:
        _dev_tensor("dres", dres, st, dev, (B, T, C))
    elif "dres" in need:
        dres = torch.empty_like(sum)
    if dgamma is not None:
        _dev_tensor("dgamma", dgamma, f32, dev, (C,))
    elif "dgamma" in need:
        dgamma = torch.empty((C,), dtype=f32, device=dev)
    if dbeta is not None:
        _dev_tensor("dbeta", dbeta, f32, dev, (C,))
    elif "dbeta" in need:
        dbeta = torch.empty((C,), dtype=f32, device=dev) if dgamma is None else torch.empty_like(dgamma)
    ws_bytes = 0
    if dgamma is not None or dbeta is not None:
        if workspace is None:
            workspace = torch.empty((max(dwnorm_bwd_workspace_bytes(B, T, C), 1),), dtype=torch.uint8, device=dev)
        _dev_tensor("workspace", workspace, torch.uint8, dev)
        ws_bytes = workspace.numel()
    _check(_lib.dwnorm_bwd(_ptr(sum), _ptr(gamma), _ptr(lengths), _ptr(mean), _ptr(rstd), _ptr(dy), _ptr(dsum),
                           _ptr(rng), _ptr(dx), _ptr(dres), _ptr(dgamma), _ptr(dbeta), _ptr(workspace), ws_bytes,
                           B, T, C, alpha, p, code, _stream(dev)))
    return dx, dres, dgamma, dbeta


def rel_buckets(num_buckets: int, reach: int, bidirectional: bool = True, device="cuda"):
    """The usual map of relative positions to buckets for `dwattn_fwd`: int32
    [2 * reach + 1], entry r + reach the bucket of a key r frames after its
    query.  One distance a bucket up to a quarter of `num_buckets` (half of
    them, in one direction), then equal ratios up to `reach`."""
    if reach < 0 or reach > 1 << 20:
        raise ValueError("reach must be between 1 and 1024")
    m = torch.empty((2 * reach + 1,), dtype=torch.int32)
    _check(_lib.dwattn_rel_buckets(_ptr(m), num_buckets, reach, int(bool(bidirectional))))
    return m.to(device)


def _heads(name, t, st, device, shape):
    """A [B, frames, heads, D] tensor whose head elements lie next to each other."""
    if type(t) is torch.Tensor and t.dtype is st and t.device == device and t.shape == shape and t.stride(3) == 1:
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != st:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {st}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"{name} must have the elements of a head next to each other")
    return t


def _attn_shape(q, k, v, table, buckets, q_lengths, k_lengths, q_pos, left, right, scale):
    """Checks the tensors; the storage type, and the fields of the C ABI's dw_attn before and after the strides of
    the gradients."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, Tq, H, D], k and v [B, Tk, Hkv, D]")
    dev = q.device
    st, code = _storage(q)
    B, Tq, H, D = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    _heads("q", q, st, dev, q.shape)
    _heads("k", k, st, dev, (B, Tk, Hkv, D))
    _heads("v", v, st, dev, (B, Tk, Hkv, D))
    if (table is None) != (buckets is None):
        raise ValueError("a bias needs both its table and its buckets")
    NB = reach = 0
    if table is not None:
        if table.dim() != 2 or table.shape[1] != H:
            raise ValueError("table must be [num_buckets, H]")
        if buckets.dim() != 1 or buckets.shape[0] % 2 == 0:
            raise ValueError("buckets must be [2 * reach + 1]")
        _dev_tensor("table", table, st, dev)
        _dev_tensor("buckets", buckets, torch.int32, dev)
        NB, reach = table.shape[0], buckets.shape[0] // 2
    for name, t in (("q_lengths", q_lengths), ("k_lengths", k_lengths), ("q_pos", q_pos)):
        _dev_tensor(name, t, torch.int32, dev, (B,), allow_none=True)
    return st, (B, Tq, Tk, H, Hkv, D, *q.stride()[:3], *k.stride()[:3], *v.stride()[:3]), (
        NB, reach, _limit(left), _limit(right), D ** -0.5 if scale is None else scale, code)


_NO_STRIDES = (0,) * 9   # dq, dk, dv of a call that has none


@functools.lru_cache(maxsize=1024)
def _attn_workspace(backward: bool, shape: bytes) -> int:
    """The library's answer for these sizes, which depends on nothing else."""
    return int((_lib.dwattn_bwd_workspace_bytes if backward else _lib.dwattn_fwd_workspace_bytes)(shape))


def _limit(n: int) -> int:
    return n if -1 <= n < 1 << 40 else (-1 if n < 0 else 1 << 40)


def dwattn_fwd_workspace_bytes(q, k, v, left: int = -1, right: int = -1) -> int:
    """Bytes of workspace `dwattn_fwd` takes for tensors of these sizes."""
    _, sizes, rest = _attn_shape(q, k, v, None, None, None, None, None, left, right, None)
    return _attn_workspace(False, _attn_struct.pack(*sizes, *_NO_STRIDES, *rest))


def dwattn_fwd(q, k, v, table=None, buckets=None, q_lengths=None, k_lengths=None, q_pos=None, left: int = -1,
               right: int = -1, scale=None, out=None, lse=None, workspace=None, need=("out", "lse")):
    """Softmax attention with a learned relative position bias: q [B,Tq,H,D],
    k, v [B,Tk,Hkv,D] (float32 or bfloat16, any strides above the last), table
    [num_buckets,H], buckets int32 [2*reach+1] (see `rel_buckets`).  q_pos
    int32 [B] places query 0 on the key axis (the cached frames before a
    streaming chunk); left and right limit the context, negative for all of
    it.  Returns (out [B,Tq,H,D], lse float32 [B,H,Tq] or None if not in
    `need`); queries without a key give 0 and -inf."""
    st, sizes, rest = _attn_shape(q, k, v, table, buckets, q_lengths, k_lengths, q_pos, left, right, scale)
    shape = _attn_struct.pack(*sizes, *_NO_STRIDES, *rest)
    dev = q.device
    B, Tq, _, H, _, D = sizes[:6]
    if out is None:
        out = torch.empty((B, Tq, H, D), dtype=st, device=dev)
    else:
        _dev_tensor("out", out, st, dev, (B, Tq, H, D))
    if lse is not None:
        _dev_tensor("lse", lse, torch.float32, dev, (B, H, Tq))
    elif "lse" in need:
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=dev)
    if workspace is not None:
        _dev_tensor("workspace", workspace, torch.uint8, dev)
    else:
        need_ws = _attn_workspace(False, shape)
        if need_ws:
            workspace = torch.empty((need_ws,), dtype=torch.uint8, device=dev)
    _check(_lib.dwattn_fwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(table), _ptr(buckets), _ptr(q_lengths),
                           _ptr(k_lengths), _ptr(q_pos), _ptr(out), _ptr(lse), _ptr(workspace),
                           0 if workspace is None else workspace.numel(), _stream(dev)))
    return out, lse


def dwattn_bwd_workspace_bytes(q, k, v, table=None, buckets=None) -> int:
    """Bytes of workspace `dwattn_bwd` takes for tensors of these sizes."""
    _, sizes, rest = _attn_shape(q, k, v, table, buckets, None, None, None, -1, -1, None)
    return _attn_workspace(True, _attn_struct.pack(*sizes, *_NO_STRIDES, *rest))


def dwattn_bwd(q, k, v, out, lse, dout, table=None, buckets=None, q_lengths=None, k_lengths=None, q_pos=None,
               left: int = -1, right: int = -1, scale=None, dq=None, dk=None, dv=None, dtable=None, workspace=None,
               need=("dq", "dk", "dv", "dtable")):
    """Gradients (dq, dk, dv, dtable) of dwattn_fwd given its out and lse and
    dout; the other arguments are the forward's.  dq, dk and dv are in the
    storage type (given ones may have any strides above the last), dtable
    float32 [num_buckets,H]; those not in `need`, and dtable without a table,
    are skipped (None)."""
    st, sizes, rest = _attn_shape(q, k, v, table, buckets, q_lengths, k_lengths, q_pos, left, right, scale)
    dev, f32 = q.device, torch.float32
    B, Tq, _, H, _, D = sizes[:6]
    _dev_tensor("out", out, st, dev, (B, Tq, H, D))
    _dev_tensor("lse", lse, f32, dev, (B, H, Tq))
    _dev_tensor("dout", dout, st, dev, (B, Tq, H, D))
    if dq is not None:
        _heads("dq", dq, st, dev, q.shape)
    elif "dq" in need:
        dq = torch.empty_like(dout)
    if dk is not None:
        _heads("dk", dk, st, dev, k.shape)
    elif "dk" in need:
        dk = torch.empty(k.shape, dtype=st, device=dev)
    if dv is not None:
        _heads("dv", dv, st, dev, k.shape)
    elif "dv" in need:
        dv = torch.empty(k.shape, dtype=st, device=dev)
    if dtable is not None:
        if table is None:
            raise ValueError("dtable needs a table")
        _dev_tensor("dtable", dtable, f32, dev, table.shape)
    elif "dtable" in need and table is not None:
        dtable = torch.empty(table.shape, dtype=f32, device=dev)
    strides = [n for t in (dq, dk, dv) for n in ((0, 0, 0) if t is None else t.stride()[:3])]
    shape = _attn_struct.pack(*sizes, *strides, *rest)
    if workspace is not None:
        _dev_tensor("workspace", workspace, torch.uint8, dev)
    else:
        workspace = torch.empty((max(_attn_workspace(True, shape), 1),), dtype=torch.uint8, device=dev)
    _check(_lib.dwattn_bwd(shape, _ptr(q), _ptr(k), _ptr(v), _ptr(table), _ptr(buckets), _ptr(q_lengths),
                           _ptr(k_lengths), _ptr(q_pos), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(dtable), _ptr(workspace), workspace.numel(), _stream(dev)))
    return dq, dk, dv, dtable
