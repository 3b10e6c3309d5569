"""The encoder block's entry points refuse bad arguments on the host, before
anything touches a GPU (the addresses here are never dereferenced)."""
import ctypes
import os

import pytest

import block_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "conv_subsampling_amd", "libdwconv.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
P, Q, R, S, W = (ctypes.c_void_p(0x1000 * i) for i in range(1, 6))
N = None
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(LIB)
    i64, vp, sz, i, f, d = (ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float,
                            ctypes.c_double)
    lib.dw_last_error.restype = ctypes.c_char_p
    lib.dwdrop_fwd.argtypes = [vp] * 4 + [i64] * 2 + [d, f, i, vp]
    lib.dwdrop_bwd.argtypes = [vp] * 3 + [i64] * 2 + [d, f, i, vp]
    lib.dwnorm_fwd.argtypes = [vp] * 10 + [i64] * 3 + [f, f, d, i, vp]
    lib.dwnorm_bwd_workspace_bytes.argtypes = [i64] * 3
    lib.dwnorm_bwd_workspace_bytes.restype = sz
    lib.dwnorm_bwd.argtypes = [vp] * 13 + [sz] + [i64] * 3 + [f, d, i, vp]
    return lib


def err(lib):
    return lib.dw_last_error().decode()


def test_dropout_validation(lib):
    f, g = lib.dwdrop_fwd, lib.dwdrop_bwd
    for p in (-0.1, 1.0, 2.0, NAN):
        assert f(P, N, Q, R, 4, 8, p, 1.0, 0, N) == INVALID and "probability" in err(lib)
        assert g(P, Q, R, 4, 8, p, 1.0, 0, N) == INVALID
    assert f(P, N, Q, N, 4, 8, 0.1, 1.0, 0, N) == INVALID and "rng" in err(lib)
    assert f(P, N, Q, R, 4, 8, 0.1, 1.0, 2, N) == INVALID and "dtype" in err(lib)
    assert f(P, N, Q, R, -4, 8, 0.1, 1.0, 0, N) == INVALID and "negative" in err(lib)
    assert f(N, N, Q, R, 4, 8, 0.1, 1.0, 0, N) == INVALID
    assert g(P, N, R, 4, 8, 0.1, 1.0, 0, N) == INVALID
    assert f(N, N, N, N, 0, 8, 0.0, 1.0, 0, N) == OK and err(lib) == ""
    assert f(N, N, N, R, 4, 0, 0.1, 1.0, 1, N) == OK
    for h in (1 << 40, 1 << 62, (1 << 63) - 1):
        assert f(P, N, Q, R, 4, h, 0.1, 1.0, 0, N) == UNSUPPORTED
        assert f(P, N, Q, R, h, (1 << 31) - 1, 0.1, 1.0, 0, N) == UNSUPPORTED and "too large" in err(lib)


def test_norm_validation(lib):
    f = lib.dwnorm_fwd
    # x, residual, gamma, beta, lengths, rng, y, sum, mean, rstd, B, T, C, eps, alpha, p, dtype, stream
    tail = (1e-5, 1.0, 0.0, 0, N)
    assert f(N, N, N, N, N, N, Q, N, N, N, 2, 3, 8, *tail) == INVALID and "NULL" in err(lib)
    assert f(P, N, N, N, N, N, N, N, N, N, 2, 3, 8, *tail) == INVALID
    assert f(P, N, N, N, N, N, Q, Q, N, N, 2, 3, 8, *tail) == INVALID and "alias" in err(lib)
    assert f(P, N, N, N, N, N, Q, N, N, N, 2, 3, -8, *tail) == INVALID
    assert f(P, N, N, N, N, N, Q, N, N, N, 2, 3, 8193, *tail) == UNSUPPORTED
    assert f(P, N, N, N, N, N, Q, N, N, N, 1 << 20, 1 << 12, 8, *tail) == UNSUPPORTED and "too large" in err(lib)
    assert f(P, N, N, N, N, N, Q, N, N, N, (1 << 63) - 1, 3, 8, *tail) == UNSUPPORTED
    for eps in (-1.0, NAN):
        assert f(P, N, N, N, N, N, Q, N, N, N, 2, 3, 8, eps, 1.0, 0.0, 0, N) == INVALID and "eps" in err(lib)
    assert f(P, N, N, N, N, N, Q, N, N, N, 2, 3, 8, 1e-5, 1.0, 0.5, 0, N) == INVALID and "rng" in err(lib)
    assert f(P, N, N, N, N, N, Q, N, N, N, 2, 3, 8, 1e-5, 1.0, 0.0, 5, N) == INVALID and "dtype" in err(lib)
    assert f(N, N, N, N, N, N, N, N, N, N, 0, 3, 8, *tail) == OK


def test_norm_backward_validation(lib):
    ws = lib.dwnorm_bwd_workspace_bytes
    need = ws(16, 750, 1024)
    assert need > 0 and ws(-1, 2, 3) == 0 and ws(0, 2, 64) == 0 and ws(2, 2, 9000) == 0 and ws(1 << 40, 2, 8) == 0
    f = lib.dwnorm_bwd
    # sum, gamma, lengths, mean, rstd, dy, dsum, rng, dx, dres, dgamma, dbeta, workspace, bytes, B, T, C, alpha, p, ...
    a = (16, 750, 1024, 1.0, 0.0, 0, N)
    assert f(P, N, N, P, P, P, N, N, Q, N, R, N, W, need - 1, *a) == WORKSPACE
    assert f(P, N, N, P, P, P, N, N, Q, N, R, N, N, need, *a) == WORKSPACE and "workspace" in err(lib)
    assert f(P, N, N, P, P, P, N, N, Q, Q, N, N, N, 0, *a) == INVALID and "alias" in err(lib)
    for bad in range(4):
        args = [P, N, N, P, P, P, N, N, Q, N, N, N, N, 0]
        args[(0, 3, 4, 5)[bad]] = N
        assert f(*args, *a) == INVALID
    assert f(P, N, N, P, P, P, N, N, N, N, N, N, N, 0, *a) == OK  # nothing asked for
    assert f(P, N, N, P, P, P, N, N, Q, N, N, N, N, 0, 16, 750, 1024, 1.0, 0.1, 0, N) == INVALID and "rng" in err(lib)
    assert f(P, N, N, P, P, P, N, N, Q, N, N, N, N, 0, 16, 750, 1024, 1.0, 0.0, 3, N) == INVALID


class Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("item", "frame", "head")]


class Attn(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int64) for n in ("B", "Tq", "Tk", "H", "Hkv", "D")] +
                [(n, Strides) for n in ("q", "k", "v", "dq", "dk", "dv")] +
                [(n, ctypes.c_int64) for n in ("buckets", "reach", "left", "right")] +
                [("scale", ctypes.c_float), ("dtype", ctypes.c_int)])


def attn(B=2, Tq=100, Tk=100, H=4, Hkv=2, D=64, buckets=32, reach=128, dtype=0, **more):
    s = Attn(B, Tq, Tk, H, Hkv, D, buckets=buckets, reach=reach, left=-1, right=-1, scale=0.125, dtype=dtype)
    for n, heads, frames in (("q", H, Tq), ("k", Hkv, Tk), ("v", Hkv, Tk), ("dq", H, Tq), ("dk", Hkv, Tk), ("dv", Hkv, Tk)):
        setattr(s, n, Strides(frames * heads * D, heads * D, D))
    for n, v in more.items():
        setattr(s, n, v)
    return s


@pytest.fixture(scope="module")
def alib(lib):
    vp, sz, p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Attn)
    lib.dwattn_rel_buckets.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    for n in ("fwd", "bwd"):
        getattr(lib, f"dwattn_{n}_workspace_bytes").argtypes = [p]
        getattr(lib, f"dwattn_{n}_workspace_bytes").restype = sz
    lib.dwattn_fwd.argtypes = [p] + [vp] * 11 + [sz, vp]
    lib.dwattn_bwd.argtypes = [p] + [vp] * 16 + [sz, vp]
    return lib


BAD_SHAPES = [(dict(B=-1), INVALID), (dict(D=-1), INVALID), (dict(H=3), INVALID), (dict(Hkv=0), INVALID),
              (dict(dtype=2), INVALID), (dict(q=Strides(-1, 1, 1)), INVALID), (dict(buckets=0), INVALID),
              (dict(reach=0), INVALID), (dict(D=129), UNSUPPORTED), (dict(reach=1025), UNSUPPORTED),
              (dict(Tq=(1 << 28) + 1), UNSUPPORTED), (dict(Tk=1 << 40), UNSUPPORTED), (dict(B=1 << 40), UNSUPPORTED),
              (dict(B=1 << 20, H=1 << 10, Hkv=1 << 10), UNSUPPORTED), (dict(k=Strides(1 << 60, 1, 1)), UNSUPPORTED),
              (dict(v=Strides(1, (1 << 62), 1)), UNSUPPORTED)]


def test_attention_validation(alib):
    f = alib.dwattn_fwd
    good = attn()
    # shape, q, k, v, table, map, q_lengths, k_lengths, q_pos, out, lse, workspace, bytes, stream
    for bad, status in BAD_SHAPES:
        assert f(attn(**bad), P, P, P, P, P, N, N, N, Q, N, W, 1 << 40, N) == status, bad
    assert f(None, P, P, P, P, P, N, N, N, Q, N, W, 1 << 40, N) == INVALID
    assert f(good, P, P, P, P, N, N, N, N, Q, N, W, 1 << 40, N) == INVALID and "map" in err(alib)
    assert f(good, P, P, P, N, P, N, N, N, Q, N, W, 1 << 40, N) == INVALID
    for i in (0, 1, 2, 8):
        args = [P, R, S, P, P, N, N, N, Q, N, W, 1 << 40, N]
        args[i] = N
        assert f(good, *args) == INVALID and "NULL" in err(alib)
    for alias in (P, R, S):
        assert f(good, P, R, S, P, P, N, N, N, alias, N, W, 1 << 40, N) == INVALID and "alias" in err(alib)
    few = attn(B=1, Tq=1, Tk=5000)
    need = alib.dwattn_fwd_workspace_bytes(few)
    assert need > 0 and f(few, P, P, P, P, P, N, N, N, Q, N, W, need - 1, N) == WORKSPACE
    assert f(few, P, P, P, P, P, N, N, N, Q, N, N, need, N) == WORKSPACE and "workspace" in err(alib)
    assert alib.dwattn_fwd_workspace_bytes(attn(B=64, Tq=1000, Tk=1000)) == 0
    assert alib.dwattn_fwd_workspace_bytes(attn(D=500)) == 0 and alib.dwattn_fwd_workspace_bytes(None) == 0
    for empty in (dict(B=0), dict(Tq=0), dict(H=0, Hkv=0), dict(D=0)):
        assert f(attn(**empty), N, N, N, N, N, N, N, N, N, N, N, 0, N) == OK


def test_attention_backward_validation(alib):
    f, good = alib.dwattn_bwd, attn()
    big = 1 << 40
    X = [ctypes.c_void_p(0x10000 * i) for i in range(1, 12)]
    # q, k, v, table, map, q_lengths, k_lengths, q_pos, out, lse, dout, dq, dk, dv, dtable, workspace
    a = [X[0], X[1], X[2], X[3], X[4], N, N, N, X[5], X[6], X[7], X[8], X[9], X[10], P, W]
    for bad, status in BAD_SHAPES + [(dict(dq=Strides(-1, 1, 1)), INVALID), (dict(dk=Strides(1 << 60, 1, 1)), UNSUPPORTED),
                                  (dict(B=1 << 16, Tq=1 << 11, H=1, Hkv=1, D=1, reach=1024), UNSUPPORTED)]:
        assert f(attn(**bad), *a, big, N) == status, bad

    def with_(**k):
        names = "q k v table map q_lengths k_lengths q_pos out lse dout dq dk dv dtable workspace".split()
        return [k.get(n, v) for n, v in zip(names, a)]

    for n in ("q", "k", "v", "out", "lse", "dout"):
        assert f(good, *with_(**{n: N}), big, N) == INVALID and "NULL" in err(alib), n
    assert f(good, *with_(table=N, map=N), big, N) == INVALID and "dtable" in err(alib)
    assert f(good, *with_(map=N), big, N) == INVALID
    for n in ("dq", "dk", "dv"):
        for o in (X[0], X[1], X[2], X[5], X[7]):
            assert f(good, *with_(**{n: o}), big, N) == INVALID and "alias" in err(alib)
    assert f(good, *with_(dq=X[9]), big, N) == INVALID and f(good, *with_(dv=X[9]), big, N) == INVALID
    need = alib.dwattn_bwd_workspace_bytes(good)
    assert need > 0 and f(good, *a, need - 1, N) == WORKSPACE and f(good, *with_(workspace=N), need, N) == WORKSPACE
    assert alib.dwattn_bwd_workspace_bytes(attn(reach=2000)) == 0 and alib.dwattn_bwd_workspace_bytes(None) == 0
    assert 0 < alib.dwattn_bwd_workspace_bytes(attn(buckets=0)) < need
    assert f(good, *with_(dq=N, dk=N, dv=N, dtable=N), 0, N) == OK  # nothing asked for
    assert f(attn(B=0), *[N] * 11, Q, R, S, N, N, 0, N) == OK


def test_bucket_map_validation(alib):
    f = alib.dwattn_rel_buckets
    m = (ctypes.c_int32 * 4096)()
    assert f(m, 32, 128, 1) == OK and f(m, 2, 1, 1) == OK and f(m, 1, 1, 0) == OK
    assert f(None, 32, 128, 1) == INVALID and "NULL" in err(alib)
    assert f(m, 1, 128, 1) == INVALID and f(m, 0, 128, 0) == INVALID and f(m, -4, 128, 0) == INVALID
    assert f(m, 32, 8, 1) == INVALID and f(m, 32, 16, 0) == INVALID and f(m, 32, 9, 1) == OK
    assert f(m, 1, 0, 0) == INVALID and f(m, 32, -5, 1) == INVALID
    assert f(m, 32, 1025, 1) == UNSUPPORTED and f(m, 1 << 40, 1 << 50, 1) == UNSUPPORTED


@pytest.mark.parametrize("bidirectional", [0, 1])
def test_bucket_map_is_exact(alib, bidirectional):
    """Distances at which the logarithms' quotient is a whole number, for reaches that are powers, products and primes
    times the exact distances; and every small pair of sizes."""
    m = (ctypes.c_int32 * 4096)()
    sizes = [(n, r) for n in range(1, 41) for r in range(1, 101)]
    sizes += [(5, 1024), (17, 729), (32, 128), (64, 512), (64, 1024), (33, 1024), (128, 1000), (512, 1024)]
    for buckets, reach in sizes:
        if alib.dwattn_rel_buckets(m, buckets, reach, bidirectional) != OK:
            continue
        want = [ref.bucket(r, buckets, reach, bool(bidirectional)) for r in range(-reach, reach + 1)]
        assert list(m[:2 * reach + 1]) == want, (buckets, reach)


def test_more_workgroups_than_a_launch_takes_are_refused(alib):
    """A launch counts its threads in 32 bits: 2^24 workgroups of 256 are too many, and are refused before it."""
    tail = (1e-5, 1.0, 0.0, 0, N)
    for B, T, C in ((1 << 15, 1 << 14, 8), (1 << 12, 1 << 12, 4096), (1 << 13, 1 << 13, 2048)):
        assert alib.dwnorm_fwd(P, N, N, N, N, N, Q, N, N, N, B, T, C, *tail) == UNSUPPORTED and "too large" in err(alib)
    assert alib.dwdrop_fwd(P, N, Q, R, 1 << 34, 8, 0.1, 1.0, 0, N) == UNSUPPORTED and "too large" in err(alib)
    assert alib.dwdrop_bwd(P, Q, R, 1 << 30, 1 << 7, 0.1, 1.0, 0, N) == UNSUPPORTED
    X = [ctypes.c_void_p(0x10000 * i) for i in range(1, 12)]
    for many in (dict(B=1 << 24, H=1, Hkv=1), dict(B=1 << 20, H=1 << 5, Hkv=1), dict(B=1 << 12, H=1 << 12, Hkv=1)):
        for dtype in (0, 1):
            shape = attn(Tq=1, Tk=1, D=1, dtype=dtype, **many)
            assert alib.dwattn_fwd(shape, P, R, S, P, P, N, N, N, Q, N, W, 1 << 40, N) == UNSUPPORTED and "too large" in err(alib)
            assert alib.dwattn_bwd(shape, X[0], X[1], X[2], X[3], X[4], N, N, N, X[5], X[6], X[7], X[8], X[9], X[10], P, W,
                                   1 << 40, N) == UNSUPPORTED and "too large" in err(alib)
            assert alib.dwattn_fwd_workspace_bytes(shape) == 0 and alib.dwattn_bwd_workspace_bytes(shape) == 0
    assert alib.dwattn_bwd(attn(buckets=1 << 23), X[0], X[1], X[2], X[3], X[4], N, N, N, X[5], X[6], X[7], X[8], X[9], X[10],
                           P, W, 1 << 40, N) == UNSUPPORTED


def test_backward_workspace_holds_for_any_context(alib):
    """The binding asks for it without the call's context limits."""
    for B, H, T in ((4, 4, 1000), (10, 8, 375), (3, 4, 333), (24, 8, 750), (30, 8, 100)):
        for D, dtype in ((64, 1), (128, 1), (64, 0), (128, 0)):
            sizes = {alib.dwattn_bwd_workspace_bytes(attn(B=B, H=H, Hkv=H, Tq=T, Tk=T, D=D, dtype=dtype, left=left, right=right))
                     for left, right in ((-1, -1), (-1, 0), (100, -1), (30, 30))}
            assert len(sizes) == 1 and sizes.pop() > 0


def test_workspaces_off_16_bytes_are_refused(alib):
    X = [ctypes.c_void_p(0x10000 * i) for i in range(1, 12)]
    few, good = attn(B=1, Tq=1, Tk=5000), attn()
    for off in (1, 4, 8):
        w = ctypes.c_void_p(0x5000 + off)
        assert alib.dwattn_fwd(few, P, P, P, P, P, N, N, N, Q, N, w, 1 << 40, N) == INVALID and "16 bytes" in err(alib)
        assert alib.dwattn_bwd(good, X[0], X[1], X[2], X[3], X[4], N, N, N, X[5], X[6], X[7], X[8], X[9], X[10], P, w, 1 << 40,
                               N) == INVALID and "16 bytes" in err(alib)
        assert alib.dwnorm_bwd(P, N, N, P, P, P, N, N, Q, N, R, N, w, 1 << 40, 16, 750, 1024, 1.0, 0.0, 0,
                               N) == INVALID and "16 bytes" in err(alib)
