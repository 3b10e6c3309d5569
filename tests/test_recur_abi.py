"""The recurrence, the rotated heads and the kept activations refuse bad
arguments on the host, before anything touches a GPU (the addresses here are
never dereferenced), and the 64-bit forms that the GPU tests use agree with
differences and with hand-worked values."""
import ctypes
import math
import os
import struct

import numpy as np
import pytest

import recur_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "conv_subsampling_amd", "libdwconv.so")
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, -1, -2, -3
A = [ctypes.c_void_p(0x1000 * i) for i in range(1, 20)]
N = None
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    lib = ctypes.CDLL(LIB)
    vp, sz, i, i64, cp = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_char_p
    lib.dw_last_error.restype = cp
    for f in ("dwscan_fwd_workspace_bytes", "dwscan_bwd_workspace_bytes", "dwrope_bwd_workspace_bytes"):
        getattr(lib, f).argtypes, getattr(lib, f).restype = [cp], sz
    lib.dwscan_fwd.argtypes = [cp] + [vp] * 9 + [sz, vp]
    lib.dwscan_bwd.argtypes = [cp] + [vp] * 15 + [sz, vp]
    lib.dwrope_fwd.argtypes = [cp] + [vp] * 13
    lib.dwrope_bwd.argtypes = [cp] + [vp] * 14 + [sz, vp]
    lib.dwact_fwd.argtypes = [i] + [vp] * 5 + [i64] * 3 + [i, vp]
    lib.dwact_bwd.argtypes = [i] + [vp] * 6 + [i64] * 3 + [i, vp]
    return lib


def err(lib):
    return lib.dw_last_error().decode()


def scan(B=2, T=5, C=8, strides=None, scale=8.0, dtype=0):
    return struct.pack("=19qfi", B, T, C, *(strides or [T * C, C] * 8), scale, dtype)


def rope(B=2, T=5, H=4, Hkv=2, D=16, R=16, S=5, strides=None, eps=1e-6, pairs=0, dtype=0):
    return struct.pack("=31qfii4x", B, T, H, Hkv, D, R, S, *(strides or [T * H * D, H * D, D] * 8), eps, pairs, dtype)


def test_scan_forward_validation(lib):
    def f(shape=scan(), x=A[0], r=A[1], g=A[2], decay=A[3], y=A[4], h=N, ws=N, n=0):
        return lib.dwscan_fwd(shape, x, r, g, decay, N, N, y, h, ws, n, N)
    for bad in (scan(B=-1), scan(T=-1), scan(C=-1)):
        assert f(bad) == INVALID and "negative size" in err(lib)
    for at in range(8):
        s = [40, 8] * 8
        s[at] = -8
        assert f(scan(strides=s)) == INVALID and "stride" in err(lib)
    for s in (0.0, -1.0, NAN, INF):
        assert f(scan(scale=s)) == INVALID and "scale" in err(lib)
    for d in (-1, 2, 1 << 30):
        assert f(scan(dtype=d)) == INVALID and "dtype" in err(lib)
    assert f(N) == INVALID
    for kw in (dict(x=N), dict(r=N), dict(g=N), dict(decay=N), dict(y=N)):
        assert f(**kw) == INVALID and "NULL" in err(lib)
    for kw in (dict(y=A[0]), dict(y=A[1]), dict(y=A[2])):
        assert f(**kw) == INVALID and "alias" in err(lib)
    assert f(scan(B=1 << 31)) == UNSUPPORTED and f(scan(T=1 << 31)) == UNSUPPORTED and f(scan(C=1 << 31)) == UNSUPPORTED
    assert f(scan(B=(1 << 31) - 1, T=(1 << 31) - 1, C=(1 << 31) - 1)) == UNSUPPORTED
    assert f(scan(strides=[40, 1 << 23] + [40, 8] * 7)) == UNSUPPORTED
    assert f(scan(strides=[1 << 58, 8] + [40, 8] * 7)) == UNSUPPORTED
    # an axis of one has no distance; what holds nothing needs nothing
    assert f(scan(B=0), N, N, N, N, N) == OK and f(scan(C=0), N, N, N, N, N) == OK and f(scan(T=0), N, N, N, N, N) == OK
    long = scan(B=1, T=6000, C=64)
    need = lib.dwscan_fwd_workspace_bytes(long)
    assert need > 0 and lib.dwscan_fwd_workspace_bytes(scan()) == 0 and lib.dwscan_fwd_workspace_bytes(scan(B=-1)) == 0
    assert f(long) == WORKSPACE and f(long, ws=A[5], n=need - 1) == WORKSPACE
    assert f(long, ws=ctypes.c_void_p(0x5008), n=need) == INVALID and "16" in err(lib)


def test_scan_backward_validation(lib):
    names = ["x", "r", "g", "decay", "lengths", "h0", "y", "dy", "dh_last", "dx", "dr", "dg", "ddecay", "dh0"]
    big = 1 << 20

    def f(shape=scan(), n=big, ws=A[18], **kw):
        given = {k: v for k, v in zip(names, A)} | {"lengths": N} | kw
        return lib.dwscan_bwd(shape, *[given[k] for k in names], ws, n, N)
    for bad in (scan(B=-1), scan(scale=NAN), scan(dtype=7), scan(strides=[40, 8] * 7 + [-1, 8])):
        assert f(bad) == INVALID
    for k in ("x", "r", "g", "decay", "y", "dy"):
        assert f(**{k: N}) == INVALID and "NULL" in err(lib)
    for o in ("dx", "dr", "dg"):
        for k in ("x", "r", "g", "y", "dy"):
            assert f(**{o: A[names.index(k)]}) == INVALID and "alias" in err(lib)
    assert f(dx=A[10]) == INVALID and f(dr=A[11]) == INVALID and f(dg=A[9]) == INVALID
    assert f(ddecay=A[3]) == INVALID and f(dh0=A[5]) == INVALID
    assert f(scan(T=1 << 31)) == UNSUPPORTED
    need = lib.dwscan_bwd_workspace_bytes(scan())
    assert need > 0 and f(n=need - 1) == WORKSPACE and f(ws=N, n=0) == WORKSPACE
    assert f(ws=ctypes.c_void_p(0x8004)) == INVALID
    none = dict(dx=N, dr=N, dg=N, ddecay=N, dh0=N)
    assert f(**none) == OK and f(scan(B=0), ddecay=N) == OK and f(scan(C=0)) == OK
    assert lib.dwscan_bwd_workspace_bytes(scan(T=1 << 31)) == 0 and lib.dwscan_bwd_workspace_bytes(N) == 0


def test_rope_validation(lib):
    def f(shape=rope(), q=A[0], k=A[1], v=A[2], freq=A[5], place=N, qo=A[6], ko=A[7], vo=A[8]):
        return lib.dwrope_fwd(shape, q, k, v, A[3], A[4], freq, N, N, place, qo, ko, vo, N)
    for bad in (rope(B=-1), rope(T=-1), rope(H=-1), rope(Hkv=-1), rope(D=0), rope(D=-1), rope(R=-2)):
        assert f(bad) == INVALID and "size" in err(lib)
    assert f(rope(R=15)) == INVALID and f(rope(R=18)) == INVALID and "pairs" in err(lib)
    assert f(rope(pairs=2)) == INVALID and f(rope(pairs=-1)) == INVALID
    assert f(rope(eps=-1e-6)) == INVALID and f(rope(eps=NAN)) == INVALID and "eps" in err(lib)
    assert f(rope(dtype=3)) == INVALID
    assert f(rope(D=129, R=128)) == UNSUPPORTED and "128" in err(lib)
    assert f(freq=N) == INVALID and "freq" in err(lib)
    for kw in (dict(q=N), dict(k=N), dict(qo=N), dict(ko=N), dict(v=N), dict(vo=N)):
        assert f(**kw) == INVALID
    for kw in (dict(qo=A[1]), dict(qo=A[2]), dict(ko=A[0]), dict(ko=A[2]), dict(vo=A[2]), dict(vo=A[0]), dict(vo=A[1]),
               dict(qo=A[7]), dict(ko=A[8]), dict(vo=A[6]), dict(ko=A[1], place=A[9])):
        assert f(**kw) == INVALID and "alias" in err(lib), kw
    other = [320, 64, 16] * 3 + [640, 128, 16] * 5
    assert f(rope(strides=other), qo=A[0]) == INVALID and f(rope(strides=other), ko=A[1]) == INVALID
    for at in (0, 4, 10, 17):
        s = [320, 64, 16] * 8
        s[at] = -1
        assert f(rope(strides=s)) == INVALID and "stride" in err(lib)
    assert f(rope(B=1 << 31)) == UNSUPPORTED and f(rope(T=(1 << 31) - 1, B=(1 << 31) - 1)) == UNSUPPORTED
    assert f(rope(strides=[1 << 58, 64, 16] * 8)) == UNSUPPORTED
    assert f(rope(S=-1), place=A[9]) == INVALID
    assert f(rope(B=0), N, N, N, N, N, N, N, N) == INVALID  # no freq
    assert f(rope(B=0), q=N, k=N, v=N, qo=N, ko=N, vo=N) == OK
    assert f(rope(T=0), q=N, k=N, v=N, qo=N, ko=N, vo=N) == OK

    def g(shape=rope(), q=A[0], k=A[1], freq=A[4], dqo=A[5], dko=A[6], dq=A[7], dk=A[8], gq=A[9], gk=A[10], ws=A[11], n=1 << 20):
        return lib.dwrope_bwd(shape, q, k, A[2], A[3], freq, N, N, dqo, dko, dq, dk, gq, gk, ws, n, N)
    for bad in (rope(B=-1), rope(R=3), rope(pairs=5), rope(eps=NAN), rope(dtype=2), rope(strides=[320, 64, 16] * 7 + [-1, 1, 1])):
        assert g(bad) == INVALID
    for kw in (dict(q=N), dict(k=N), dict(dqo=N), dict(dko=N), dict(freq=N)):
        assert g(**kw) == INVALID and ("freq" if "freq" in kw else "NULL") in err(lib)
    for kw in (dict(dq=A[1]), dict(dq=A[6]), dict(dq=A[8]), dict(dk=A[0]), dict(dk=A[5]), dict(gq=A[10])):
        assert g(**kw) == INVALID and "alias" in err(lib), kw
    mixed = [320, 64, 16] * 6 + [640, 128, 16] * 2
    for kw in (dict(dq=A[0]), dict(dq=A[5]), dict(dk=A[1]), dict(dk=A[6])):
        assert g(rope(strides=mixed), **kw) == INVALID
    need = lib.dwrope_bwd_workspace_bytes(rope())
    assert need > 0 and g(n=need - 1) == WORKSPACE and g(ws=N, n=0) == WORKSPACE and g(ws=ctypes.c_void_p(0x8008)) == INVALID
    assert g(dq=N, dk=N, gq=N, gk=N) == OK and g(rope(B=0), gq=N, gk=N) == OK
    assert lib.dwrope_bwd_workspace_bytes(rope(D=200)) == 0 and lib.dwrope_bwd_workspace_bytes(N) == 0


def test_outputs_that_overlap_are_refused(lib):
    """Distances of an output shorter than what is written there; an input may have them, and an axis of one has none."""
    def fwd(strides, **kw):
        return lib.dwscan_fwd(scan(strides=strides, **kw), A[0], A[1], A[2], A[3], N, N, A[4], N, N, 0, N)

    def bwd(strides, **out):
        o = [out.get(k, A[9 + j]) for j, k in enumerate(("dx", "dr", "dg"))]
        return lib.dwscan_bwd(scan(strides=strides), A[0], A[1], A[2], A[3], N, N, A[6], A[7], N, *o, N, N, N, 0, N)
    for bad in ([0, 8], [40, 0], [7, 8], [40, 7]):
        assert fwd([40, 8] * 3 + bad + [40, 8] * 4) == INVALID and "overlap" in err(lib)
        for j, k in enumerate(("dx", "dr", "dg")):
            s = [40, 8] * 5 + [40, 8] * j + bad + [40, 8] * (2 - j)
            assert bwd(s) == INVALID and "overlap" in err(lib)
            assert bwd(s, **{k: N}) == WORKSPACE  # not written, so the next check answers
    long = scan(B=1, T=6000, C=64, strides=[0, 64] * 8)
    assert lib.dwscan_fwd(long, A[0], A[1], A[2], A[3], N, N, A[4], N, N, 0, N) == WORKSPACE
    assert bwd([0, 0] * 5 + [40, 8] * 3) == WORKSPACE

    def rope_fwd(j, bad):
        return lib.dwrope_fwd(rope(strides=[320, 64, 16] * (3 + j) + bad + [320, 64, 16] * (4 - j)), A[0], A[1], A[2], A[3], A[4],
                              A[5], N, N, N, A[6], A[7], A[8], N)

    def rope_bwd(j, bad):
        return lib.dwrope_bwd(rope(strides=[320, 64, 16] * (6 + j) + bad + [320, 64, 16] * (1 - j)), A[0], A[1], A[2], A[3], A[4],
                              N, N, A[5], A[6], A[7], A[8], N, N, N, 0, N)
    for bad in ([15, 64, 16], [0, 64, 16], [320, 0, 16], [320, 64, 15], [320, 64, 0]):
        for j in range(3):
            assert rope_fwd(j, bad) == INVALID and "overlap" in err(lib)
        for j in range(2):
            assert rope_bwd(j, bad) == INVALID and "overlap" in err(lib)


def test_act_validation(lib):
    def f(act=1, x=A[0], y=A[1], kept=A[2], codes=A[3], B=2, T=3, C=8, dtype=0):
        return lib.dwact_fwd(act, x, N, y, kept, codes, B, T, C, dtype, N)

    def g(act=1, kept=A[2], codes=A[3], dy=A[4], dx=A[5], y=A[6], B=2, T=3, C=8, dtype=0):
        return lib.dwact_bwd(act, kept, codes, N, dy, dx, y, B, T, C, dtype, N)
    for h in (f, g):
        for kw in (dict(act=3), dict(act=-1), dict(dtype=2), dict(B=-1), dict(T=-1), dict(C=-1)):
            assert h(**kw) == INVALID
        for kw in (dict(B=1 << 31), dict(T=1 << 31), dict(C=(1 << 31) - 1), dict(B=1 << 30, T=1 << 30), dict(T=1 << 30, C=1 << 30)):
            assert h(**kw) == UNSUPPORTED, kw
        for kw in (dict(B=0), dict(T=0), dict(C=0)):
            assert h(**kw) == OK
    assert f(x=N) == INVALID and f(kept=N) == INVALID and f(codes=N) == INVALID and f(y=N, kept=N, codes=N) == OK
    assert f(2, y=A[0]) == INVALID and f(kept=A[0]) == INVALID and f(codes=A[1]) == INVALID and f(codes=A[2]) == INVALID
    assert g(kept=N) == INVALID and g(codes=N) == INVALID and g(dy=N) == INVALID and g(dx=N, y=N) == OK
    assert g(2, dx=A[4]) == INVALID and g(dx=A[6]) == INVALID and g(dx=A[2]) == INVALID and g(y=A[3]) == INVALID and g(y=A[4]) == INVALID


# ---------------------------------------------------------------------------
# The 64-bit forms themselves
# ---------------------------------------------------------------------------
def central(f, at, step=1e-6):
    out = np.zeros_like(at)
    for k in np.ndindex(at.shape):
        keep = at[k]
        at[k] = keep + step
        up = f()
        at[k] = keep - step
        out[k] = (up - f()) / (2 * step)
        at[k] = keep
    return out


def test_scan_forms_against_differences():
    rng = np.random.RandomState(0)
    B, T, C, L = 2, 6, 3, [6, 4]
    x, r, g, dy = (rng.randn(B, T, C) for _ in range(4))
    decay, h0, dh = rng.randn(C) - 2, rng.randn(B, C), rng.randn(B, C)

    def loss():
        y, h, *_ = ref.scan_fwd(x, r, g, decay, L, h0)
        return float((y * dy).sum() + (h * dh).sum())
    got = ref.scan_bwd(x, r, g, decay, ref.scan_fwd(x, r, g, decay, L, h0)[0], dy, L, h0, dh)
    for n, at in (("dx", x), ("dr", r), ("dg", g), ("ddecay", decay), ("dh0", h0)):
        assert np.abs(got[n] - central(loss, at)).max() < 1e-7, n


def test_scan_by_hand():
    """softplus(log(e^(ln 2 / 4) - 1)) = ln 2 / 4, so with an open gate half of sigmoid(0) and scale 8 the decay is 1/2."""
    decay = np.array([math.log(math.expm1(math.log(2) / 4))])
    y, h, *_ = ref.scan_fwd(np.ones((1, 2, 1)), np.zeros((1, 2, 1)), np.zeros((1, 2, 1)), decay, None, np.array([[4.0]]))
    step = math.sqrt(0.75) / 2
    assert np.allclose(y[0, :, 0], [2 + step, 1 + 1.5 * step]) and np.allclose(h, y[:, -1])


@pytest.mark.parametrize("kind", ["halves", "neighbours"])
@pytest.mark.parametrize("R", [0, 4, 6])
def test_rope_forms_against_differences(kind, R):
    rng = np.random.RandomState(R)
    x, d, gamma = rng.randn(2, 3, 2, 7), rng.randn(2, 3, 2, 7), rng.randn(7)
    freq, L, pos = 1.0 / (1 + np.arange(R // 2)), [3, 2], [5, 1000]

    def loss():
        return float((ref.rope_fwd(x, gamma, freq, L, pos, kind, 1e-3)[0] * d).sum())
    dx, _, dg, _ = ref.rope_bwd(x, gamma, freq, L, pos, kind, 1e-3, d)
    assert np.abs(dx - central(loss, x)).max() < 1e-7 and np.abs(dg - central(loss, gamma)).max() < 1e-7


def test_rope_by_hand():
    """A quarter turn takes (a, b) to (-b, a)."""
    x = np.array([3.0, 4.0, 5.0, 6.0]).reshape(1, 1, 1, 4)
    norm = math.sqrt((9 + 16 + 25 + 36) / 4)
    for kind, want in (("halves", [-5.0, -6.0, 3.0, 4.0]), ("neighbours", [-4.0, 3.0, -6.0, 5.0])):
        out, _ = ref.rope_fwd(x, None, np.full(2, math.pi / 2), None, [1], kind, 0.0)
        assert np.allclose(out[0, 0, 0] * norm, want)


def test_pack_by_hand():
    x = np.zeros((6, 33))
    x[0, :2], x[1, 0], x[2, 0], x[3, 32], x[4, 0] = (127.0, -64.5), 127.5, 2.0 ** -140, -3.0, np.inf
    kept, codes = ref.pack(x, 1)
    assert codes[:5].tolist() == [[127, 1], [128, 1], [1, 1], [1, 122], [255, 1]]
    assert kept[0, :2].tolist() == [127, -64] and kept[1, 0] == 64 and kept[2, 0] == 0 and kept[3, 32] == -96
    assert not kept[4:].any() and np.isnan(ref.unpack(kept, codes, 1)[4, :32]).all()


@pytest.mark.parametrize("kind", ["none", "silu", "glu"])
def test_act_forms_against_differences(kind):
    rng = np.random.RandomState(3)
    x, dy = 2 * rng.randn(3, 4), rng.randn(3, 2 if kind == "glu" else 4)
    assert np.abs(ref.act_grad(x, dy, kind)[0] - central(lambda: float((ref.act(x, kind) * dy).sum()), x)).max() < 1e-8
