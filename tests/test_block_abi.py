"""The encoder block's entry points refuse bad arguments on the host, before
anything touches a GPU (the addresses here are never dereferenced)."""
import ctypes
import os

import pytest

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
