"""Outputs of the recurrence and of the rotated heads that would be written twice are refused on the host, whichever distances collide;
layouts that do not collide are not.  The addresses here are never dereferenced: calls that are not refused end at a missing workspace."""
import itertools

import pytest

from test_recur_abi import INVALID, N, UNSUPPORTED, WORKSPACE, A, err, lib, rope, scan  # noqa: F401

X, R_, G, DECAY, LEN, H0, Y, DY, DH, DX, DR, DG, DD, DH0 = A[:14]


def scan_fwd(lib, shape, y=Y, h_last=N, h0=N):
    return lib.dwscan_fwd(shape, X, R_, G, DECAY, N, h0, y, h_last, N, 0, N)


def scan_bwd(lib, shape, dx=DX, dr=DR, dg=DG, ddecay=DD, dh0=DH0, h0=H0, dh_last=DH):
    return lib.dwscan_bwd(shape, X, R_, G, DECAY, N, h0, Y, DY, dh_last, dx, dr, dg, ddecay, dh0, N, 0, N)


def rope_bwd(lib, shape, dq=A[7], dk=A[8], gq=A[9], gk=A[10]):
    return lib.dwrope_bwd(shape, A[0], A[1], A[2], A[3], A[4], N, N, A[5], A[6], dq, dk, gq, gk, N, 0, N)


def rope_fwd(lib, shape, place=N):
    return lib.dwrope_fwd(shape, A[0], A[1], A[2], A[3], A[4], A[5], N, N, place, A[6], A[7], A[8], N)


def collide(sizes, steps, piece):
    """By trying every pair of places."""
    at = sorted(sum(i * s for i, s in zip(where, steps)) for where in itertools.product(*(range(n) for n in sizes)))
    return any(b - a < piece for a, b in zip(at, at[1:]))


# distances of items and frames, in elements, for 600 frames of 8 channels: enough frames that the forward asks for a workspace
COLLIDING = [[8, 8], [8, 12], [16, 8], [4792, 8], [8, 15], [24, 12], [4799, 8], [9, 10]]
APART = [[4800, 8], [8, 16], [8, 17], [9, 18], [4801, 8], [12, 24], [1 << 40, 9], [8, 1 << 20]]


@pytest.mark.parametrize("steps", COLLIDING + APART)
def test_frames(lib, steps):  # noqa: F811
    bad = steps in COLLIDING
    assert bad == collide((2, 600), steps, 8)
    rest = [4800, 8]
    for got in (scan_fwd(lib, scan(B=2, T=600, strides=rest * 3 + steps + rest * 4)),
                *(scan_bwd(lib, scan(B=2, T=600, strides=rest * (5 + j) + steps + rest * (2 - j))) for j in range(3))):
        assert got == (INVALID if bad else WORKSPACE)
        assert not bad or "overlap" in err(lib)


def test_an_axis_of_one_has_no_distance(lib):  # noqa: F811
    rest = [0, 8]
    assert scan_fwd(lib, scan(B=1, T=600, strides=rest * 8)) == WORKSPACE
    assert scan_bwd(lib, scan(B=600, T=1, strides=[8, 0] * 8)) == WORKSPACE
    assert scan_bwd(lib, scan(B=1, T=1, strides=[0, 0] * 8)) == WORKSPACE


def test_inputs_may_overlap(lib):  # noqa: F811
    assert scan_fwd(lib, scan(B=2, T=600, strides=[8, 8] * 3 + [4800, 8] * 5)) == WORKSPACE
    assert scan_bwd(lib, scan(B=2, T=600, strides=[8, 8] * 5 + [4800, 8] * 3)) == WORKSPACE


HEADS_COLLIDING = [[320, 64, 64], [64, 64, 16], [320, 16, 16], [16, 80, 16], [320, 48, 16], [319, 64, 16], [16, 32, 32], [64, 16, 48],
                   [32, 160, 16]]
HEADS_APART = [[320, 64, 16], [64, 128, 16], [16, 32, 160], [16, 128, 32], [80, 16, 160], [321, 64, 16], [400, 80, 17], [1 << 40, 64, 16]]


@pytest.mark.parametrize("steps", HEADS_COLLIDING + HEADS_APART)
def test_heads(lib, steps):  # noqa: F811
    """Two items of 5 frames of 4 heads of 16."""
    bad = steps in HEADS_COLLIDING
    assert bad == collide((2, 5, 4), steps, 16)
    plain = [320, 64, 16]
    for j in range(2):
        shape = rope(H=4, Hkv=4, strides=plain * (6 + j) + steps + plain * (1 - j))
        assert rope_bwd(lib, shape) == (INVALID if bad else WORKSPACE)
        assert not bad or "overlap" in err(lib)
    if bad:  # the forward has no workspace to end at
        for j in range(3):
            shape = rope(H=4, Hkv=4, strides=plain * (3 + j) + steps + plain * (4 - j))
            assert rope_fwd(lib, shape) == INVALID and "overlap" in err(lib)


def test_caches_are_as_long_as_they_say(lib):  # noqa: F811
    """Two caches of 9 frames 5 frames apart, though 5 frames are written."""
    plain = [320, 64, 16]
    for j in (1, 2):
        shape = rope(H=4, Hkv=4, S=9, strides=plain * 8)
        assert rope_fwd(lib, shape, place=A[9]) == INVALID and "overlap" in err(lib)


def test_states_that_alias(lib):  # noqa: F811
    long = scan(B=2, T=600, strides=[4800, 8] * 8)
    for other in (X, R_, G, Y, DECAY):
        assert scan_fwd(lib, long, h_last=other) == INVALID and "alias" in err(lib)
    assert scan_fwd(lib, long, h_last=H0, h0=H0) == WORKSPACE
    for other in (X, R_, G, DECAY, Y, DY, DX, DR, DG, DD, H0):
        assert scan_bwd(lib, long, dh0=other) == INVALID and "alias" in err(lib)
    assert scan_bwd(lib, long, dh0=DH) == WORKSPACE and scan_bwd(lib, long, dh0=N, h0=N) == WORKSPACE
    for other in (X, R_, G, DECAY, Y, DY, DX, DR, DG, DH0, H0, DH):
        assert scan_bwd(lib, long, ddecay=other) == INVALID and "alias" in err(lib)
    # of no frames only the states and the decay are there
    none = scan(B=2, T=0)
    assert scan_bwd(lib, none, dh0=DD) == INVALID and scan_bwd(lib, none, dh0=X) == WORKSPACE


def test_gammas_gradients_that_alias(lib):  # noqa: F811
    shape = rope(H=4, Hkv=4, strides=[320, 64, 16] * 8)
    for kw in (dict(gq=A[7]), dict(gq=A[8]), dict(gk=A[7]), dict(gk=A[8]), dict(gq=A[10])):
        assert rope_bwd(lib, shape, **kw) == INVALID and "alias" in err(lib)
    assert rope_bwd(lib, shape) == WORKSPACE


def test_far_distances_do_not_wrap(lib):  # noqa: F811
    assert scan_bwd(lib, scan(B=3, T=600, strides=[4800, 8] * 5 + [1 << 58, 8] * 3)) == UNSUPPORTED


def test_outputs_in_a_small_operand(lib):  # noqa: F811
    """decay, lengths, states, weights, frequencies, positions: no output starts where one of them does."""
    long = scan(B=2, T=600, strides=[4800, 8] * 8)
    names = ["x", "r", "g", "decay", "lengths", "h0", "y", "h_last"]

    def fwd(**kw):
        given = dict(zip(names, A)) | kw
        return lib.dwscan_fwd(long, *[given[k] for k in names], N, 0, N)
    assert fwd() == WORKSPACE and fwd(h_last=A[5]) == WORKSPACE
    for k in ("decay", "lengths", "h0"):
        assert fwd(y=A[names.index(k)]) == INVALID and "alias" in err(lib), k
    for k in ("decay", "lengths", "y"):
        assert fwd(h_last=A[names.index(k)]) == INVALID and "alias" in err(lib), k

    back = ["x", "r", "g", "decay", "lengths", "h0", "y", "dy", "dh_last", "dx", "dr", "dg", "ddecay", "dh0"]

    def bwd(**kw):
        given = dict(zip(back, A)) | kw
        return lib.dwscan_bwd(long, *[given[k] for k in back], N, 0, N)
    assert bwd() == WORKSPACE and bwd(dh0=A[8]) == WORKSPACE
    for o in ("dx", "dr", "dg", "ddecay", "dh0"):
        for k in ("decay", "lengths", "h0", "dh_last"):
            if (o, k) != ("dh0", "dh_last"):
                assert bwd(**{o: A[back.index(k)]}) == INVALID and "alias" in err(lib), (o, k)

    heads = ["q", "k", "v", "q_gamma", "k_gamma", "freq", "lengths", "pos", "place", "q_out", "k_out", "v_out"]
    for o in ("q_out", "k_out", "v_out"):  # the forward has no workspace to end at: refusals alone
        for k in ("q_gamma", "k_gamma", "freq", "lengths", "pos", "place"):
            given = dict(zip(heads, A)) | {o: A[heads.index(k)]}
            got = lib.dwrope_fwd(rope(H=4, Hkv=4, strides=[320, 64, 16] * 8), *[given[n] for n in heads], N)
            assert got == INVALID and "alias" in err(lib), (o, k)

    hback = ["q", "k", "q_gamma", "k_gamma", "freq", "lengths", "pos", "dq_out", "dk_out", "dq", "dk", "dq_gamma", "dk_gamma"]

    def heads_bwd(**kw):
        given = dict(zip(hback, A)) | kw
        return lib.dwrope_bwd(rope(H=4, Hkv=4, strides=[320, 64, 16] * 8), *[given[k] for k in hback], N, 0, N)
    assert heads_bwd() == WORKSPACE and heads_bwd(dq=A[7], dk=A[8]) == WORKSPACE and heads_bwd(dq=A[0], dk=A[1]) == WORKSPACE
    for o in ("dq", "dk", "dq_gamma", "dk_gamma"):
        for k in ("q_gamma", "k_gamma", "freq", "lengths", "pos") + (("q", "k", "dq_out", "dk_out") if "gamma" in o else ()):
            assert heads_bwd(**{o: A[hback.index(k)]}) == INVALID and "alias" in err(lib), (o, k)

    for o in range(3):  # y, kept, codes
        out = [A[2 + j] if j != o else A[1] for j in range(3)]
        assert lib.dwact_fwd(1, A[0], A[1], *out, 2, 3, 8, 0, N) == INVALID and "alias" in err(lib)
    for o in range(2):  # dx, y
        out = [A[4 + j] if j != o else A[2] for j in range(2)]
        assert lib.dwact_bwd(1, A[0], A[1], A[2], A[3], *out, 2, 3, 8, 0, N) == INVALID and "alias" in err(lib)
