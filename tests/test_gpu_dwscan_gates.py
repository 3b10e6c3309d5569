"""The recurrence where its factors are small: decays near 0, closed halves of
the gates, and the gates themselves, against the definition in 64 bits.

Tolerances count roundings of 2^-24 (U), as in test_gpu_dwscan.py, in sums that
keep no term above what is left of it.  In float32 a gate is off by 8 U: its
exponential by 2 of the instruction, 1 of the product that mends its exponent
and 1 of that factor, the sum 1, the reciprocal 2.  The rate is off by 8, so w by 17; a thread's
sum of 16 of them by 16 more: 40 U of w bend a product of decays.  1 - a is a
series of 4 U, sqrt(1 - a^2) another 4, the products of a term 8: 40 U with
the gates'.  bf16 gates are those of one rounded product, |r| U more.
Products of decays below 2^-126 are flushed, twice on a state's way at most: 4 of them times the largest value that
they scale.
"""
import numpy as np
import pytest
import torch

import datagen
import recur_exact as exact
from test_gpu_dwscan import BF16, DEV, F32, NAMES, U, grads, h, lib, say, within

pytestmark = pytest.mark.gpu


def rel(dt):
    return 40 if dt == F32 else 64


def check(s):
    """Forward and gradients of s against 64 bits."""
    dt, T, e = s["dt"], s["T"], rel(s["dt"])
    got = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"])
    back = grads(s, got[0])
    torch.cuda.synchronize()
    y, last, ys, ls, yb, lb = exact.scan_fwd(*(h(s[k]) for k in ("x", "r", "g", "decay", "lengths", "h0")))
    n = e + 40 + 2 * (-(-T // 64))
    held, back_held = (4 * 2.0 ** -126 * max(float(s[k].abs().max()) for k in keys) for keys in (("x", "h0"), ("dy", "dh_last")))
    within(got[0], y, U * (n * ys + e * yb) + held, dt, "y")
    within(got[1], last, U * (n * ls + e * lb) + held, F32, "h_last")
    want = exact.scan_bwd(*(h(s[k]) for k in ("x", "r", "g", "decay")), h(got[0]), h(s["dy"]), h(s["lengths"]), h(s["h0"]),
                          h(s["dh_last"]))
    # a gradient of a gate multiplies what is carried by a value held and by w, under 32
    held = {"dx": back_held, "dh0": back_held, "dg": back_held * float(s["x"].abs().max())}
    held["dr"] = 32 * back_held * max(float(s[k].abs().max()) for k in ("x", "h0"))
    held["ddecay"] = held["dr"] * s["B"] * T
    for name, g in zip(NAMES, back):
        n = 2 * e + 64 + 2 * (-(-T // 64)) + (T // 16 + 32 if name == "ddecay" else 0)
        within(g, want[name], U * (n * want[name + "_size"] + e * want[name + "_bent"]) + held[name],
               dt if name in ("dx", "dr", "dg") else F32, name)


def spikes(shape, name):
    """Large values at one frame in three, zeros between: what is left of them is all there is."""
    at = datagen.uniform(shape, 0.0, 3.0, name + "/at", device=DEV) < 1
    return datagen.normal(shape, 1e8, name, device=DEV) * at


# one thread's run, a wave, a tile, several tiles in turn and linked ones, in both directions
FRAMES = [1, 3, 8, 12, 40, 130, 300, 700, 1500]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", FRAMES)
def test_decays_near_zero_keep_their_digits(T, dt):
    """-log of the decay from 3 to 25 a frame: a state of 1e6 leaves 5e4 to 1e-5."""
    B, C = 3, 70
    n = lambda name, var=1.0: datagen.normal((B, T, C), var, f"near/{T}/{name}", device=DEV).to(dt)  # noqa: E731
    s = dict(B=B, T=T, C=C, dt=dt, r=n("r", 0.04), g=n("g"), x=spikes((B, T, C), f"near/{T}/x").to(dt),
             dy=spikes((B, T, C), f"near/{T}/dy").to(dt), lengths=torch.tensor([T, max(0, T - 2), T // 2], dtype=torch.int32, device=DEV))
    w = datagen.uniform((C,), 3.0, 25.0, "near/w", device=DEV).double()
    s["decay"] = torch.log(torch.expm1(w / 4)).float()
    s["h0"], s["dh_last"] = (datagen.normal((B, C), 1e12, f"near/{k}", device=DEV) for k in ("h0", "dh"))
    say("scan near zero", T, dt)
    check(s)


@pytest.mark.parametrize("w", [0.3, 0.69, 0.6931, 0.6932, 0.7, 5.0, 14.0, 16.0, 17.0, 17.5, 20.0, 60.0])
def test_what_one_step_leaves(w):
    """a h0 by itself, from the first frame to the last of a run, and the same of the gradient."""
    T, C = 24, 64
    zero = torch.zeros((1, T, C), device=DEV)
    h0 = datagen.normal((1, C), 1e12, "left/h0", device=DEV)
    decay = torch.full((C,), float(np.log(np.expm1(w / 4))), device=DEV)
    y, last = lib().dwscan_fwd(zero, zero, zero, decay, h0=h0)
    _, _, _, _, dh0 = lib().dwscan_bwd(zero, zero, zero, decay, y, zero, h0=h0, dh_last=h0)
    rate = 4 * np.log1p(np.exp(h(decay)))
    left = h(h0)[:, None] * np.exp(-rate * (1 + np.arange(T))[:, None])
    bound = U * (40 + 40 * rate * (1 + np.arange(T))[:, None]) * np.abs(left) + 1e-31  # 2^-126 of a million is where decays end
    assert (np.abs(h(y) - left) <= bound).all()
    assert (np.abs(h(last) - left[:, -1]) <= bound[:, -1]).all() and (np.abs(h(dh0) - left[:, -1]) <= bound[:, -1]).all()


@pytest.mark.parametrize("dt,top", [(F32, 80.0), (F32, 20.0), (BF16, 20.0)], ids=["f32-80", "f32-20", "bf16-20"])
@pytest.mark.parametrize("T", [1, 12, 130, 700])
def test_the_closed_halves_of_gates_keep_their_digits(T, dt, top):
    """Gates of both signs up to 20 and 80: 1 - sigmoid of down to 2e-35 scales their gradients."""
    B, C = 2, 70

    def gate(name):
        v = datagen.uniform((B, T, C), 4.0, top, f"shut/{T}/{top}/{name}", device=DEV)
        return (v * torch.sign(datagen.normal((B, T, C), 1.0, f"shut/{T}/{top}/{name}/sign", device=DEV))).to(dt)
    n = lambda name: datagen.normal((B, T, C), 1.0, f"shut/{T}/{name}", device=DEV).to(dt)  # noqa: E731
    s = dict(B=B, T=T, C=C, dt=dt, r=gate("r"), g=gate("g"), x=n("x"), dy=n("dy"), lengths=None,
             decay=datagen.uniform((C,), -8.0, 0.0, "shut/decay", device=DEV))
    s["h0"], s["dh_last"] = (datagen.normal((B, C), 1.0, f"shut/{k}", device=DEV) for k in ("h0", "dh"))
    say("scan closed halves", T, dt, top)
    check(s)


def test_a_slow_channel_has_the_whole_gate():
    """softplus(decay) = 1e-31: a rate that small is still w's own, and 1 - sigmoid(r) does not come from it."""
    C = 64
    r = datagen.uniform((1, 1, C), -3.0, 12.0, "slow/r", device=DEV)
    one, decay = torch.ones((1, 1, C), device=DEV), torch.full((C,), -71.4, device=DEV)
    h0 = torch.zeros((1, C), device=DEV)
    y, _ = lib().dwscan_fwd(one, r, one, decay, h0=h0)
    _, dr, _, _, _ = lib().dwscan_bwd(one, r, one, decay, y, one, h0=h0)
    want = exact.scan_bwd(h(one), h(r), h(one), h(decay), h(y), h(one), None, h(h0))
    within(dr, want["dr"], U * 144 * want["dr_size"], F32, "dr")


def test_float_gates():
    """Both gates by themselves, from -80 to 80.  With a = 0 and x = 1 an output is sigmoid(g): 8 U.  With g = 100 it is
    sqrt(1 - a^2): w is off by 8 of the gate and 2 of rate and product, the series and 1 - a^2 by 6, the root halves both and adds 2:
    10 U (softplus(30) is 30 and 1e-13)."""
    C = 4096
    v = datagen.uniform((1, 1, C), -80.0, 80.0, "gate/v", device=DEV)
    one = torch.ones_like(v)
    y, _ = lib().dwscan_fwd(one, one * 100, v, torch.full((C,), 1e4, device=DEV))
    want = exact.sigmoid(h(v))
    assert (np.abs(h(y) - want) <= 8 * U * want).all()
    y, _ = lib().dwscan_fwd(one, v, one * 100, torch.full((C,), 30.0, device=DEV), scale=1.0)
    want = np.sqrt(-np.expm1(-60 * want))
    assert (np.abs(h(y) - want) <= 10 * U * want).all()


def test_float_gates_of_infinity_and_nan():
    v = torch.tensor([float("inf"), -float("inf"), float("nan"), 3e38, -3e38, 200.0, -200.0], device=DEV).view(1, 1, 7)
    one, decay = torch.ones_like(v), torch.full((7,), 1e4, device=DEV)
    y, _ = lib().dwscan_fwd(one, one, v, decay)
    assert y[0, 0, [0, 3, 5]].tolist() == [1.0] * 3 and y[0, 0, [1, 4, 6]].tolist() == [0.0] * 3 and y[0, 0, 2].isnan()
    y, _ = lib().dwscan_fwd(one * 0, v, one, decay, h0=torch.ones((1, 7), device=DEV))
    assert y[0, 0, [0, 3, 5]].tolist() == [0.0] * 3 and y[0, 0, [1, 4, 6]].tolist() == [1.0] * 3 and y[0, 0, 2].isnan()
    back = lib().dwscan_bwd(one, v, v, decay, y, one)
    for t in back[:3]:
        assert t[0, 0, [0, 1, 3, 4, 5, 6]].isfinite().all()
