"""Layer norm with the residual add and dropout in front of it, and dropout
alone, against the definitions in 64 bits.

Tolerances.  Forward and dx, dres are float32 arithmetic on unit-scale rows:
each value passes through fewer than 60 roundings of quantities of the size of
the row's largest, and 1e-5 * (1 + |ref|) is over twice that.  bf16 storage
adds one rounding, at most 2^-8 of the value.  The weight gradients are sums:
no term passes through more than 60 float32 roundings of partial sums that the
sum of the absolute terms bounds, then fp64.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import datagen
from gpu_util import Guarded, host64, say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16


def lib():
    import conv_subsampling_amd as dw
    return dw


def near(got, want, dt, what, extra=0.0):
    g = host64(got)
    assert g.shape == want.shape, what
    tol = 1e-5 * (1 + np.abs(want)) + extra + (ref.U16 * np.abs(want) if dt == BF16 else 0.0)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.abs(g - want)[bad].max():.3e} at {np.argwhere(bad)[0]}"


def make(B, T, C, dt, residual=True, p=0.1, alpha=0.5, seed=0, lengths=None):
    tag = f"norm/{B}/{T}/{C}/{seed}"
    n = lambda shape, name, var=1.0: datagen.normal(shape, var, f"{tag}/{name}", device=DEV).to(dt)  # noqa: E731
    s = dict(B=B, T=T, C=C, dt=dt, p=p, alpha=alpha, x=n((B, T, C), "x"), gamma=n((C,), "g"), beta=n((C,), "b"),
             residual=n((B, T, C), "r", 2.0) if residual else None, dy=n((B, T, C), "dy"),
             dsum=n((B, T, C), "ds") if residual else None)
    L = list(range(T, T - B, -1)) if lengths is None else lengths
    s["lengths"] = torch.tensor(L, dtype=torch.int32, device=DEV)
    s["seed"], s["stream"] = 0x1234_5678_9ABC_DEF0 + seed, 77 + seed
    s["rng"] = torch.tensor([s["seed"], s["stream"]], dtype=torch.int64, device=DEV) if p else None
    s["factor"] = ref.drop_factor(B * T, C, s["seed"], s["stream"], p).reshape(B, T, C) if p else np.ones((B, T, C))
    return s


def h(t):
    return None if t is None else host64(t)


def check_fwd(s, got=None):
    got = got or lib().dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=s["rng"],
                                  p=s["p"], alpha=s["alpha"], sum=torch.empty_like(s["x"]))
    torch.cuda.synchronize()
    want = ref.norm_fwd(h(s["x"]), h(s["gamma"]), h(s["beta"]), h(s["lengths"]), h(s["residual"]), s["factor"], s["alpha"])
    for name, g, w in zip(("y", "s", "mean", "rstd"), got, want):
        near(g, w, s["dt"] if name in "ys" else F32, name)
    for name, g, w in zip("ys", got, want):  # frames past the length are exact zeros
        dead = np.arange(s["T"])[None, :] >= np.clip(h(s["lengths"]), 0, s["T"])[:, None]
        assert not host64(g)[dead].any(), name
    return got, want


def check_bwd(s, total, mean, rstd, need=("dx", "dres", "dgamma", "dbeta")):
    got = lib().dwnorm_bwd(total, s["gamma"], s["lengths"], mean, rstd, s["dy"], dsum=s["dsum"], rng=s["rng"], p=s["p"],
                           alpha=s["alpha"], need=need)
    torch.cuda.synchronize()
    dx, dres, dg, db, ag, ab = ref.norm_bwd(h(total), h(s["gamma"]), h(s["lengths"]), h(mean), h(rstd), h(s["dy"]),
                                            h(s["dsum"]), s["factor"], s["alpha"])
    big = np.abs(dres).max(initial=1.0)
    for name, g, w, extra in (("dx", got[0], dx, 1e-5 * big), ("dres", got[1], dres, 1e-5 * big),
                              ("dgamma", got[2], dg, 60 * ref.U32 * ag), ("dbeta", got[3], db, 60 * ref.U32 * ab)):
        assert (g is not None) == (name in need)
        if g is not None:
            near(g, w, s["dt"] if name in ("dx", "dres") else F32, name, extra)
    return got


# widths of every form: partial groups, rows that share a wave, one group a lane, several, a row per workgroup
WIDTHS = [1, 3, 7, 8, 50, 64, 65, 128, 200, 256, 333, 512, 1000, 1024, 1025, 2048, 2100, 4096, 4097, 8191, 8192]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", WIDTHS)
def test_norm_forward_and_backward(C, dt):
    B, T = (3, 23) if C <= 2048 else (2, 5)
    for residual, p, alpha in ((True, 0.1, 0.5), (False, 0.0, 1.0)):
        s = make(B, T, C, dt, residual, p, alpha)
        say("norm", C, dt, residual, p)
        got, want = check_fwd(s)
        check_bwd(s, got[1], got[2], got[3])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_training_batch_and_many_rows(dt):
    for B, T, C in ((4, 375, 1024), (5, 333, 200), (40, 200, 8)):
        s = make(B, T, C, dt, lengths=[T - 7 * b for b in range(B)])
        say("norm batch", B, T, C, dt)
        got, _ = check_fwd(s)
        check_bwd(s, got[1], got[2], got[3])


@pytest.mark.parametrize("C", [50, 256, 2100])
def test_lengths_out_of_range_empty_items_and_unread_masked_frames(C):
    B, T = 4, 9
    s = make(B, T, C, F32, lengths=[0, -5, 100, 4])
    for name in ("x", "residual", "dy", "dsum"):
        clean = s[name].clone()
        for b, n in ((0, 0), (1, 0), (3, 4)):
            s[name][b, n:] = float("nan") if name in ("x", "dy") else float("inf")
        s[name + "_clean"] = clean
    y, total, mean, rstd = lib().dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"],
                                            rng=s["rng"], p=s["p"], alpha=s["alpha"])
    got = lib().dwnorm_bwd(total, s["gamma"], s["lengths"], mean, rstd, s["dy"], dsum=s["dsum"], rng=s["rng"], p=s["p"],
                           alpha=s["alpha"])
    torch.cuda.synchronize()
    for name in ("x", "residual", "dy", "dsum"):
        s[name] = s[name + "_clean"]
    check_fwd(s, (y, total, mean, rstd))
    for a, b in zip(got, check_bwd(s, total, mean, rstd)):
        assert torch.equal(a, b)


def test_empty_batches():
    dw = lib()
    for B, T, C in ((0, 5, 64), (3, 0, 64), (2, 4, 0)):
        x = torch.empty((B, T, C), device=DEV)
        y, s, mean, rstd = dw.dwnorm_fwd(x, lengths=None)
        dx, dres, dg, db = dw.dwnorm_bwd(x, None, None, mean, rstd, x)
        torch.cuda.synchronize()
        assert y.shape == x.shape and dg.shape == (C,) and not dg.any() and not db.any()
    assert dw.dwdrop_fwd(torch.empty((0, 8), device=DEV), None, 0.0).shape == (0, 8)


def test_rows_without_spread_and_with_a_large_mean():
    """A constant row has no variance: y is beta; a row far from zero keeps its digits by the second pass."""
    dw = lib()
    x = torch.full((1, 3, 512), 3.0, device=DEV)
    x[0, 2] = datagen.normal((512,), 1.0, "far", device=DEV) + 4096.0
    beta = datagen.normal((512,), 1.0, "beta", device=DEV)
    y, _, mean, rstd = dw.dwnorm_fwd(x, None, beta)
    torch.cuda.synchronize()
    assert torch.equal(y[0, 0], beta) and torch.equal(y[0, 1], beta)
    want = ref.norm_fwd(h(x), np.ones(512), h(beta), [3], None, np.ones((1, 3, 512)), 1.0)
    # the mean is off by at most 12 roundings of 4096 (its partial sums, per term), and y by that times rstd ~ 1
    near(y, want[0], F32, "y", extra=12 * ref.U32 * 4100)


def test_nan_and_inf_stay_in_their_row():
    s = make(1, 6, 256, F32, residual=False, p=0.0, alpha=1.0, lengths=[6])
    s["x"][0, 2, 5], s["x"][0, 4, 7] = float("nan"), float("inf")
    y, _, mean, rstd = lib().dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"])
    torch.cuda.synchronize()
    fine = torch.isfinite(y[0]).all(-1).tolist()
    assert fine == [True, True, False, True, False, True]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [40, 256, 1001])
def test_unaligned_storage_and_guard_bands(C, dt):
    """Inputs that start one element past a 16-byte boundary, outputs between canaries."""
    B, T = 2, 7
    s = make(B, T, C, dt)
    for name in ("x", "residual", "dy", "dsum", "gamma", "beta"):
        odd = torch.empty(s[name].numel() + 1, dtype=dt, device=DEV)
        odd[1:] = s[name].reshape(-1)
        s[name] = odd[1:].view(s[name].shape)
    outs = {n: Guarded((B, T, C), dt, DEV) for n in ("y", "s", "dx", "dres")}
    outs |= {n: Guarded(shape, F32, DEV) for n, shape in (("mean", (B, T)), ("rstd", (B, T)), ("dg", (C,)), ("db", (C,)))}
    dw = lib()
    ws = Guarded((dw.dwnorm_bwd_workspace_bytes(B, T, C),), torch.uint8, DEV, G=4096)
    o = {n: g.t for n, g in outs.items()}
    got = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=s["rng"], p=s["p"],
                        alpha=s["alpha"], y=o["y"], sum=o["s"], mean=o["mean"], rstd=o["rstd"])
    dw.dwnorm_bwd(o["s"], s["gamma"], s["lengths"], o["mean"], o["rstd"], s["dy"], dsum=s["dsum"], rng=s["rng"],
                  p=s["p"], alpha=s["alpha"], dx=o["dx"], dres=o["dres"], dgamma=o["dg"], dbeta=o["db"], workspace=ws.t)
    torch.cuda.synchronize()
    for n, g in outs.items():
        g.check(n)
        assert g.untouched_inside() == 0, n
    ws.check("workspace")
    check_fwd(s, got)
    for n, g in zip(("dx", "dres", "dg", "db"), check_bwd(s, o["s"], o["mean"], o["rstd"])):
        assert torch.equal(g, o[n]), n


def test_in_place():
    """The residual stream updated where it lies, and gradients over their inputs."""
    dw = lib()
    s = make(2, 11, 320, BF16)
    y, total, mean, rstd = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"],
                                         rng=s["rng"], p=s["p"], alpha=s["alpha"])
    x, r = s["x"].clone(), s["residual"].clone()
    y2, s2, _, _ = dw.dwnorm_fwd(x, s["gamma"], s["beta"], s["lengths"], residual=r, rng=s["rng"], p=s["p"],
                                 alpha=s["alpha"], y=x, sum=r)
    assert torch.equal(y, y2) and torch.equal(total, s2)
    dx, dres, dg, db = dw.dwnorm_bwd(total, s["gamma"], s["lengths"], mean, rstd, s["dy"], dsum=s["dsum"], rng=s["rng"],
                                     p=s["p"], alpha=s["alpha"])
    a, b = s["dy"].clone(), s["dsum"].clone()
    got = dw.dwnorm_bwd(total, s["gamma"], s["lengths"], mean, rstd, a, dsum=b, rng=s["rng"], p=s["p"], alpha=s["alpha"],
                        dx=a, dres=b)
    for u, v in zip((dx, dres, dg, db), got):
        assert torch.equal(u, v)
    d = dw.dwdrop_fwd(s["x"], s["rng"], 0.1, residual=s["residual"], alpha=2.0)
    z = s["x"].clone()
    assert torch.equal(d, dw.dwdrop_fwd(z, s["rng"], 0.1, residual=s["residual"], alpha=2.0, y=z))


def test_optional_outputs_and_repeatability():
    dw = lib()
    s = make(3, 50, 1024, BF16)
    full = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=s["rng"], p=s["p"],
                         alpha=s["alpha"])
    y, total, mean, rstd = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"],
                                         rng=s["rng"], p=s["p"], alpha=s["alpha"], need=("y",))
    assert total is None and mean is None and rstd is None and torch.equal(y, full[0])
    a = check_bwd(s, full[1], full[2], full[3])
    for need in (("dx",), ("dres",), ("dgamma",), ("dbeta", "dx")):
        b = check_bwd(s, full[1], full[2], full[3], need=need)
        for name, u, v in zip(("dx", "dres", "dgamma", "dbeta"), a, b):
            assert v is None if name not in need else torch.equal(u, v)


def test_gradients_against_differences():
    """<dL, v> of the backward calls against (L(+h) - L(-h)) / 2h of the forward, L = <y, w> + <s, w2> in fp64 of
    fp32 outputs.  The forward's rounding leaves about sqrt(N) * 3e-7 / h, the curvature about h^2: at h = 1e-2 and
    N = 2 * 6 * 96 values both are under 2e-3."""
    dw = lib()
    s = make(2, 6, 96, F32, lengths=[6, 4])
    kw = dict(rng=s["rng"], p=s["p"], alpha=s["alpha"])

    def loss(x, r, g, b):
        y, t, _, _ = dw.dwnorm_fwd(x, g, b, s["lengths"], residual=r, **kw)
        return float((y.double() * s["dy"].double()).sum() + (t.double() * s["dsum"].double()).sum())

    _, total, mean, rstd = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], **kw)
    grads = dw.dwnorm_bwd(total, s["gamma"], s["lengths"], mean, rstd, s["dy"], dsum=s["dsum"], **kw)
    at = [s["x"], s["residual"], s["gamma"], s["beta"]]
    for i, g in enumerate(grads):
        v = datagen.normal(tuple(at[i].shape), 1.0, f"dir/{i}", device=DEV)
        v /= v.norm()
        e = 1e-2
        up, down = ([a + f * v if k == i else a for k, a in enumerate(at)] for f in (e, -e))
        diff = (loss(*up) - loss(*down)) / (2 * e)
        exact = float((g.double() * v.double()).sum())
        assert abs(diff - exact) <= 2e-3 * max(1.0, abs(exact)), (i, diff, exact)


# ---------------------------------------------------------------------------
# Dropout
# ---------------------------------------------------------------------------
def test_generator_known_answers():
    """Philox4x32-10's published answer for a zero counter and key, read out of the kernel through its threshold, and
    another counter and key from the definition."""
    dw = lib()
    assert ref.philox4x32([0] * 4, [0] * 2) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    for seed, stream, row in ((0, 0, 0), (0x0123456789ABCDEF, 0xFEDCBA987654321, 3)):
        words = ref.philox4x32([row, 0, stream & 0xFFFFFFFF, stream >> 32], [seed & 0xFFFFFFFF, seed >> 32])
        halves = [f(w) for w in words for f in (lambda w: w & 0xFFFF, lambda w: w >> 16)]
        rng = torch.tensor([seed, stream], dtype=torch.int64, device=DEV)
        x = torch.ones((row + 1, 8), device=DEV)
        for e, u in enumerate(halves):
            assert u + 1 < 65535
            assert dw.dwdrop_fwd(x, rng, u / 65536)[row, e] != 0
            assert dw.dwdrop_fwd(x, rng, (u + 1) / 65536)[row, e] == 0


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (5, 8), (3, 50), (2, 9, 333), (17, 1024), (4100, 8), (1, 20000)])
def test_dropout(shape, dt):
    dw = lib()
    C, rows = shape[-1], int(np.prod(shape[:-1]))
    seed, stream = 0x7FFF_1234_0000_5678, (1 << 40) + 3
    rng = torch.tensor([seed, stream], dtype=torch.int64, device=DEV)
    x = datagen.normal(shape, 1.0, f"drop/{shape}", device=DEV).to(dt)
    r = datagen.normal(shape, 1.0, f"drop/r/{shape}", device=DEV).to(dt)
    for p, alpha in ((0.1, 1.0), (0.5, 0.5), (0.0, 2.0), (0.999999, 1.0)):
        f = ref.drop_factor(rows, C, seed, stream, p).reshape(shape)
        for res in (None, r):
            got = dw.dwdrop_fwd(x, rng, p, residual=res, alpha=alpha)
            want = alpha * f * h(x) + (0.0 if res is None else h(res))
            g = host64(got)
            tol = 4 * ref.U32 * (np.abs(alpha * f * h(x)) + np.abs(want)) + (ref.U16 * np.abs(want) if dt == BF16 else 0)
            assert (np.abs(g - want) <= tol).all()
            if res is None:
                assert ((g == 0) == (want == 0)).all()
                assert torch.equal(dw.dwdrop_bwd(x, rng, p, alpha=alpha), got)


def test_dropout_keeps_its_share():
    """2^22 elements at p = 0.1: the kept share is within 5 standard deviations, and streams differ."""
    dw = lib()
    x = torch.ones((4096, 1024), device=DEV)
    masks = []
    for stream in (0, 1):
        rng = torch.tensor([9, stream], dtype=torch.int64, device=DEV)
        masks.append(dw.dwdrop_fwd(x, rng, 0.1) != 0)
        share = float(masks[-1].double().mean())
        q = 1 - 6554 / 65536
        assert abs(share - q) < 5 * np.sqrt(q * (1 - q) / x.numel())
    both = float((masks[0] & masks[1]).double().mean())
    assert abs(both - q * q) < 5 * np.sqrt(q * q * (1 - q * q) / x.numel())


def test_norm_and_dropout_share_one_mask():
    """The fused norm drops what dwdrop_fwd drops for the same seed and stream."""
    dw = lib()
    s = make(2, 9, 200, F32, lengths=[9, 9])
    _, total, _, _ = dw.dwnorm_fwd(s["x"], lengths=s["lengths"], residual=s["residual"], rng=s["rng"], p=0.1, alpha=0.5)
    assert torch.equal(total, dw.dwdrop_fwd(s["x"], s["rng"], 0.1, residual=s["residual"], alpha=0.5))


# ---------------------------------------------------------------------------
# Streams and graphs
# ---------------------------------------------------------------------------
def test_on_another_stream():
    dw = lib()
    s = make(4, 64, 512, BF16)
    want = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=s["rng"], p=s["p"],
                         alpha=s["alpha"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=s["rng"], p=s["p"],
                            alpha=s["alpha"])
        grads = dw.dwnorm_bwd(got[1], s["gamma"], s["lengths"], got[2], got[3], s["dy"], dsum=s["dsum"], rng=s["rng"],
                              p=s["p"], alpha=s["alpha"])
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    for a, b in zip(grads, check_bwd(s, want[1], want[2], want[3])):
        assert torch.equal(a, b)


def test_captured_graph_follows_the_generator_state():
    """A captured forward and backward replayed with a new stream number each time, against eager calls."""
    dw = lib()
    s = make(3, 40, 256, BF16)
    o = {n: torch.empty_like(s["x"]) for n in ("y", "s", "dx", "dres")}
    m = {n: torch.empty((3, 40), device=DEV) for n in ("mean", "rstd")}
    w = {n: torch.empty((256,), device=DEV) for n in ("dg", "db")}
    ws = torch.empty((dw.dwnorm_bwd_workspace_bytes(3, 40, 256),), dtype=torch.uint8, device=DEV)
    kw = dict(rng=s["rng"], p=s["p"], alpha=s["alpha"])

    def step():
        dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], y=o["y"], sum=o["s"], **m, **kw)
        dw.dwnorm_bwd(o["s"], s["gamma"], s["lengths"], m["mean"], m["rstd"], s["dy"], dsum=s["dsum"], dx=o["dx"],
                      dres=o["dres"], dgamma=w["dg"], dbeta=w["db"], workspace=ws, **kw)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    seen = []
    for k in range(4):
        s["rng"][1] = 1000 + k
        for t in [*o.values(), *m.values(), *w.values()]:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in [*o.values(), *m.values(), *w.values()]]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, [*o.values(), *m.values(), *w.values()]):
            assert torch.equal(a, b)
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])


def test_binding_refusals():
    dw = lib()
    x = torch.zeros((2, 3, 16), device=DEV)
    rng = torch.zeros(2, dtype=torch.int64, device=DEV)
    with pytest.raises(TypeError):
        dw.dwnorm_fwd(x.half())
    with pytest.raises(ValueError):
        dw.dwnorm_fwd(x[0])
    with pytest.raises(ValueError):
        dw.dwnorm_fwd(x.transpose(1, 2))
    with pytest.raises(TypeError):
        dw.dwnorm_fwd(x, gamma=torch.ones(16, device=DEV, dtype=BF16))
    with pytest.raises(ValueError, match="rng"):
        dw.dwnorm_fwd(x, p=0.1)
    with pytest.raises(TypeError):
        dw.dwdrop_fwd(x, rng.int(), 0.1)
    with pytest.raises(dw.DwconvError, match="probability"):
        dw.dwdrop_fwd(x, rng, 1.0)
    with pytest.raises(dw.DwconvError, match="probability"):
        dw.dwdrop_fwd(x, rng, float("nan"))
    with pytest.raises(dw.DwconvError, match="8192"):
        dw.dwnorm_fwd(torch.zeros((1, 1, 8193), device=DEV))
    with pytest.raises(dw.DwconvError, match="alias"):
        dw.dwnorm_fwd(x, residual=x, y=x, sum=x)
    with pytest.raises(dw.DwconvError, match="workspace"):
        m = torch.zeros((2, 3), device=DEV)
        dw.dwnorm_bwd(x, None, None, m, m, x, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_plain_norm_in_place_keeps_its_input_for_the_gradients(dt):
    """y over x without a residual: the sum that comes back is the input, not y, and the gradients are the same."""
    dw = lib()
    s = make(2, 11, 320, dt, residual=False, p=0.0, alpha=1.0, lengths=[11, 7])
    args = (s["gamma"], s["beta"], s["lengths"])
    y, total, mean, rstd = dw.dwnorm_fwd(s["x"], *args)
    x = s["x"].clone()
    y2, total2, mean2, rstd2 = dw.dwnorm_fwd(x, *args, y=x)
    assert y2 is x and torch.equal(y, y2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    live = s["lengths"].tolist()
    for b, n in enumerate(live):
        assert torch.equal(total[b, :n], total2[b, :n])
    for a, b in zip(check_bwd(s, total, mean, rstd), check_bwd(s, total2, mean2, rstd2)):
        assert torch.equal(a, b)
    assert dw.dwnorm_fwd(s["x"].clone(), *args, y=x, need=("y",))[1] is None
    assert dw.dwnorm_fwd(s["x"], *args)[1] is s["x"]
