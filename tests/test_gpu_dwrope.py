"""The norm of heads with the rotation by positions, and its gradients, against
the definition in 64 bits.

Tolerances count roundings of 2^-24 (U).  The mean square adds up to 16 terms
a lane and 4 levels of lanes, all positive: 12, halved by the root; with the
root's own, the products and the angle (2 of its half turn, pi of it in
radians, and 2 of the polynomials) an output is within 32 of the sum of its
two absolute terms.  A gradient passes through both norms' sums: 64.  The
gammas' gradients add their rows one by one in each team, then 6 levels and 4
waves, then 64 bits.  bf16 storage adds one rounding.
"""
import numpy as np
import pytest
import torch

import datagen
import recur_ref as ref
from gpu_util import Guarded, host64, say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16
U = ref.U32


def lib():
    import conv_subsampling_amd as dw
    return dw


def h(t):
    """On the host in 64 bits, whole numbers and frequencies whole."""
    if t is None or t.dtype in (F32, BF16):
        return None if t is None else host64(t)
    return t.cpu().numpy()


def within(got, want, tol, dt, what):
    g = h(got)
    assert g.shape == want.shape, what
    tol = tol + (ref.U16 * np.abs(want) if dt == BF16 else 0.0)
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.abs(g - want)[bad].max():.3e} at {np.argwhere(bad)[0]}"


def make(B, T, H, Hkv, D, R, dt, pairs="halves", lengths=None, pos=None, gamma=True, seed=0):
    n = lambda shape, name, var=1.0: datagen.normal(shape, var, f"rope/{B}/{T}/{H}/{D}/{seed}/{name}", device=DEV).to(dt)  # noqa: E731
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(B=B, T=T, H=H, Hkv=Hkv, D=D, dt=dt, pairs=pairs, q=n((B, T, H, D), "q", 4.0), k=n((B, T, Hkv, D), "k", 4.0),
                v=n((B, T, Hkv, D), "v"), dq=n((B, T, H, D), "dq"), dk=n((B, T, Hkv, D), "dk"),
                qg=(1 + n((D,), "qg", 0.04)) if gamma else None, kg=(1 + n((D,), "kg", 0.04)) if gamma else None,
                freq=lib().rope_frequencies(R) if R else None, lengths=i32(lengths), pos=i32(pos))


def forward(s, **kw):
    return lib().dwrope_fwd(s["q"], s["k"], s["qg"], s["kg"], s["freq"], s["lengths"], s["pos"], pairs=s["pairs"], **kw)


def backward(s, **kw):
    return lib().dwrope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["qg"], s["kg"], s["freq"], s["lengths"], s["pos"], pairs=s["pairs"], **kw)


def check_fwd(s, got=None):
    got = got or forward(s)
    torch.cuda.synchronize()
    for name, x, g, out in (("q", s["q"], s["qg"], got[0]), ("k", s["k"], s["kg"], got[1])):
        want, size = ref.rope_fwd(h(x), h(g), h(s["freq"]), h(s["lengths"]), h(s["pos"]), s["pairs"], 1e-6)
        within(out, want, 32 * U * size, s["dt"], name)
        gone = np.arange(s["T"])[None] >= ref.clip(h(s["lengths"]), s["B"], s["T"])[:, None]
        assert not h(out)[gone].any()
    return got


def check_bwd(s, got=None):
    got = got or backward(s)
    torch.cuda.synchronize()
    freq = h(s["freq"])
    for name, x, g, d, dx, dg in (("q", s["q"], s["qg"], s["dq"], got[0], got[2]), ("k", s["k"], s["kg"], s["dk"], got[1], got[3])):
        want, size, wg, gsize = ref.rope_bwd(h(x), h(g), freq, h(s["lengths"]), h(s["pos"]), s["pairs"], 1e-6, h(d))
        rows = s["B"] * s["T"] * x.shape[2]
        if dx is not None:
            within(dx, want, 64 * U * size, s["dt"], "d" + name)
        if dg is not None:
            within(dg, wg, (80 + rows / 64) * U * gsize + 1e-37, F32, name + "_gamma")
    return got


HEADS = [(1, 0), (2, 2), (3, 2), (4, 4), (7, 0), (8, 8), (8, 6), (16, 16), (20, 12), (31, 30), (32, 32), (33, 8), (50, 32), (50, 50),
         (64, 64), (64, 40), (72, 36), (80, 80), (100, 100), (127, 126), (128, 128), (128, 64), (128, 0), (128, 20)]


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D,R", HEADS)
def test_heads(D, R, dt, pairs):
    for B, T, H, Hkv in ((2, 7, 4, 2), (1, 1, 3, 1)):
        s = make(B, T, H, Hkv, D, R, dt, pairs, [T, T - 2][:B], [0, 12345][:B])
        say("rope", B, T, H, Hkv, D, R, dt, pairs)
        check_fwd(s)
        check_bwd(s)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,H,Hkv", [(1, 1, 1, 1), (64, 1, 8, 2), (3, 5, 32, 1), (1, 9, 70, 5), (2, 40, 6, 6), (5, 333, 4, 2), (2, 1, 1, 9),
                                       (16, 200, 8, 8), (1, 3000, 3, 3)])
def test_frames_and_heads(B, T, H, Hkv, dt):
    s = make(B, T, H, Hkv, 64, 64, dt, lengths=[max(0, T - 3 * b) for b in range(B)], pos=[7 * b for b in range(B)])
    say("rope", B, T, H, Hkv, dt)
    check_fwd(s)
    check_bwd(s)


@pytest.mark.parametrize("H,Hkv", [(3, 0), (0, 2)])
def test_queries_or_keys_alone(H, Hkv):
    s = make(2, 6, H, Hkv, 48, 48, F32, lengths=[6, 3])
    check_fwd(s)
    check_bwd(s)


def test_far_positions_keep_their_angles():
    """Positions up to the end of 32 bits, below zero and past its end with the frame added, against angles in 64 bits.  The
    reference's own product is off by 2^-53 of up to 2^31 radians: 2.4e-7, under 4 U of a value."""
    top = (1 << 31) - 1
    s = make(6, 5, 2, 1, 64, 64, F32, pos=[0, 1_000_000, 123_456_789, top - 4, -7, -1_000_000], gamma=False)
    check_fwd(s)
    check_bwd(s)
    s = make(1, 3, 1, 1, 8, 8, F32, pos=[top])
    check_fwd(s)


@pytest.mark.parametrize("D,R,pairs", [(64, 64, "halves"), (50, 32, "neighbours")])
def test_lengths_out_of_range_and_unread_frames(D, R, pairs):
    L = [0, -5, 100, 4]
    s = make(4, 9, 3, 2, D, R, F32, pairs, L)
    keys = ("q", "k", "v", "dq", "dk")
    clean = {k: s[k].clone() for k in keys}
    for k in keys:
        for b, n in enumerate(L):
            s[k][b, max(0, n):] = float("nan") if k in "qk" else float("inf")
    f, v = forward(s, v=s["v"]), s["v"]
    g = backward(s)
    torch.cuda.synchronize()
    s |= clean
    check_fwd(s, f)
    check_bwd(s, g)
    for b, n in enumerate(L):
        n = max(0, min(9, n))
        assert torch.equal(f[2][b, :n], v[b, :n]) and not f[2][b, n:].any()


def test_zero_rows_and_no_eps():
    """A head of zeros has no norm without eps: NaN there and nowhere else; masked frames add nothing to the weights' gradients."""
    dw = lib()
    s = make(2, 4, 2, 1, 16, 16, F32, lengths=[4, 2])
    s["q"][0, 1, 0] = 0
    args = (s["qg"], s["kg"], s["freq"], s["lengths"])
    q, k, _ = dw.dwrope_fwd(s["q"], s["k"], *args, eps=0.0)
    assert q[0, 1, 0].isnan().all() and q.isnan().sum() == 16 and k.isfinite().all()
    q, _, _ = dw.dwrope_fwd(s["q"], s["k"], *args, eps=1e-6)
    assert not q[0, 1, 0].any()
    _, dk, _, gk = dw.dwrope_bwd(s["q"], s["k"], s["dq"], s["dk"], *args, eps=0.0)
    assert dk.isfinite().all() and gk.isfinite().all()


def test_infinities_and_nan_stay_in_their_head():
    s = make(1, 3, 4, 1, 32, 32, BF16)
    s["q"][0, 1, 2, 5], s["q"][0, 2, 0, 31] = float("nan"), float("inf")
    q, k, _ = forward(s)
    bad = ~q.isfinite().all(-1)[0]
    assert bad.nonzero().tolist() == [[1, 2], [2, 0]] and k.isfinite().all()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D,R,pairs", [(64, 64, "halves"), (80, 48, "halves"), (50, 32, "neighbours"), (44, 44, "halves")])
def test_slices_of_a_projection_and_in_place(D, R, pairs, dt):
    """q, k and v as slices of one tensor that starts off its alignment, written over, gradients into slices of another."""
    B, T, H, Hkv = 2, 11, 4, 2
    s = make(B, T, H, Hkv, D, R, dt, pairs, [11, 8], [3, 0])
    want, grad = check_fwd(s), check_bwd(s)

    def sliced(parts):
        flat = torch.full((B * T * (H + 2 * Hkv) * D + 1,), 5.0, dtype=dt, device=DEV)
        views = flat[1:].view(B, T, H + 2 * Hkv, D).split([H, Hkv, Hkv], 2)
        for a, b in zip(views, parts):
            a.copy_(b)
        return views
    q, k, v = sliced((s["q"], s["k"], s["v"]))
    got = forward(s | {"q": q, "k": k})
    for a, b in zip(got[:2], want):
        assert torch.equal(a, b)
    out = torch.empty((T, H, B, D), dtype=dt, device=DEV).permute(2, 0, 1, 3)
    assert torch.equal(forward(s | {"q": q, "k": k}, q_out=out)[0], want[0])
    dq, dk, rest = sliced((s["dq"], s["dk"], s["v"]))
    keep = rest.clone()
    again = backward(s | {"q": q, "k": k, "dq": dq, "dk": dk}, dq=dq, dk=dk)
    for a, b in zip(again, grad):
        assert torch.equal(a, b)
    assert torch.equal(rest, keep)
    forward(s | {"q": q, "k": k}, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, s["v"])


def test_broadcast_inputs():
    """One key head's tensor for all items, one gradient for all frames."""
    s = make(3, 6, 2, 2, 32, 32, F32, lengths=[6, 5, 1])
    s["k"] = s["k"][:1].expand(3, 6, 2, 32)
    s["dq"] = s["dq"][:, :1].expand(3, 6, 2, 32)
    check_fwd(s)
    check_bwd(s)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 64), (8, 128), (5, 50)])
def test_into_caches(T, D, dt):
    """Frames to their places; ones past the length, before the cache or behind it are not written, nor is anything else."""
    B, H, Hkv, S = 6, 4, 2, 20
    place = [0, 3, S - T, S - 1, -1, S + 4]
    lengths = [T, max(0, T - 2), T, T, T, T]
    s = make(B, T, H, Hkv, D, D - D % 2, dt, lengths=lengths, pos=[5, 0, 1 << 20, 9, 2, 77])
    k1, v1 = (torch.full((B, S, Hkv, D), 9.0, dtype=dt, device=DEV) for _ in range(2))
    both = torch.full((B, S, 2, Hkv, D), 9.0, dtype=dt, device=DEV)  # keys and values frame by frame
    k2, v2 = both.unbind(2)
    q, k, v = forward(s, v=s["v"])
    at = torch.tensor(place, dtype=torch.int32, device=DEV)
    q1, kk, vv = forward(s, v=s["v"], place=at, k_out=k1, v_out=v1)
    assert kk is k1 and vv is v1
    forward(s, v=s["v"], place=at, k_out=k2, v_out=v2)
    k3 = torch.full_like(k1, 9.0)
    forward(s, place=at, k_out=k3)
    torch.cuda.synchronize()
    check_fwd(s, (q1, k))
    wk, wv = torch.full_like(k1, 9.0), torch.full_like(v1, 9.0)
    for b in range(B):
        for t in range(lengths[b]):
            if 0 <= place[b] + t < S:
                wk[b, place[b] + t], wv[b, place[b] + t] = k[b, t], s["v"][b, t]
    for got, want in ((k1, wk), (v1, wv), (k2, wk), (v2, wv), (k3, wk)):
        assert torch.equal(got, want)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("D,R,pairs", [(64, 64, "halves"), (40, 8, "neighbours"), (33, 32, "halves"), (7, 4, "neighbours"), (128, 128, "halves")])
def test_guard_bands(D, R, pairs, dt):
    B, T, H, Hkv = 2, 5, 3, 2
    s = make(B, T, H, Hkv, D, R, dt, pairs, [5, 3])
    o = {n: Guarded((B, T, H if n.endswith("q") else Hkv, D), dt, DEV) for n in ("q", "k", "v", "dq", "dk")}
    o |= {n: Guarded((D,), F32, DEV) for n in ("gq", "gk")}
    t = {n: g.t for n, g in o.items()}
    dw = lib()
    ws = Guarded((dw.dwrope_bwd_workspace_bytes(B, T, H, Hkv, D),), torch.uint8, DEV, G=4096)
    f = forward(s, v=s["v"], q_out=t["q"], k_out=t["k"], v_out=t["v"])
    g = backward(s, dq=t["dq"], dk=t["dk"], dq_gamma=t["gq"], dk_gamma=t["gk"], workspace=ws.t)
    torch.cuda.synchronize()
    for n, x in o.items():
        x.check(n)
        assert x.untouched_inside() == 0, n
    ws.check("workspace")
    check_fwd(s, f)
    check_bwd(s, g)


def test_empty_batches():
    dw = lib()
    for B, T, H, Hkv in ((0, 5, 2, 1), (3, 0, 2, 1), (2, 4, 0, 0)):
        s = make(B, T, H, Hkv, 16, 16, F32)
        q, k, _ = forward(s)
        dq, dk, gq, gk = backward(s)
        torch.cuda.synchronize()
        assert q.shape == s["q"].shape and k.shape == s["k"].shape and not gq.any() and not gk.any()
    s = make(2, 1, 2, 1, 16, 16, F32)
    none = torch.empty((2, 0, 1, 16), device=DEV)
    assert torch.equal(forward(s, place=torch.zeros(2, dtype=torch.int32, device=DEV), k_out=none)[0], forward(s)[0])


def test_optional_outputs_and_repeatability():
    s = make(4, 300, 4, 2, 64, 64, BF16, lengths=[300, 200, 9, 0])
    full = check_bwd(s)
    names = ("dq", "dk", "dq_gamma", "dk_gamma")
    for need in (("dq",), ("dk",), ("dq_gamma",), ("dk_gamma", "dq")):
        for name, a, b in zip(names, full, backward(s, need=need)):
            assert b is None if name not in need else torch.equal(a, b)


def test_gradients_against_differences():
    """(L(+e) - L(-e)) / 2e of the forward, L = <q', dq> + <k', dk>: rounding of sqrt(N) 3e-7 / e and a curvature of e^2, both under 2e-3
    at e = 1e-2."""
    dw = lib()
    s = make(2, 6, 3, 2, 40, 24, F32, "neighbours", [6, 4], [2, 900])
    kw = dict(pairs="neighbours")

    def loss(q, k, qg, kg):
        a, b, _ = dw.dwrope_fwd(q, k, qg, kg, s["freq"], s["lengths"], s["pos"], **kw)
        return float((a.double() * s["dq"].double()).sum() + (b.double() * s["dk"].double()).sum())
    at = [s["q"], s["k"], s["qg"], s["kg"]]
    for i, g in enumerate(backward(s)):
        v = datagen.normal(tuple(at[i].shape), 1.0, f"rope/dir/{i}", device=DEV)
        v /= v.norm()
        up, down = ([a + f * v if k == i else a for k, a in enumerate(at)] for f in (1e-2, -1e-2))
        diff, exact = (loss(*up) - loss(*down)) / 2e-2, float((g.double() * v.double()).sum())
        assert abs(diff - exact) <= 2e-3 * max(1.0, abs(exact)), (i, diff, exact)


def test_past_32_bit_offsets():
    """Items 2^31 + 3 elements apart, as inputs, as a cache and as gradients."""
    B, T, H, D = 2, 3, 2, 64
    s = make(B, T, H, H, D, D, BF16, lengths=[3, 2])
    want, grad = check_fwd(s), check_bwd(s)
    far = (1 << 31) + 3
    big = torch.empty(far + T * H * D, dtype=BF16, device=DEV)
    view = big.as_strided((B, T, H, D), (far, H * D, D, 1))
    for k in ("q", "k", "dq", "dk"):
        t = s | {k: view.copy_(s[k])}
        assert all(torch.equal(a, b) for a, b in zip(forward(t)[:2], want))
        assert all(torch.equal(a, b) for a, b in zip(backward(t), grad))
    assert torch.equal(forward(s, k_out=view)[1], want[1])
    assert torch.equal(backward(s, dq=view)[0], grad[0])
    frames = (1 << 31) // (H * D) + 5
    cache = torch.empty((1, frames, H, D), dtype=BF16, device=DEV)
    one = make(1, T, H, H, D, D, BF16, pos=[frames - 4])
    forward(one, place=torch.tensor([frames - 4], dtype=torch.int32, device=DEV), k_out=cache)
    assert torch.equal(cache[:, frames - 4:frames - 1], check_fwd(one)[1])


def test_streams_and_graph():
    """A decoding step on another stream, then captured with its positions moving on between replays."""
    dw = lib()
    s = make(5, 1, 4, 2, 64, 64, BF16, pos=[0, 3, 9, 2, 5])
    kc, vc = torch.zeros((5, 30, 2, 64), dtype=BF16, device=DEV), torch.zeros((5, 30, 2, 64), dtype=BF16, device=DEV)
    q = torch.empty_like(s["q"])

    def step():
        forward(s, v=s["v"], place=s["pos"], q_out=q, k_out=kc, v_out=vc)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check_fwd(s, (q, torch.stack([kc[b, p:p + 1] for b, p in enumerate(s["pos"].tolist())])))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        s["pos"].add_(1)
        s["q"].copy_(datagen.normal((5, 1, 4, 64), 1.0, f"rope/graph/{k}", device=DEV))
        q.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        check_fwd(s, (q, torch.stack([kc[b, p:p + 1] for b, p in enumerate(s["pos"].tolist())])))
        assert all(torch.equal(vc[b, p], s["v"][b, 0]) for b, p in enumerate(s["pos"].tolist()))

    t = make(2, 50, 4, 2, 64, 64, BF16, lengths=[50, 20])
    want = check_bwd(t)
    o = [torch.empty_like(w) for w in want]
    ws = torch.empty((dw.dwrope_bwd_workspace_bytes(2, 50, 4, 2, 64),), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        backward(t, dq=o[0], dk=o[1], dq_gamma=o[2], dk_gamma=o[3], workspace=ws)
    for _ in range(3):
        for x in o:
            x.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_binding_refusals():
    dw = lib()
    q, k, f = torch.zeros((2, 3, 4, 16), device=DEV), torch.zeros((2, 3, 2, 16), device=DEV), dw.rope_frequencies(16)
    at = torch.zeros(2, dtype=torch.int32, device=DEV)
    with pytest.raises(TypeError):
        dw.dwrope_fwd(q.half(), k.half())
    with pytest.raises(ValueError):
        dw.dwrope_fwd(q[0], k[0])
    with pytest.raises(ValueError):
        dw.dwrope_fwd(q, k[:, :2])
    with pytest.raises(ValueError, match="pairs"):
        dw.dwrope_fwd(q, k, pairs="quarters")
    with pytest.raises(TypeError):
        dw.dwrope_fwd(q, k, freq=f.float())
    with pytest.raises(ValueError, match="next to each other"):
        dw.dwrope_fwd(torch.zeros((2, 3, 16, 4), device=DEV).transpose(2, 3), k)
    with pytest.raises(ValueError, match="caches"):
        dw.dwrope_fwd(q, k, place=at)
    with pytest.raises(ValueError, match="v_out"):
        dw.dwrope_fwd(q, k, v_out=k.clone())
    with pytest.raises(dw.DwconvError, match="rotated"):
        dw.dwrope_fwd(q, k, freq=dw.rope_frequencies(18))
    with pytest.raises(dw.DwconvError, match="128"):
        dw.dwrope_fwd(torch.zeros((1, 1, 1, 129), device=DEV), torch.zeros((1, 1, 1, 129), device=DEV))
    with pytest.raises(dw.DwconvError, match="eps"):
        dw.dwrope_fwd(q, k, eps=-1.0)
    with pytest.raises(dw.DwconvError, match="alias"):
        dw.dwrope_fwd(k, k, q_out=k, k_out=k)
    with pytest.raises(ValueError):
        dw.rope_frequencies(3)
    with pytest.raises(dw.DwconvError, match="workspace"):
        dw.dwrope_bwd(q, k, q, k, freq=f, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))


def test_tensors_of_the_host_are_refused():
    dw = lib()
    x = torch.zeros((2, 3, 4, 16))
    with pytest.raises(ValueError):
        dw.dwrope_fwd(x, x)
    with pytest.raises(ValueError):
        dw.dwrope_bwd(x, x, x, x)
