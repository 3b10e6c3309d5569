"""The activations kept in 8 bits against the definition in 64 bits.

The checkpoint is exact: its scales are powers of two, and the one rounding is
that of the definition.  Values pass through an exponential (whose argument for
bf16 is one rounded product: |x| * 1.5 more), a reciprocal and at most six
products: 16 roundings of 2^-24, and for bf16 storage one of its own.
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
KINDS = ["none", "silu", "glu"]


def lib():
    import conv_subsampling_amd as dw
    return dw


def make(B, T, C, dt, kind, lengths=None, seed=0):
    parts = 2 if kind == "glu" else 1
    n = lambda shape, name, var: datagen.normal(shape, var, f"act/{B}/{T}/{C}/{kind}/{seed}/{name}", device=DEV)  # noqa: E731
    x = n((B, T, parts * C), "x", 4.0) * torch.exp2(torch.round(8 * n((1, 1, parts * C), "s", 1.0)))
    return dict(B=B, T=T, C=C, dt=dt, kind=kind, parts=parts, x=x.to(dt), dy=n((B, T, C), "dy", 1.0).to(dt),
                lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV))


def dead(s):
    L = ref.clip(None if s["lengths"] is None else host64(s["lengths"]), s["B"], s["T"])
    return np.arange(s["T"])[None] >= L[:, None]


def near(got, want, size, x, dt, what):
    g = host64(got)
    reach = np.minimum(np.abs(x).max(initial=0.0), 130.0) if dt == BF16 else 0.0  # past 2^-190 nothing is left of a sigmoid
    tol = (16 + 1.5 * reach) * U * size + (ref.U16 * np.abs(want) if dt == BF16 else 0.0) + 1e-37
    with np.errstate(invalid="ignore"):
        bad = ~((np.abs(g - want) <= tol) | (g == want) | (np.isnan(g) & np.isnan(want)))
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.abs(g - want)[bad].max():.3e} at {np.argwhere(bad)[0]}"


def check(s, fwd=None, bwd=None):
    dw = lib()
    y, kept = fwd or dw.dwact_fwd(s["x"], s["kind"], s["lengths"])
    dx, y2 = bwd or dw.dwact_bwd(kept, s["dy"], s["kind"], s["lengths"], need=("dx", "y"))
    torch.cuda.synchronize()
    rows, gone, x = s["B"] * s["T"], dead(s), host64(s["x"])
    x = np.where(gone[..., None], 0.0, x)
    q, codes = ref.pack(x.reshape(rows, -1), s["parts"])
    codes = np.where(gone.reshape(rows, 1), 0, codes)
    assert np.array_equal(kept[0].cpu().numpy().reshape(rows, -1), q)
    assert np.array_equal(kept[1].cpu().numpy().reshape(rows, -1), codes)
    want = ref.act(x, s["kind"])
    near(y, want, np.abs(want), x, s["dt"], "y")
    xk = ref.unpack(q, codes, s["parts"]).reshape(x.shape)
    want = ref.act(xk, s["kind"])
    near(y2, want, np.abs(want), xk, s["dt"], "kept y")
    if s["kind"] == "none":
        assert np.array_equal(host64(y2), xk, equal_nan=True)  # exact in either type
    d = np.where(gone[..., None], 0.0, host64(s["dy"]))
    want, size = ref.act_grad(xk, d, s["kind"])
    near(dx, want, size, xk, s["dt"], "dx")
    for t in (y, y2, dx):
        assert not host64(t)[gone].any()
    return y, kept, dx, y2


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 3, 7, 8, 9, 24, 31, 32, 33, 40, 63, 64, 65, 100, 200, 256, 1000, 1024, 1025])
def test_widths(C, dt, kind):
    for B, T in ((1, 1), (3, 5), (2, 41)):
        s = make(B, T, C, dt, kind, [max(0, T - 2 * b) for b in range(B)])
        say("act", B, T, C, dt, kind)
        check(s)


@pytest.mark.parametrize("kind", KINDS)
def test_training_batch(kind):
    for dt in (F32, BF16):
        s = make(4, 750, 512, dt, kind, [750, 700, 400, 376])
        s["x"].clamp_(-30, 30)
        check(s)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [8, 50, 72])
def test_lengths_out_of_range_and_unread_frames(C, kind):
    L = [0, -5, 100, 4]
    s = make(4, 9, C, F32, kind, L)
    clean = {k: s[k].clone() for k in ("x", "dy")}
    for k in clean:
        for b, n in enumerate(L):
            s[k][b, max(0, n):] = float("nan")
    fwd = lib().dwact_fwd(s["x"], kind, s["lengths"])
    kept = [t.clone() for t in fwd[1]]
    for b, n in enumerate(L):
        kept[1][b, max(0, n):] = 255
    bwd = lib().dwact_bwd(kept, s["dy"], kind, s["lengths"], need=("dx", "y"))
    torch.cuda.synchronize()
    s |= clean
    check(s, fwd, bwd)


def test_scales_at_the_ends_of_the_range():
    """Groups of zeros, of subnormals, at both sides of 127 times a power of two, and of the type's largest."""
    x = torch.zeros((1, 14, 32), device=DEV)
    tops = [0.0, 2.0 ** -149, 2.0 ** -126, 127 * 2.0 ** -126, 127.00001 * 2.0 ** -126, 1.0, 127.0, 127.00001, 126.99999, 254.0, 254.1,
            3.4028234e38, 3.376e38, 127 * 2.0 ** 121]
    for r, v in enumerate(tops):
        x[0, r] = torch.linspace(-v, v, 32, device=DEV) if v else 0.0
        x[0, r, 7] = v
    s = dict(B=1, T=14, C=32, dt=F32, kind="none", parts=1, x=x, dy=torch.ones_like(x), lengths=None)
    check(s)
    s["x"] = x.bfloat16()
    check(s | {"dt": BF16, "dy": s["dy"].bfloat16()})


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_the_largest_values(dt):
    top = torch.finfo(dt).max
    x = torch.tensor([top, -top, top / 2, top / 254, 1.0] * 8, device=DEV, dtype=dt).view(1, 1, 40)
    s = dict(B=1, T=1, C=40, dt=dt, kind="none", parts=1, x=x, dy=torch.ones_like(x), lengths=None)
    _, kept, _, y = check(s)
    assert kept[1].tolist() == [[[248, 248]]] and torch.isfinite(y).all()


@pytest.mark.parametrize("kind", KINDS)
def test_infinities_and_nan_stay_in_their_group(kind):
    dw = lib()
    s = make(1, 3, 64, F32, kind)
    s["x"] = s["x"].clamp(-4, 4).contiguous()
    s["x"][0, 0, 5], s["x"][0, 1, 40], s["x"][0, 2, 63] = float("inf"), float("nan"), float("-inf")
    y, kept = dw.dwact_fwd(s["x"], kind)
    dx, y2 = dw.dwact_bwd(kept, s["dy"], kind, need=("dx", "y"))
    torch.cuda.synchronize()
    hit = torch.zeros((3, 2 * s["parts"]), dtype=torch.bool, device=DEV)
    hit[0, 0] = hit[1, 1] = hit[2, 1] = True
    assert torch.equal(kept[1][0] == 255, hit) and not kept[0][0].reshape(3, -1, 32)[hit].any()
    assert y2[0].reshape(3, 2, 32)[hit[:, :2]].isnan().all() and torch.isfinite(y2[0].reshape(3, 2, 32)[~hit[:, :2]]).all()
    if kind != "none":
        assert dx[0].reshape(3, -1, 32)[~hit].isfinite().sum() >= 3 * 32 and dx.isnan().any()
    assert torch.isfinite(y[0].reshape(3, 2, 32)[~hit[:, :2]]).all()


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("C", [5, 40, 96, 129])
def test_unaligned_storage_and_guard_bands(C, kind, dt):
    B, T = 2, 7
    s = make(B, T, C, dt, kind, [7, 4])
    dw, W = lib(), s["parts"] * C
    for k in ("x", "dy"):
        odd = torch.empty(s[k].numel() + 1, dtype=dt, device=DEV)
        odd[1:] = s[k].reshape(-1)
        s[k] = odd[1:].view(s[k].shape)
    o = {"y": Guarded((B, T, C), dt, DEV), "y2": Guarded((B, T, C), dt, DEV), "dx": Guarded((B, T, W), dt, DEV)}
    n = [B * T * W, B * T * s["parts"] * -(-C // 32)]
    raw = [torch.full((k + 2 * 1025,), -93, dtype=torch.int8, device=DEV) for k in n]
    q, codes = (r[1025:1025 + k].view(B, T, -1) for r, k in zip(raw, n))
    codes = codes.view(torch.uint8)
    fwd = dw.dwact_fwd(s["x"], kind, s["lengths"], y=o["y"].t, kept=(q, codes))
    bwd = dw.dwact_bwd((q, codes), s["dy"], kind, s["lengths"], dx=o["dx"].t, y=o["y2"].t)
    torch.cuda.synchronize()
    for name, g in o.items():
        g.check(name)
        assert g.untouched_inside() == 0, name
    for r, k in zip(raw, n):
        assert (r[:1025] == -93).all() and (r[1025 + k:] == -93).all()
    check(s, fwd, bwd)


def test_in_place_and_optional_outputs():
    dw = lib()
    for kind in KINDS:
        s = make(3, 20, 72, BF16, kind, [20, 11, 0])
        y, kept, dx, y2 = check(s)
        a, none = dw.dwact_fwd(s["x"], kind, s["lengths"], need=("y",))
        assert none is None and torch.equal(a, y)
        none, again = dw.dwact_fwd(s["x"], kind, s["lengths"], need=("kept",))
        assert none is None and all(torch.equal(u, v) for u, v in zip(again, kept))
        a, none = dw.dwact_bwd(kept, s["dy"], kind, s["lengths"])
        assert none is None and torch.equal(a, dx)
        none, a = dw.dwact_bwd(kept, None, kind, s["lengths"], dtype=BF16, need=("y",))
        assert none is None and torch.equal(a, y2)
        if kind != "glu":
            x, d = s["x"].clone(), s["dy"].clone()
            assert torch.equal(dw.dwact_fwd(x, kind, s["lengths"], y=x)[0], y) and torch.equal(x, y)
            assert torch.equal(dw.dwact_bwd(kept, d, kind, s["lengths"], dx=d)[0], dx) and torch.equal(d, dx)


def test_empty():
    dw = lib()
    for shape in ((0, 5, 64), (3, 0, 64), (2, 4, 0)):
        for kind in KINDS:
            x = torch.empty(shape, device=DEV)
            y, kept = dw.dwact_fwd(x, kind)
            dx, _ = dw.dwact_bwd(kept, y, kind)
            torch.cuda.synchronize()
            assert dx.shape == x.shape


def test_gradient_of_the_kept_input_against_differences():
    """(act(x + e) - act(x - e)) / 2e around inputs that 8 bits hold: e^2 / 6 of a third derivative under 1, rounding of 1e-7 / e."""
    dw = lib()
    for kind in ("silu", "glu"):
        W = 128 if kind == "glu" else 64
        x = (torch.randint(-100, 101, (1, 50, W), generator=torch.Generator().manual_seed(5)).float() / 32).to(DEV)
        x[..., ::32] = 100 / 32  # the group's scale is 1/32
        dy = datagen.normal((1, 50, 64), 1.0, "act/diff", device=DEV)
        _, kept = dw.dwact_fwd(x, kind)
        dx, y = dw.dwact_bwd(kept, dy, kind, need=("dx", "y"))
        assert torch.equal(y, dw.dwact_fwd(x, kind)[0])
        v = datagen.normal((1, 50, W), 1.0, "act/dir", device=DEV)
        e = 1e-2
        loss = lambda z: float((dw.dwact_fwd(z, kind, need=("y",))[0].double() * dy.double()).sum())  # noqa: E731
        diff, exact = (loss(x + e * v) - loss(x - e * v)) / (2 * e), float((dx.double() * v.double()).sum())
        assert abs(diff - exact) <= 5e-3 * max(1.0, abs(exact))


def test_more_than_32_bits_of_bytes():
    """A tensor of 2.6e9 elements: its first, last and some rows between."""
    dw = lib()
    T, C = 40000, 65536
    x = torch.zeros((1, T, C), dtype=BF16, device=DEV)
    rows = [0, 1, 16383, 16384, 32767, 32768, 32769, T - 1]
    part = datagen.normal((1, len(rows), C), 1.0, "act/far", device=DEV).to(BF16)
    x[:, rows] = part
    y, kept = dw.dwact_fwd(x, "silu")
    dx, _ = dw.dwact_bwd(kept, x, "silu")
    y1, kept1 = dw.dwact_fwd(part, "silu")
    dx1, _ = dw.dwact_bwd(kept1, part, "silu")
    torch.cuda.synchronize()
    assert torch.equal(y[:, rows], y1) and torch.equal(dx[:, rows], dx1) and torch.equal(kept[0][:, rows], kept1[0])


def test_streams_and_graph():
    dw = lib()
    s = make(2, 60, 200, BF16, "glu", [60, 33])
    want = check(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y, kept = dw.dwact_fwd(s["x"], "glu", s["lengths"])
        dx, y2 = dw.dwact_bwd(kept, s["dy"], "glu", s["lengths"], need=("dx", "y"))
    side.synchronize()
    for a, b in zip(want, (y, kept, dx, y2)):
        assert torch.equal(a, b) if isinstance(a, torch.Tensor) else all(torch.equal(u, v) for u, v in zip(a, b))

    def step():
        dw.dwact_fwd(s["x"], "glu", s["lengths"], y=y, kept=kept)
        dw.dwact_bwd(kept, s["dy"], "glu", s["lengths"], dx=dx, y=y2)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        s["x"].copy_(datagen.normal((2, 60, 400), 1.0, f"act/graph/{k}", device=DEV))
        g.replay()
        torch.cuda.synchronize()
        check(s, (y, kept), (dx, y2))


def test_binding_refusals():
    dw = lib()
    x = torch.zeros((2, 3, 16), device=DEV)
    kept = (torch.zeros((2, 3, 16), dtype=torch.int8, device=DEV), torch.zeros((2, 3, 1), dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="kind"):
        dw.dwact_fwd(x, "gelu")
    with pytest.raises(ValueError):
        dw.dwact_fwd(x[..., :15].contiguous(), "glu")
    with pytest.raises(TypeError):
        dw.dwact_fwd(x.half(), "silu")
    with pytest.raises(ValueError):
        dw.dwact_fwd(x.transpose(0, 1), "silu")
    with pytest.raises(ValueError):
        dw.dwact_fwd(x, "silu", kept=(kept[0], kept[1][:, :2]))
    with pytest.raises(TypeError):
        dw.dwact_bwd((kept[0].view(torch.uint8), kept[1]), x, "silu")
    with pytest.raises(ValueError, match="dy"):
        dw.dwact_bwd(kept, None, "silu", dtype=F32)
    with pytest.raises(TypeError):
        dw.dwact_bwd(kept, None, "silu", need=("y",))
    with pytest.raises(dw.DwconvError, match="alias"):
        wide = torch.zeros((2, 3, 32), device=DEV)
        dw.dwact_fwd(wide, "glu", y=wide.view(-1)[:96].view(2, 3, 16))


def test_tensors_of_the_host_are_refused():
    dw = lib()
    x = torch.zeros((2, 3, 16))
    with pytest.raises(ValueError):
        dw.dwact_fwd(x, "silu")
    with pytest.raises(ValueError):
        dw.dwact_bwd((x.to(torch.int8), torch.zeros((2, 3, 1), dtype=torch.uint8)), x, "silu")
