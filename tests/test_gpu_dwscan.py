"""The gated linear recurrence and its gradients against the definition in 64
bits.

Tolerances count roundings of 2^-24 (U).  A step's -log of the decay (w), 1 - a
and sqrt(1 - a^2) each pass through two functions of a few units, the products
and a series or difference of 8 U at most: 40 U together, and the exponential of
a gate is that of one rounded product, off by |r| U: 16 more for what
is at most 16 of a gate that is not closed.  An error of
56 U in w changes a product of decays by 56 U times its -log: the sum "bent",
the absolute terms weighted by that.  The state itself is rounded twice a frame
of a thread's run (8), twice a run of a tile on the way (8), and once more a
tile; each such rounding is at most U of the sum of absolute terms, which
decays no faster than the error.  bf16 storage adds one rounding.
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
    return None if t is None else host64(t)


def rel(dt):
    return 56


def within(got, want, tol, dt, what):
    g = h(got)
    assert g.shape == want.shape, what
    tol = tol + (ref.U16 * np.abs(want) if dt == BF16 else 0.0) + 1e-37
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} off, worst {np.abs(g - want)[bad].max():.3e} against "
                           f"{np.broadcast_to(tol, g.shape)[bad].min():.3e} at {np.argwhere(bad)[0]}")


def make(B, T, C, dt, lengths=None, state=True, seed=0, tag="scan"):
    n = lambda shape, name: datagen.normal(shape, 1.0, f"{tag}/{B}/{T}/{C}/{seed}/{name}", device=DEV)  # noqa: E731
    s = dict(B=B, T=T, C=C, dt=dt, **{k: n((B, T, C), k).to(dt) for k in ("x", "r", "g", "dy")})
    # slow and fast channels: decays of 0.9998 to 0.5 a frame, and two at the ends of the range
    s["decay"] = datagen.uniform((C,), -8.0, 0.0, f"{tag}/{C}/decay", device=DEV)
    if C > 6:
        s["decay"][4], s["decay"][5] = -200.0, 90.0
    s["h0"], s["dh_last"] = (n((B, C), k) if state else None for k in ("h0", "dh"))
    s["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return s


def check_fwd(s, got=None):
    got = got or lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"])
    torch.cuda.synchronize()
    y, last, ys, ls, yb, lb = ref.scan_fwd(*(h(s[k]) for k in ("x", "r", "g", "decay", "lengths", "h0")))
    n = rel(s["dt"]) + 40 + 2 * (-(-s["T"] // 64))
    within(got[0], y, U * (n * ys + rel(s["dt"]) * yb), s["dt"], "y")
    within(got[1], last, U * (n * ls + rel(s["dt"]) * lb), F32, "h_last")
    if s["lengths"] is not None:
        dead = np.arange(s["T"])[None] >= np.clip(h(s["lengths"]), 0, s["T"])[:, None]
        assert not h(got[0])[dead].any()
    return got


def grads(s, y, **kw):
    return lib().dwscan_bwd(s["x"], s["r"], s["g"], s["decay"], y, s["dy"], s["lengths"], h0=s["h0"], dh_last=s["dh_last"], **kw)


NAMES = ("dx", "dr", "dg", "ddecay", "dh0")


def check_bwd(s, y, got=None):
    got = got or grads(s, y)
    torch.cuda.synchronize()
    want = ref.scan_bwd(*(h(s[k]) for k in ("x", "r", "g", "decay")), h(y), h(s["dy"]), h(s["lengths"]), h(s["h0"]), h(s["dh_last"]))
    e = rel(s["dt"])
    for name, g in zip(NAMES, got):
        if g is None:
            continue
        # the products around G are some 24 more roundings; a thread adds its frames (a sixteenth of them at least) one by one
        n = 2 * e + 64 + 2 * (-(-s["T"] // 64)) + (s["T"] // 16 + 32 if name == "ddecay" else 0)
        within(g, want[name], U * (n * want[name + "_size"] + e * want[name + "_bent"]),
               s["dt"] if name in ("dx", "dr", "dg") else F32, name)
    return got


# lengths around a thread's run, a wave's and a tile's frames in both directions, and enough to be shared out
FRAMES = [1, 2, 4, 5, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 255, 256, 257, 300, 511, 513, 700]
WIDTHS = [1, 2, 3, 4, 5, 7, 8, 60, 63, 64, 65, 68, 100, 130, 200]


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", FRAMES)
def test_frames(T, dt):
    for B, C, seed in ((3, 70, 0), (2, 64, 1)):
        s = make(B, T, C, dt, [T, max(0, T - 3), T // 2][:B], seed=seed)
        say("scan", B, T, C, dt)
        check_bwd(s, check_fwd(s)[0])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(C, dt):
    for B, T in ((19, 1), (18, 6), (5, 23), (2, 77), (1, 600)):
        s = make(B, T, C, dt, state=C % 2 == 0)
        say("scan", B, T, C, dt)
        check_bwd(s, check_fwd(s)[0])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,C", [(16, 333, 1100), (130, 260, 130), (4, 1500, 256), (1, 5000, 66)])
def test_many_workgroups_and_long_sequences(B, T, C, dt):
    s = make(B, T, C, dt, [max(1, T - (b * T) // (2 * B)) for b in range(B)])
    say("scan", B, T, C, dt)
    check_bwd(s, check_fwd(s)[0])


@pytest.mark.parametrize("T", [1, 6, 20, 90, 700])
def test_lengths_out_of_range_empty_items_and_unread_frames(T):
    L = [0, -5, T + 100, T // 3]
    s = make(4, T, 66, F32, L)
    clean = {k: s[k].clone() for k in ("x", "r", "g", "dy")}
    for k in clean:
        for b, n in enumerate(L):
            s[k][b, max(0, n):] = float("nan") if k in "xr" else float("inf")
    y, last = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"])
    ynan = y.clone()
    for b, n in enumerate(L):
        ynan[b, max(0, n):] = float("nan")
    got = grads(s, ynan)
    torch.cuda.synchronize()
    s |= clean
    check_fwd(s, (y, last))
    check_bwd(s, y, got)
    for b in (0, 1):
        assert torch.equal(last[b], s["h0"][b]) and torch.equal(got[4][b], s["dh_last"][b])


def test_empty_batches_and_no_frames():
    dw = lib()
    for B, T, C in ((0, 5, 8), (3, 0, 8), (2, 4, 0)):
        s = make(B, T, C, F32)
        y, last = dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], h0=s["h0"])
        got = grads(s, y)
        torch.cuda.synchronize()
        assert y.shape == (B, T, C) and not got[3].any()
        if T == 0:
            assert torch.equal(last, s["h0"]) and torch.equal(got[4], s["dh_last"])


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [3, 30, 600])
def test_slices_of_a_projection_and_broadcast_inputs(T, dt):
    """Gates as slices of one tensor, gradients into slices of another, an input shared by all items, an odd start."""
    B, C = 2, 72
    s = make(B, T, C, dt, [T, T - 1])
    wide = torch.empty((B, T, 3 * C + 1), dtype=dt, device=DEV)
    for k, key in enumerate(("x", "r", "g")):
        wide[..., 1 + k * C:1 + (k + 1) * C] = s[key]
        s[key] = wide[..., 1 + k * C:1 + (k + 1) * C]
    s["dy"] = s["dy"][:1, :1].expand(B, T, C)
    y = torch.empty((T, B, C), dtype=dt, device=DEV).transpose(0, 1)
    got = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], y=y)
    assert got[0] is y
    check_fwd(s, got)
    into = torch.full((B, T, 3 * C + 1), 7.0, dtype=dt, device=DEV)
    parts = [into[..., 1 + k * C:1 + (k + 1) * C] for k in range(3)]
    check_bwd(s, y, grads(s, y, dx=parts[0], dr=parts[1], dg=parts[2]))
    assert (into[..., 0] == 7).all()
    dense = [t.contiguous() for t in (s["x"], s["r"], s["g"])]
    again, _ = lib().dwscan_fwd(*dense, s["decay"], s["lengths"], h0=s["h0"])
    assert torch.equal(again, y)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("B,T,C", [(17, 1, 61), (3, 7, 64), (2, 29, 67), (2, 130, 72), (1, 900, 100)])
def test_guard_bands(B, T, C, dt):
    s = make(B, T, C, dt, [T - b for b in range(B)])
    dw = lib()
    o = {n: Guarded((B, T, C), dt, DEV) for n in ("y", "dx", "dr", "dg")}
    o |= {"h_last": Guarded((B, C), F32, DEV), "ddecay": Guarded((C,), F32, DEV), "dh0": Guarded((B, C), F32, DEV)}
    t = {n: g.t for n, g in o.items()}
    ws = [Guarded((max(16, n),), torch.uint8, DEV, G=4096) for n in (dw.dwscan_fwd_workspace_bytes(B, T, C), dw.dwscan_bwd_workspace_bytes(B, T, C))]
    dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], y=t["y"], h_last=t["h_last"], workspace=ws[0].t)
    got = grads(s, t["y"], workspace=ws[1].t, **{n: t[n] for n in NAMES})
    torch.cuda.synchronize()
    for n, g in [*o.items(), *zip("ab", ws)]:
        g.check(n)
        assert n in "ab" or g.untouched_inside() == 0, n
    check_fwd(s, (t["y"], t["h_last"]))
    check_bwd(s, t["y"], got)


def test_infinities_and_nan_stay_in_their_channel():
    s = make(1, 40, 16, F32, state=False)
    s["r"][0, 3, 0], s["r"][0, 3, 1], s["g"][0, 5, 2], s["g"][0, 5, 3] = float("inf"), float("-inf"), float("inf"), float("-inf")
    check_bwd(s, check_fwd(s)[0])
    s["x"][0, 9, 4], s["r"][0, 9, 5], s["g"][0, 9, 6], s["x"][0, 9, 7] = float("nan"), float("nan"), float("nan"), float("inf")
    y, last = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"])
    torch.cuda.synchronize()
    assert torch.isfinite(y[0, :9]).all() and torch.isfinite(y[0, :, [0, 1, 2, 3] + list(range(8, 16))]).all()
    assert y[0, 9:, 4:7].isnan().all() and torch.isinf(y[0, 9, 7])


def test_a_decay_of_one_keeps_its_state_and_a_decay_of_zero_forgets_it():
    B, T, C = 2, 500, 8
    s = make(B, T, C, F32)
    s["decay"][:4], s["decay"][4:] = -200.0, 1e30
    y, last = check_fwd(s)
    assert torch.equal(last[:, :4], s["h0"][:, :4]) and torch.equal(y[:, 250, :4], s["h0"][:, :4])
    check_bwd(s, y)


def test_slow_decays_keep_their_digits():
    """1 - a = 1e-6 over 3000 frames without an input: the state is exp(-3e-3) of its start.  The error counts the
    roundings of w (40 U times its sum) and of the state."""
    T, C = 3000, 64
    zero = torch.zeros((1, T, C), device=DEV)
    decay = torch.full((C,), float(np.log(np.expm1(1e-6 / 4))), device=DEV)
    h0 = torch.ones((1, C), device=DEV)
    y, last = lib().dwscan_fwd(zero, zero, zero, decay, h0=h0)
    rate = 8 * np.log1p(np.exp(float(decay[0]))) / 2
    want = np.exp(-rate * (1 + np.arange(T)))[None, :, None] * np.ones(C)
    within(y, want, U * (200 + 40 * 3e-3), F32, "y")


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("T", [1, 5, 200, 1500])
def test_in_place_state(T, dt):
    s = make(3, T, 65, dt, [T, T - 1, 0])
    y, last = check_fwd(s)
    state = s["h0"].clone()
    y2, last2 = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=state, h_last=state)
    assert last2 is state and torch.equal(state, last) and torch.equal(y, y2)
    got = check_bwd(s, y)
    d = s["dh_last"].clone()
    s2 = s | {"dh_last": d}
    again = grads(s2, y, dh0=d)
    for a, b in zip(got, again):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
def test_a_stream_gives_what_the_whole_gives(dt):
    """Chunks of 1 to 300 frames with a state in place, some streams pausing (length 0), against each stream's whole."""
    B, C = 3, 96
    T = [420, 300, 77]
    s = make(B, 420, C, dt, T)
    y, last = check_fwd(s)
    state, done = s["h0"].clone(), [0] * B
    for chunk in (1, 1, 8, 40, 300, 130):
        n = [min(chunk if (chunk + b) % 4 else 0, T[b] - done[b]) for b in range(B)] if chunk != 130 else [T[b] - done[b] for b in range(B)]
        w = max(chunk, *n)
        part = {k: torch.zeros((B, w, C), dtype=dt, device=DEV) for k in ("x", "r", "g")}
        for b in range(B):
            for k in part:
                part[k][b, :n[b]] = s[k][b, done[b]:done[b] + n[b]]
        out, _ = lib().dwscan_fwd(part["x"], part["r"], part["g"], s["decay"], torch.tensor(n, dtype=torch.int32, device=DEV), h0=state,
                                  h_last=state)
        for b in range(B):
            # both are within half the bound of the truth: compare as tests of the whole do, by 64 bits
            whole = y[b, done[b]:done[b] + n[b]].float()
            assert torch.allclose(out[b, :n[b]].float(), whole, rtol=1e-4 if dt == F32 else 2 ** -7, atol=1e-4), chunk
            done[b] += n[b]
    check_fwd(s, (y, state))


def test_optional_outputs_and_repeatability():
    for T in (40, 900):
        s = make(2, T, 130, BF16, [T, T - 9])
        y, last = check_fwd(s)
        y2, none = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], need=("y",))
        assert none is None and torch.equal(y, y2)
        full = check_bwd(s, y)
        for need in (("dx",), ("dr", "ddecay"), ("dg", "dh0"), ("ddecay",), ("dh0",)):
            for name, a, b in zip(NAMES, full, grads(s, y, need=need)):
                assert b is None if name not in need else torch.equal(a, b)


def test_gradients_against_differences():
    """<dL, v> against (L(+e) - L(-e)) / 2e, L = <y, dy> + <h_last, dh> in fp64 of fp32 outputs.  The forward's rounding leaves about
    sqrt(N) 1e-6 / e, the curvature about e^2: with N = 2 * 50 * 20 and e = 1e-2 both are under 1e-2."""
    s = make(2, 50, 20, F32, [50, 31])
    s["decay"].clamp_(-6, 0)
    keys = ("x", "r", "g", "decay", "h0")

    def loss(t):
        y, last = lib().dwscan_fwd(*t[:4], s["lengths"], h0=t[4])
        return float((y.double() * s["dy"].double()).sum() + (last.double() * s["dh_last"].double()).sum())
    at = [s[k] for k in keys]
    got = grads(s, lib().dwscan_fwd(*at[:4], s["lengths"], h0=at[4])[0])
    for i, g in enumerate(got):
        v = datagen.normal(tuple(at[i].shape), 1.0, f"scan/dir/{i}", device=DEV)
        v /= v.norm()
        up, down = ([a + f * v if k == i else a for k, a in enumerate(at)] for f in (1e-2, -1e-2))
        diff, exact = (loss(up) - loss(down)) / 2e-2, float((g.double() * v.double()).sum())
        assert abs(diff - exact) <= 1e-2 * max(1.0, abs(exact)), (keys[i], diff, exact)


@pytest.mark.parametrize("T", [12, 800])
def test_items_past_32_bit_offsets(T):
    """Items 2^31 + 3 elements apart: the second lies past 4 GB of the first."""
    B, C = 2, 68
    s = make(B, T, C, BF16, [T, T - 2])
    far = (1 << 31) + 3
    big = torch.empty(far + T * C, dtype=BF16, device=DEV)
    place = lambda t: big.as_strided((B, T, C), (far, C, 1)).copy_(t)  # noqa: E731
    for k in ("x", "r", "g", "dy"):
        want = check_fwd(s)
        grad = check_bwd(s, want[0])
        keep = s[k]
        s[k] = place(keep)
        got = lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"])
        assert torch.equal(got[0], want[0])
        for a, b in zip(grads(s, want[0]), grad):
            assert torch.equal(a, b)
        s[k] = keep
    y = big.as_strided((B, T, C), (far, C, 1))
    lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], y=y)
    assert torch.equal(y, want[0])
    for a, b in zip(grads(s, y), grad):
        assert torch.equal(a, b)
    into = big.as_strided((B, T, C), (far, C, 1))
    assert torch.equal(grads(s, want[0], dx=into)[0], grad[0])


def test_frames_past_32_bit_offsets():
    """Frames 2^22 + 1 elements apart: a tile spans more than 2^29 of them, the sequence more than 2^31."""
    T, C, fs = 600, 8, (1 << 22) + 1
    s = make(1, T, C, BF16)
    want = check_fwd(s)
    big = torch.empty((T - 1) * fs + C, dtype=BF16, device=DEV)
    x = big.as_strided((1, T, C), (0, fs, 1)).copy_(s["x"])
    got = lib().dwscan_fwd(x, s["r"], s["g"], s["decay"], h0=s["h0"])
    assert torch.equal(got[0], want[0])
    y = big.as_strided((1, T, C), (0, fs, 1))
    lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], h0=s["h0"], y=y)
    assert torch.equal(y, want[0])
    for a, b in zip(grads(s, y), grads(s, want[0])):
        assert torch.equal(a, b)


def test_on_another_stream_and_two_at_once():
    s = [make(2, T, 200, BF16, [T, T // 2]) for T in (30, 1000)]
    want = [(check_fwd(a), None) for a in s]
    want = [(f, check_bwd(a, f[0])) for a, (f, _) in zip(s, want)]
    streams = [torch.cuda.Stream() for _ in s]
    torch.cuda.synchronize()
    got = []
    for a, side in zip(s, streams):
        with torch.cuda.stream(side):
            f = lib().dwscan_fwd(a["x"], a["r"], a["g"], a["decay"], a["lengths"], h0=a["h0"])
            got.append((f, grads(a, f[0])))
    torch.cuda.synchronize()
    for (wf, wb), (gf, gb) in zip(want, got):
        for a, b in zip(wf + wb, gf + gb):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [1, 20, 700])
def test_captured(T):
    """A stream's step and a training step in a graph, replayed over new inputs, against eager calls."""
    dw = lib()
    s = make(2, T, 72, BF16, [T, max(0, T - 1)])
    o = {n: torch.empty_like(s["x"]) for n in ("y", "dx", "dr", "dg")}
    state, dh0, dd = s["h0"].clone(), torch.empty_like(s["h0"]), torch.empty((72,), device=DEV)
    ws = [torch.empty((max(16, n),), dtype=torch.uint8, device=DEV) for n in (dw.dwscan_fwd_workspace_bytes(2, T, 72), dw.dwscan_bwd_workspace_bytes(2, T, 72))]
    start = torch.empty_like(state)

    def step():
        start.copy_(state)
        dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=state, h_last=state, y=o["y"], workspace=ws[0])
        grads(s | {"h0": start}, o["y"], dx=o["dx"], dr=o["dr"], dg=o["dg"], ddecay=dd, dh0=dh0, workspace=ws[1])
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        s["x"].copy_(datagen.normal((2, T, 72), 1.0, f"scan/graph/{k}", device=DEV))
        before = state.clone()
        for t in (*o.values(), dd, dh0):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*o.values(), dd, dh0, state)]
        state.copy_(before)
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (*o.values(), dd, dh0, state)):
            assert torch.equal(a, b)


def test_two_graphs_of_one_workspace():
    """Linked tiles in two captured graphs that share their workspace, replayed in turn with eager calls between."""
    dw = lib()
    sizes = ((2, 700), (1, 1500))
    n = max(f(B, T, 72) for B, T in sizes for f in (dw.dwscan_fwd_workspace_bytes, dw.dwscan_bwd_workspace_bytes))
    ws = torch.empty((n,), dtype=torch.uint8, device=DEV)
    problems, graphs, want = [], [], []
    for B, T in sizes:
        s = make(B, T, 72, BF16, [T] * B)
        o = {k: torch.empty_like(s["x"]) for k in ("y", "dx", "dr", "dg")}
        o |= {"ddecay": torch.empty((72,), device=DEV), "dh0": torch.empty_like(s["h0"])}

        def step(s=s, o=o):
            dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], y=o["y"], workspace=ws, need=("y",))
            grads(s, o["y"], workspace=ws, **{k: t for k, t in o.items() if k != "y"})
        step()
        torch.cuda.synchronize()
        want.append({k: t.clone() for k, t in o.items()})
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        problems.append((step, o))
        graphs.append(g)
    for k in range(4):
        for (step, o), g, w in zip(problems, graphs, want):
            for t in o.values():
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            for name, t in o.items():
                assert torch.equal(t, w[name]), (k, name)
            step()


def test_a_scale_that_changes():
    """The scale is the value given, not the object that gave it."""
    dw = lib()
    s = make(2, 9, 16, F32, [9, 9])
    scale, out = torch.tensor(8.0), []
    for v in (8.0, 2.0, 8.0):
        scale.fill_(v)
        out.append(dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], scale=scale)[0])
        assert torch.equal(out[-1], dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], scale=v)[0])
    assert torch.equal(out[0], out[2]) and not torch.equal(out[0], out[1])


def test_binding_refusals():
    dw = lib()
    x, d, m = torch.zeros((2, 3, 16), device=DEV), torch.zeros(16, device=DEV), torch.zeros((2, 16), device=DEV)
    with pytest.raises(TypeError):
        dw.dwscan_fwd(x.half(), x.half(), x.half(), d)
    with pytest.raises(ValueError):
        dw.dwscan_fwd(x[0], x[0], x[0], d)
    with pytest.raises(TypeError):
        dw.dwscan_fwd(x, x.bfloat16(), x, d)
    with pytest.raises(ValueError):
        dw.dwscan_fwd(x, x[:, :2], x, d)
    with pytest.raises(ValueError, match="next to each other"):
        dw.dwscan_fwd(x, torch.zeros((2, 16, 3), device=DEV).transpose(1, 2), x, d)
    with pytest.raises(TypeError):
        dw.dwscan_fwd(x, x, x, d.bfloat16())
    with pytest.raises(ValueError):
        dw.dwscan_fwd(x, x, x, d, h0=m[:1])
    with pytest.raises(ValueError, match="cpu"):
        dw.dwscan_fwd(x, x, x, d.cpu())
    with pytest.raises(dw.DwconvError, match="scale"):
        dw.dwscan_fwd(x, x, x, d, scale=-1.0)
    with pytest.raises(dw.DwconvError, match="alias"):
        dw.dwscan_fwd(x, x, x, d, y=x)
    with pytest.raises(dw.DwconvError, match="alias"):
        dw.dwscan_bwd(x, x, x, d, x, x, dx=x)
    with pytest.raises(dw.DwconvError, match="workspace"):
        dw.dwscan_bwd(x, x, x, d, x, x, workspace=torch.zeros(8, dtype=torch.uint8, device=DEV))


def test_tensors_of_the_host_are_refused():
    dw = lib()
    x, d = torch.zeros((2, 3, 16)), torch.zeros(16)
    with pytest.raises(ValueError):
        dw.dwscan_fwd(x, x, x, d)
    with pytest.raises(ValueError):
        dw.dwscan_bwd(x, x, x, d, x, x)
