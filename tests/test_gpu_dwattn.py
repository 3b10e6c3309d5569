"""Attention with a bucketed relative position bias, forward, against the
definition in 64 bits.

Tolerances.  Scores here stay below 32 in units of log2, so float32 arithmetic
moves a weight by at most a few 2^-24 * 32 of itself, and out, a weighted mean
of values below 6, by less than 2e-5.  bf16: each weight is rounded once, by at
most 2^-8 of itself, and so is out: 2^-8 * (max |v|) holds the two together
unless the weights' errors all have the sign of their values while the values
all lie near the largest.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import datagen
from gpu_util import Guarded, host64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16


def lib():
    import conv_subsampling_amd as dw
    return dw


def make(B, Tq, Tk, H, Hkv, D, dt, NB=16, reach=40, q_len=None, k_len=None, pos=None, left=-1, right=-1, bias=True, seed=0):
    tag = f"attn/{B}/{Tq}/{Tk}/{H}/{D}/{seed}"
    n = lambda shape, name, var=1.0: datagen.normal(shape, var, f"{tag}/{name}", device=DEV).to(dt)  # noqa: E731
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    s = dict(B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, D=D, dt=dt, left=left, right=right, q=n((B, Tq, H, D), "q"),
             k=n((B, Tk, Hkv, D), "k"), v=n((B, Tk, Hkv, D), "v"), dout=n((B, Tq, H, D), "do"), table=None, buckets=None,
             q_lengths=i32(q_len), k_lengths=i32(k_len), q_pos=i32(pos))
    if bias:
        s["table"], s["buckets"] = n((NB, H), "t"), lib().rel_buckets(NB, reach, device=DEV)
    return s


def call(s, **kw):
    return lib().dwattn_fwd(s["q"], s["k"], s["v"], s["table"], s["buckets"], s["q_lengths"], s["k_lengths"], s["q_pos"],
                            s["left"], s["right"], **kw)


def host(s):
    B, Tq, Tk = s["B"], s["Tq"], s["Tk"]
    h = lambda t: None if t is None else host64(t)  # noqa: E731
    ints = lambda t, d: [d] * B if t is None else t.tolist()  # noqa: E731
    return (h(s["q"]), h(s["k"]), h(s["v"]), h(s["table"]), None if s["buckets"] is None else s["buckets"].tolist(),
            ints(s["q_lengths"], Tq), ints(s["k_lengths"], Tk), ints(s["q_pos"], 0), s["left"], s["right"], s["D"] ** -0.5)


def check(s, got=None, what=""):
    out, lse = got or call(s)
    torch.cuda.synchronize()
    want, wlse = ref.attn(*host(s))
    g, gl = host64(out), host64(lse)
    assert np.isfinite(g).all(), what
    tol = 2e-5 + (ref.U16 * np.abs(host64(s["v"])).max(initial=0) if s["dt"] == BF16 else 0)
    assert np.abs(g - want).max(initial=0) <= tol, f"{what}: out off by {np.abs(g - want).max():.3e}"
    empty = np.isinf(wlse)
    assert np.array_equal(empty, np.isinf(gl)) and (gl[empty] < 0).all(), what
    assert np.abs(gl[~empty] - wlse[~empty]).max(initial=0) <= 1e-5 * (1 + np.abs(wlse[~empty]).max(initial=0)), what
    assert not g[empty.transpose(0, 2, 1)].any(), what
    return out, lse


DT = pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])


@DT
@pytest.mark.parametrize("D", [1, 7, 16, 32, 44, 50, 64, 72, 96, 100, 127, 128])
def test_head_widths(D, dt):
    check(make(2, 70, 70, 2, 2, D, dt, q_len=[70, 41], k_len=[70, 41]))


@DT
@pytest.mark.parametrize("Tq,Tk", [(1, 1), (1, 33), (31, 32), (33, 65), (64, 64), (127, 129), (129, 260), (300, 7)])
def test_lengths_around_the_tiles(Tq, Tk, dt):
    check(make(2, Tq, Tk, 3, 3, 64, dt))


@DT
@pytest.mark.parametrize("B,H", [(48, 4), (1, 2)])
def test_both_forms_over_several_tiles(B, H, dt):
    """Enough workgroups for 128 queries each, and few enough to split the keys."""
    check(make(B, 200, 200, H, H, 64 if B > 1 else 128, dt, q_len=[200 - b for b in range(B)],
               k_len=[200 - b for b in range(B)]))


@DT
def test_shared_key_heads(dt):
    check(make(2, 50, 90, 8, 2, 32, dt, pos=[40, 0]))
    check(make(2, 1, 200, 6, 1, 64, dt, pos=[199, 100]))


@DT
@pytest.mark.parametrize("Tq,H,Hkv,D,reach", [(1, 8, 1, 64, 40), (1, 32, 1, 32, 8), (4, 8, 1, 50, 40), (7, 8, 2, 128, 40),
                                              (3, 4, 2, 96, 40), (16, 4, 2, 64, 40), (1, 32, 1, 64, 1024), (2, 6, 3, 16, 40)])
def test_shared_key_heads_of_few_queries(Tq, H, Hkv, D, reach, dt):
    """A group's heads side by side in one tile (and, at the largest reach, not): ragged queries, windows, splits."""
    check(make(3, Tq, 300, H, Hkv, D, dt, reach=reach, NB=32 if reach > 8 else 16, k_len=[300, 5, 131],
               q_len=[Tq, max(Tq - 1, 1), Tq], pos=[300 - Tq, 0, 100]))
    check(make(2, Tq, 700, H, Hkv, D, dt, reach=reach, NB=16, k_len=[700, 333], pos=[650, 330], left=200, right=3))
    check(make(2, Tq, 90, H, Hkv, D, dt, bias=False, q_len=[Tq, 0]))


@DT
@pytest.mark.parametrize("left,right", [(-1, 0), (0, 0), (5, -1), (30, 10), (0, 40), (1000000000000, 3)])
def test_context_windows(left, right, dt):
    check(make(2, 150, 150, 2, 2, 64, dt, q_len=[150, 77], k_len=[150, 77], left=left, right=right))


@DT
def test_queries_without_keys(dt):
    """Empty items, windows that leave rows nothing, positions far outside the keys."""
    s = make(6, 90, 100, 2, 2, 64, dt, q_len=[0, 90, -3, 50, 90, 200], k_len=[100, 0, 7, -2, 100, 300],
             pos=[0, 0, 0, 0, 80, 0], left=20, right=5)
    out, lse = check(s)
    assert torch.isinf(lse[4, :, 60:]).all()  # 80 + 60 - 20 is past the last key
    for far in (2_000_000_000, -2_000_000_000):
        check(make(2, 40, 60, 2, 2, 32, dt, pos=[far, 3]))
        check(make(2, 40, 60, 2, 2, 32, dt, pos=[far, 3], left=50, right=50))


@DT
def test_streaming_chunks_and_steps_over_a_cache(dt):
    """Chunks of 1 and 8 frames over caches of different fill; the split key axis against the whole utterance."""
    for Tq, Tk, k_len in ((1, 700, [700, 1, 333]), (8, 520, [520, 8, 131]), (40, 2500, [2500, 41, 1300])):
        pos = [n - Tq for n in k_len]
        for left, right in ((-1, -1), (300, Tq - 1)):
            s = make(3, Tq, Tk, 4, 4, 64, dt, k_len=k_len, pos=pos, left=left, right=right)
            assert lib().dwattn_fwd_workspace_bytes(s["q"], s["k"], s["v"], left, right) > 0
            check(s, what=f"{Tq} {Tk} {left}")


@DT
def test_masked_frames_are_not_read(dt):
    s = make(3, 100, 100, 2, 2, 64, dt, q_len=[100, 37, 0], k_len=[100, 64, 5])
    want = call(s)
    for name, L in (("q", s["q_lengths"]), ("k", s["k_lengths"]), ("v", s["k_lengths"])):
        s[name] = s[name].clone()
        for b in range(3):
            s[name][b, int(L[b]):] = float("nan") if name != "k" else float("inf")
    got = call(s)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@DT
def test_bias_of_the_lowest_value_and_of_minus_infinity(dt):
    """-inf forbids a bucket; the type's lowest value does too, unless a row holds nothing else: then it weighs alike."""
    low = torch.finfo(dt).min
    s = make(1, 60, 60, 2, 2, 32, dt, NB=8, reach=20)
    s["table"][0] = float("-inf")
    s["table"][5] = low
    check(s)
    s = make(1, 60, 60, 1, 1, 32, dt, NB=8, reach=20)
    s["table"][:] = low
    out, lse = call(s)
    torch.cuda.synchronize()
    tol = 2e-5 + (2 * ref.U16 * host64(s["v"]).max() if dt == BF16 else 0)
    assert np.abs(host64(out)[0, :, 0] - host64(s["v"])[0, :, 0].mean(0)).max() <= tol
    s["table"][:] = float("-inf")
    out, lse = call(s)
    assert not out.any() and torch.isinf(lse).all()


def test_large_scores_and_a_rising_maximum():
    """Scores that grow along the keys by hundreds, past every rescaling step."""
    s = make(1, 40, 300, 1, 1, 32, F32, bias=False)
    s["k"] = s["k"] * torch.linspace(0, 40, 300, device=DEV)[None, :, None, None]
    got = call(s)
    torch.cuda.synchronize()
    want, wlse = ref.attn(*host(s))
    # scores up to about 1000 are off by 2^-24 of themselves times their depth's square root, and weights with them
    assert np.abs(host64(got[1]) - wlse).max() <= 2e-3 and np.abs(host64(got[0]) - want).max() <= 5e-3


@DT
def test_strided_inputs_and_guard_bands(dt):
    """Slices of one projection's output, a cache with other strides, an odd start, a broadcast input; guarded outputs."""
    B, T, H, D = 2, 75, 3, 40
    s = make(B, T, T, H, H, D, dt)
    qkv = torch.cat([s["q"], s["k"], s["v"]], 2).view(B, T, 3, H, D)
    want = check(s)
    s["q"], s["k"], s["v"] = qkv.unbind(2)
    cache = torch.empty((H, B, T + 5, D + 3), dtype=dt, device=DEV)
    odd = cache[:, :, 3:T + 3, 1:D + 1].permute(1, 2, 0, 3)
    odd.copy_(s["k"])
    s["k"] = odd
    o, l = Guarded((B, T, H, D), dt, DEV), Guarded((B, H, T), F32, DEV)
    got = call(s, out=o.t, lse=l.t)
    torch.cuda.synchronize()
    o.check("out"), l.check("lse")
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    s["v"] = s["v"][:1, :, :1].expand(B, T, H, D)
    check(s)


def test_workspace_is_exactly_used():
    s = make(2, 1, 3000, 2, 2, 50, BF16, pos=[2999, 100])
    n = lib().dwattn_fwd_workspace_bytes(s["q"], s["k"], s["v"])
    ws = Guarded((n,), torch.uint8, DEV, G=4096)
    check(s, call(s, workspace=ws.t))
    ws.check("workspace")
    with pytest.raises(lib().DwconvError, match="workspace"):
        call(s, workspace=ws.t[:n - 1])


def test_map_past_the_table_and_one_bucket():
    s = make(1, 40, 40, 2, 2, 32, F32)
    good = call(s)
    low, high = int(s["buckets"].argmin()), int(s["buckets"].argmax())
    s["buckets"][low], s["buckets"][high] = -5, 1 << 30  # held to the table's first and last bucket
    assert s["buckets"].shape and torch.equal(good[0], call(s)[0])
    s = make(1, 40, 40, 2, 2, 32, F32, NB=2, reach=1)
    check(s)
    check(make(1, 300, 300, 1, 1, 32, F32, NB=64, reach=1024))
    check(make(1, 40, 40, 2, 2, 32, F32, bias=False))


def test_empty_problems():
    for B, Tq, Tk in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        out, lse = call(make(B, Tq, Tk, 2, 2, 32, F32))
        torch.cuda.synchronize()
        assert not out.any() and torch.isinf(lse).all()


def test_a_cache_whose_offsets_pass_32_bits():
    """A key cache over 4 GiB: the last frames' offsets need more than 32 bits."""
    D, H, Tk = 64, 2, 70_000
    frame = 33_000                                     # elements from frame to frame: the cache spans 4.6 GB in bf16
    store = torch.zeros((Tk * frame,), dtype=BF16, device=DEV)
    k = store.as_strided((1, Tk, H, D), (0, frame, D, 1))
    v = store.as_strided((1, Tk, H, D), (0, frame, D, 1), 128)
    k.copy_(datagen.normal((1, Tk, H, D), 1.0, "far/k", device=DEV))
    v.copy_(datagen.normal((1, Tk, H, D), 1.0, "far/v", device=DEV))
    s = make(1, 1, 8, H, H, D, BF16, pos=[Tk - 1])
    s["Tk"], s["k"], s["v"] = Tk, k, v
    check(s)


def test_on_another_stream_and_in_a_graph():
    s = make(2, 8, 500, 4, 4, 64, BF16, k_len=[500, 300], pos=[492, 292])
    want = call(s)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(s)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty((lib().dwattn_fwd_workspace_bytes(s["q"], s["k"], s["v"]),), dtype=torch.uint8, device=DEV)
    call(s, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(s, out=out, lse=lse, workspace=ws)
    for n in (500, 499, 17, 500):
        s["k_lengths"][0] = n
        s["q_pos"][0] = n - 8
        out.fill_(float("nan")), lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        a, b = out.clone(), lse.clone()
        eager = call(s)
        torch.cuda.synchronize()
        assert torch.equal(a, eager[0]) and torch.equal(b, eager[1])


@pytest.mark.parametrize("buckets,reach,both", [(32, 128, True), (32, 128, False), (16, 64, True), (2, 1, True), (1, 5, False),
                                                (10, 33, True), (512, 1024, True)])
def test_bucket_map(buckets, reach, both):
    got = lib().rel_buckets(buckets, reach, both, device="cpu").tolist()
    assert got == [ref.bucket(r, buckets, reach, both) for r in range(-reach, reach + 1)]


def test_binding_refusals():
    dw = lib()
    s = make(1, 8, 8, 2, 2, 32, F32)
    a = (s["q"], s["k"], s["v"])
    with pytest.raises(ValueError, match="buckets"):
        dw.dwattn_fwd(*a, s["table"])
    with pytest.raises(ValueError, match="next to each other"):
        dw.dwattn_fwd(s["q"].transpose(2, 3).contiguous().transpose(2, 3), s["k"], s["v"])
    with pytest.raises(TypeError):
        dw.dwattn_fwd(s["q"], s["k"].bfloat16(), s["v"])
    with pytest.raises(dw.DwconvError, match="multiple"):
        dw.dwattn_fwd(torch.zeros((1, 8, 3, 32), device=DEV), s["k"], s["v"])
    with pytest.raises(dw.DwconvError, match="128"):
        z = torch.zeros((1, 8, 1, 129), device=DEV)
        dw.dwattn_fwd(z, z, z)
    with pytest.raises(dw.DwconvError, match="1024"):
        dw.dwattn_fwd(*a, s["table"], torch.zeros(2051, dtype=torch.int32, device=DEV))
    with pytest.raises(dw.DwconvError, match="alias"):
        dw.dwattn_fwd(*a, out=s["q"])
    for bad in ((32, 8), (0, 9), (32, 2000)):
        with pytest.raises(dw.DwconvError):
            dw.rel_buckets(*bad)


def far_and_near(dt, far, T=200, seed=0):
    """Rows whose tiles lie within and past the map's reach, the far buckets of one value, and one far pair with a
    product of 1120 (a score of 198) that no other pair shares."""
    s = make(1, T, T, 2, 1, 32, dt, NB=8, reach=20, seed=seed)
    for r in (0, -1):
        s["table"][int(s["buckets"][r])] = far
    s["q"][..., 0], s["k"][..., 0] = 0, 0
    s["q"][0, 130, :, 0], s["k"][0, 10, 0, 0] = 80, 14
    return s


@DT
@pytest.mark.parametrize("far", ["lowest", -1e30, -1e10, -1e6])
def test_far_buckets_of_a_huge_negative_value(far, dt):
    """The forbidden pair's score vanishes in its bias: the row stays finite and goes by its near keys."""
    check(far_and_near(dt, torch.finfo(dt).min if far == "lowest" else far), what=str(far))


@DT
@pytest.mark.parametrize("sign", [-1, 1])
def test_rows_of_nothing_but_the_lowest_or_largest_value(sign, dt):
    """A table of the lowest value alone weighs near and far keys alike; far buckets at the largest, only the far ones."""
    T = 200
    s = far_and_near(dt, sign * torch.finfo(dt).max, T)
    if sign < 0:
        s["table"][:] = torch.finfo(dt).min
    out, _ = call(s)
    torch.cuda.synchronize()
    place = np.asarray(s["buckets"].tolist())[np.clip(np.arange(T)[None, :] - np.arange(T)[:, None], -20, 20) + 20]
    w = np.ones((T, T)) if sign < 0 else np.isin(place, [place[-1, 0], place[0, -1]]).astype(float)
    v = host64(s["v"])[0, :, 0]
    want = w @ v / w.sum(1, keepdims=True)
    # equal weights: one float32 sum of at most 200 terms; bf16 rounds out
    tol = 2e-5 + (ref.U16 * np.abs(v).max() if dt == BF16 else 0)
    assert np.abs(host64(out)[0] - want[:, None]).max() <= tol


def test_rows_whose_elements_pass_32_bits():
    """2^26 rows of 128: outputs of 17 GB.  With one key its weight is 1, and every row is that item's value."""
    B, T, D = 1 << 20, 64, 128
    q = torch.ones((1, 1, 1, D), dtype=BF16, device=DEV).expand(B, T, 1, D)
    k, v = (datagen.normal((B, 1, 1, D), 1.0, f"rows/{n}", device=DEV).to(BF16) for n in "kv")
    out, lse = lib().dwattn_fwd(q, k, v)
    torch.cuda.synchronize()
    for b in (0, 1, B // 2 + 1, B - 1):
        assert torch.equal(out[b], v[b].expand(T, 1, D))
    assert torch.equal(out[::4097].float().sum((1, 2)), v[::4097].float().sum((1, 2)) * T)
    want = k.float().sum(-1) * D ** -0.5          # [B, 1, 1]; sums of 128 terms in another order
    assert float((lse - want.view(B, 1, 1)).abs().max()) <= 128 * ref.U32 * 100
