"""Attention with a bucketed relative position bias, gradients, against the
definition in 64 bits (given the forward's rounded out, as the call is).

Tolerances.  P and dS come from float32 scores below 32 in units of log2 and
dot products of at most 128 terms: each is off by at most 2^-24 * 64 of its
terms' sizes.  dq, dk, dv and dtable are sums of such terms, so they are held to
2e-5 of the sum of absolute terms that bounds them.  bf16 (8 significant bits:
a rounding moves a value by at most 2^-8 of itself) rounds P and dS for the
products with dout, q and k, each term once, and the gradient once.
dtable takes no such rounding.
"""
import numpy as np
import pytest
import torch

import block_ref as ref
import datagen
from gpu_util import Guarded, host64
from test_gpu_dwattn import BF16, DEV, DT, F32, call, far_and_near, host, lib, make

pytestmark = pytest.mark.gpu


def grads(s, out, lse, **kw):
    return lib().dwattn_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], s["table"], s["buckets"], s["q_lengths"],
                            s["k_lengths"], s["q_pos"], s["left"], s["right"], **kw)


def absolute(a):
    """The same gradients with every term made positive: a bound of the sums' terms."""
    q, k, v, table, buckets, q_len, k_len, pos, left, right, scale, dout, out, lse = a
    B, Tq, H, D = q.shape
    G = H // k.shape[2]
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    R = 0 if buckets is None else len(buckets) // 2
    for b in range(B):
        nq, nk = int(np.clip(q_len[b], 0, Tq)), int(np.clip(k_len[b], 0, k.shape[1]))
        if not nq or not nk:
            continue
        rel = np.arange(nk)[None, :] - np.arange(nq)[:, None] - int(pos[b])
        seen = ((left < 0) | (rel >= -left)) & ((right < 0) | (rel <= right))
        for h in range(H):
            S = scale * q[b, :nq, h] @ k[b, :nk, h // G].T
            if table is not None:
                S = S + table[np.asarray(buckets)[np.clip(rel, -R, R) + R], h]
            ls = lse[b, h, :nq, None]
            P = np.where(np.isinf(ls) | ~seen, 0, np.exp(S - np.where(np.isinf(ls), 0, ls)))
            do = np.abs(dout[b, :nq, h])
            dS = P * (do @ np.abs(v[b, :nk, h // G]).T + (do * np.abs(out[b, :nq, h])).sum(1, keepdims=True))
            bq[b, :nq, h] = scale * dS @ np.abs(k[b, :nk, h // G])
            bk[b, :nk, h // G] += scale * dS.T @ np.abs(q[b, :nq, h])
            bv[b, :nk, h // G] += P.T @ do
    return bq, bk, bv


def check(s, what="", got=None, fwd=None):
    out, lse = fwd or call(s)
    got = got or grads(s, out, lse)
    torch.cuda.synchronize()
    a = host(s) + (host64(s["dout"]), host64(out), host64(lse))
    want, bound = ref.attn(*a), absolute(a)
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        g = host64(g)
        assert np.isfinite(g).all(), f"{what} {name}"
        tol = 2e-5 * (b + 1e-6) + (ref.U16 * b + ref.U16 * np.abs(w) if s["dt"] == BF16 else 0)
        off = np.abs(g - w)
        assert (off <= tol).all(), f"{what} {name}: {off.max():.3e} at {np.argwhere(off > tol)[0]}"
        assert not g[b == 0].any(), f"{what} {name}: not zero where nothing flows"
    if s["table"] is None:
        assert got[3] is None
    else:
        off = np.abs(host64(got[3]) - want[3])
        # dS itself is off by up to 2e-5 of its absolute terms, which exceed |dS|: the terms' bound, bucket by bucket
        at = table_bound(a)
        assert (off <= 2e-5 * (at + 1e-6)).all(), f"{what} dtable: {off.max():.3e} of {at.min():.3e}"
    return got


def table_bound(a):
    """Sums over each bucket of P * (|dout| . |v| + |dout| . |out|)."""
    q, k, v, table, buckets, q_len, k_len, pos, left, right, scale, dout, out, lse = a
    t = np.zeros_like(table)
    B, Tq, H, D = q.shape
    G, R = H // k.shape[2], len(buckets) // 2
    for b in range(B):
        nq, nk = int(np.clip(q_len[b], 0, Tq)), int(np.clip(k_len[b], 0, k.shape[1]))
        if not nq or not nk:
            continue
        rel = np.arange(nk)[None, :] - np.arange(nq)[:, None] - int(pos[b])
        seen = ((left < 0) | (rel >= -left)) & ((right < 0) | (rel <= right))
        place = np.asarray(buckets)[np.clip(rel, -R, R) + R]
        for h in range(H):
            ls = lse[b, h, :nq, None]
            x = scale * q[b, :nq, h] @ k[b, :nk, h // G].T + table[place, h]
            P = np.where(np.isinf(ls) | ~seen, 0, np.exp(x - np.where(np.isinf(ls), 0, ls)))
            do = np.abs(dout[b, :nq, h])
            np.add.at(t[:, h], place, P * (do @ np.abs(v[b, :nk, h // G]).T +
                                           (do * np.abs(out[b, :nq, h])).sum(1, keepdims=True)))
    return t


@DT
@pytest.mark.parametrize("D", [1, 7, 32, 44, 50, 64, 96, 100, 127, 128])
def test_head_widths(D, dt):
    check(make(2, 70, 70, 2, 2, D, dt, q_len=[70, 41], k_len=[70, 41]))


@DT
@pytest.mark.parametrize("Tq,Tk", [(1, 1), (1, 33), (31, 32), (33, 65), (64, 64), (127, 129), (129, 260), (300, 7)])
def test_lengths_around_the_tiles(Tq, Tk, dt):
    check(make(2, Tq, Tk, 3, 3, 64, dt))


@DT
def test_shared_key_heads(dt):
    check(make(2, 50, 90, 8, 2, 32, dt, pos=[40, 0]))
    check(make(2, 140, 140, 6, 1, 64, dt, left=30, right=11))


@DT
@pytest.mark.parametrize("left,right", [(-1, 0), (0, 0), (5, -1), (30, 10), (0, 40), (1000000000000, 3)])
def test_context_windows(left, right, dt):
    check(make(2, 150, 150, 2, 2, 64, dt, q_len=[150, 77], k_len=[150, 77], left=left, right=right))


@DT
@pytest.mark.parametrize("NB,reach", [(2, 1), (16, 5), (16, 31), (32, 128), (64, 1024)])
def test_reach_below_at_and_past_the_tiles(NB, reach, dt):
    check(make(1, 300, 300, 2, 2, 32, dt, NB=NB, reach=reach))


@DT
def test_queries_without_keys_and_keys_without_queries(dt):
    check(make(6, 90, 100, 2, 2, 64, dt, q_len=[0, 90, -3, 50, 90, 200], k_len=[100, 0, 7, -2, 100, 300],
               pos=[0, 0, 0, 0, 80, 0], left=20, right=5))
    for far in (2_000_000_000, -2_000_000_000):
        check(make(2, 40, 60, 2, 2, 32, dt, pos=[far, 3]))
        check(make(2, 40, 60, 2, 2, 32, dt, pos=[far, 3], left=50, right=50))


@DT
def test_masked_frames_are_not_read(dt):
    s = make(3, 100, 100, 2, 2, 64, dt, q_len=[100, 37, 0], k_len=[100, 64, 5])
    out, lse = call(s)
    want = grads(s, out, lse)
    out, lse = out.clone(), lse.clone()
    for b in range(3):
        nq, nk = int(s["q_lengths"][b]), int(s["k_lengths"][b])
        lse[b, :, nq:] = float("nan")
        for t, n in ((s["q"], nq), (s["k"], nk), (s["v"], nk), (s["dout"], nq), (out, nq)):
            t[b, n:] = float("nan") if t is not s["v"] else float("inf")
    for a, b in zip(want, grads(s, out, lse)):
        assert torch.equal(a, b)


@DT
def test_bias_of_the_lowest_value_and_of_minus_infinity(dt):
    s = make(1, 60, 60, 2, 2, 32, dt, NB=8, reach=20)
    s["table"][0], s["table"][5] = float("-inf"), torch.finfo(dt).min
    out, lse = call(s)
    got = grads(s, out, lse)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(g).all()) for g in got) and not got[3][0].any() and not got[3][5].any()
    check(s, got=got, fwd=(out, lse))


@DT
def test_a_training_batch(dt):
    check(make(3, 375, 375, 4, 4, 64, dt, NB=32, reach=128, q_len=[375, 300, 188], k_len=[375, 300, 188]))
    check(make(1, 260, 260, 2, 2, 128, dt, NB=32, reach=100))


@DT
def test_without_a_bias_and_partial_requests(dt):
    s = make(2, 150, 150, 2, 2, 64, dt, bias=False)
    check(s)
    s = make(2, 150, 150, 2, 1, 64, dt)
    out, lse = call(s)
    full = grads(s, out, lse)
    for need in (("dq",), ("dk",), ("dv",), ("dtable",), ("dk", "dtable")):
        for name, a, b in zip(("dq", "dk", "dv", "dtable"), full, grads(s, out, lse, need=need)):
            assert b is None if name not in need else torch.equal(a, b)


@DT
def test_strides_and_guard_bands(dt):
    """Gradients written into slices of one projection's gradient; canaries around outputs and workspace."""
    B, T, H, D = 2, 75, 3, 40
    s = make(B, T, T, H, H, D, dt)
    out, lse = call(s)
    want = check(s, fwd=(out, lse))
    qkv = torch.cat([s["q"], s["k"], s["v"]], 2).view(B, T, 3, H, D)
    s["q"], s["k"], s["v"] = qkv.unbind(2)
    g = Guarded((B, T, 3, H, D), dt, DEV)
    t = Guarded((16, H), F32, DEV)
    ws = Guarded((lib().dwattn_bwd_workspace_bytes(s["q"], s["k"], s["v"], s["table"], s["buckets"]),), torch.uint8, DEV,
                 G=4096)
    dq, dk, dv = g.t.unbind(2)
    got = grads(s, out, lse, dq=dq, dk=dk, dv=dv, dtable=t.t, workspace=ws.t)
    torch.cuda.synchronize()
    for n, x in (("gradients", g), ("dtable", t), ("workspace", ws)):
        x.check(n)
    assert g.untouched_inside() == 0
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    with pytest.raises(lib().DwconvError, match="workspace"):
        grads(s, out, lse, workspace=ws.t[:-1])


def test_empty_problems():
    for B, Tq, Tk in ((0, 4, 4), (2, 0, 4), (2, 4, 0)):
        s = make(B, Tq, Tk, 2, 2, 32, F32)
        out, lse = call(s)
        got = grads(s, out, lse)
        torch.cuda.synchronize()
        assert not any(bool(g.any()) for g in got)


def test_gradients_against_differences():
    """<dL, x> of the backward against (L(+h) - L(-h)) / 2h of the forward, L = <out, w> in fp64 of fp32 outputs.  The
    forward's rounding leaves about sqrt(N) * 3e-7 / h, the curvature about h^2: at h = 1e-2 and N = 2 * 40 * 2 * 32
    values both are under 3e-3."""
    dw = lib()
    s = make(2, 40, 40, 2, 1, 32, F32, q_len=[40, 25], k_len=[40, 25], left=30, right=20)
    names = ("q", "k", "v", "table")

    def loss(**t):
        return float((call({**s, **t})[0].double() * s["dout"].double()).sum())

    got = grads(s, *call(s))
    for name, g in zip(names, got):
        x = datagen.normal(tuple(s[name].shape), 1.0, f"dir/{name}", device=DEV)
        x /= x.norm()
        e = 1e-2
        diff = (loss(**{name: s[name] + e * x}) - loss(**{name: s[name] - e * x})) / (2 * e)
        exact = float((g.double() * x.double()).sum())
        assert abs(diff - exact) <= 3e-3 * max(1.0, abs(exact)), (name, diff, exact)


def test_on_another_stream_and_in_a_graph():
    s = make(2, 200, 200, 4, 2, 64, BF16, q_len=[200, 130], k_len=[200, 130])
    out, lse = call(s)
    want = grads(s, out, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = grads(s, out, lse)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    o = [torch.empty_like(w) for w in want]
    ws = torch.empty((lib().dwattn_bwd_workspace_bytes(s["q"], s["k"], s["v"], s["table"], s["buckets"]),),
                     dtype=torch.uint8, device=DEV)
    kw = dict(dq=o[0], dk=o[1], dv=o[2], dtable=o[3], workspace=ws)
    grads(s, out, lse, **kw)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        grads(s, out, lse, **kw)
    for k in range(3):
        s["dout"].normal_()
        for t in o:
            t.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        seen = [t.clone() for t in o]
        for a, b in zip(seen, grads(s, out, lse)):
            assert torch.equal(a, b)


def check_by_weights(s, absorbed, rel=2e-5, what=""):
    """The gradients and their terms' bounds from the softmax of the scores, instead of from lse: for rows whose lse
    says nothing.  A bias of magnitude `absorbed` or more swallows the products it is added to."""
    out, lse = call(s)
    got = grads(s, out, lse)
    torch.cuda.synchronize()
    q, k, v, table, buckets, q_len, k_len, pos, left, right, scale = host(s)
    do, o = host64(s["dout"]), host64(out)
    B, Tq, H, D = q.shape
    G, R = H // k.shape[2], len(buckets) // 2
    w = [np.zeros_like(x) for x in (q, k, v, table)]
    bound = [np.zeros_like(x) for x in w]
    for b in range(B):
        nq, nk = int(np.clip(q_len[b], 0, Tq)), int(np.clip(k_len[b], 0, k.shape[1]))
        rel_ = np.arange(nk)[None, :] - np.arange(nq)[:, None] - int(pos[b])
        seen = ((left < 0) | (rel_ >= -left)) & ((right < 0) | (rel_ <= right))
        place = np.asarray(buckets)[np.clip(rel_, -R, R) + R]
        for h in range(H):
            kk, vv, bias = k[b, :nk, h // G], v[b, :nk, h // G], table[place, h]
            S = np.where(np.abs(bias) >= absorbed, bias, scale * q[b, :nq, h] @ kk.T + bias)
            S = np.where(seen, S, -np.inf)
            P = np.exp(S - S.max(1, keepdims=True))
            P /= P.sum(1, keepdims=True)
            g, oo = do[b, :nq, h], o[b, :nq, h]
            dS = P * (g @ vv.T - (g * oo).sum(1, keepdims=True))
            aS = P * (np.abs(g) @ np.abs(vv).T + (np.abs(g) * np.abs(oo)).sum(1, keepdims=True))
            for into, ds, p, f in ((w, dS, P, lambda x: x), (bound, aS, P, np.abs)):
                into[0][b, :nq, h] = scale * ds @ f(kk)
                into[1][b, :nk, h // G] += scale * ds.T @ f(q[b, :nq, h])
                into[2][b, :nk, h // G] += p.T @ f(g)
                np.add.at(into[3][:, h], place, ds)
    for name, g, x, b in zip(("dq", "dk", "dv", "dtable"), got, w, bound):
        g = host64(g)
        assert np.isfinite(g).all(), f"{what} {name}"
        tol = rel * (b + 1e-6) + (ref.U16 * b + ref.U16 * np.abs(x) if s["dt"] == BF16 and name != "dtable" else 0)
        off = np.abs(g - x)
        assert (off <= tol).all(), f"{what} {name}: {off.max():.3e} at {np.argwhere(off > tol)[0]}"


@DT
@pytest.mark.parametrize("low", ["lowest", -1e30, -1e9, 1e9])
def test_rows_of_nothing_but_one_huge_bias(low, dt):
    """Such rows weigh their keys alike in both passes: over near and far tiles, ragged items, windows down to one key,
    shared key heads."""
    low = torch.finfo(dt).min if low == "lowest" else low
    for s in (make(2, 170, 170, 4, 2, 32, dt, NB=8, reach=20, q_len=[170, 101], k_len=[170, 101]),
              make(1, 90, 90, 2, 2, 50, dt, NB=8, reach=20, left=7, right=0),
              make(2, 5, 300, 2, 1, 128, dt, NB=8, reach=20, pos=[295, 7])):
        s["table"][:] = low
        check_by_weights(s, absorbed=1e8, what=str(s["Tq"]))


@DT
def test_rows_of_lowest_values_beside_ordinary_rows(dt):
    """Near buckets at the lowest value: the rows that see only near keys are uniform, the others ordinary; and far
    buckets at it, with a huge score among them."""
    low = torch.finfo(dt).min
    s = make(2, 170, 170, 2, 2, 64, dt, NB=8, reach=20, k_len=[170, 12])
    ends = [int(s["buckets"][0]), int(s["buckets"][-1])]
    for n in range(8):
        if n not in ends:
            s["table"][n] = low
    check_by_weights(s, absorbed=1e8)
    check_by_weights(far_and_near(dt, low), absorbed=1e8)
    check(far_and_near(dt, low))


@DT
def test_rows_of_a_large_bias(dt):
    """A whole table at -2000: scores near 2885 in units of log2 are rounded to 2^-13, twice, in both passes alike: a
    weight is off by 2 * 2^-13 * ln 2 = 1.7e-4 of itself, and its row's sum by as much."""
    s = make(2, 170, 170, 2, 2, 64, dt, NB=8, reach=20, q_len=[170, 99], k_len=[170, 99])
    s["table"][:] = -2000.0
    check_by_weights(s, absorbed=1e8, rel=4e-4)


def test_a_workspace_asked_for_without_the_context_serves_a_causal_call():
    s = make(10, 375, 375, 4, 4, 32, BF16, left=-1, right=0)
    out, lse = call(s)
    n = lib().dwattn_bwd_workspace_bytes(s["q"], s["k"], s["v"], s["table"], s["buckets"])
    ws = Guarded((n,), torch.uint8, DEV, G=4096)
    got = grads(s, out, lse, workspace=ws.t)
    torch.cuda.synchronize()
    ws.check("workspace")
    for a, b in zip(got, grads(s, out, lse)):
        assert torch.equal(a, b)


@DT
def test_key_heads_that_no_query_head_reads_get_zero_gradients(dt):
    k = datagen.normal((2, 40, 2, 32), 1.0, "lone/k", device=DEV).to(dt)
    q = torch.empty((2, 30, 0, 32), dtype=dt, device=DEV)
    table, buckets = torch.empty((16, 0), dtype=dt, device=DEV), lib().rel_buckets(16, 40, device=DEV)
    out, lse = lib().dwattn_fwd(q, k, k, table, buckets)
    dk, dv = (torch.full_like(k, float("nan")) for _ in range(2))
    dq, dk, dv, dt_ = lib().dwattn_bwd(q, k, k, out, lse, out, table, buckets, dk=dk, dv=dv)
    torch.cuda.synchronize()
    assert dq.shape == q.shape and dt_.shape == (16, 0) and not dk.any() and not dv.any()
