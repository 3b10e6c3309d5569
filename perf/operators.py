"""Performance cases of the encoder block's operators: layer norm with the
residual add and dropout in front of it, dropout by itself, and self-attention
with a learned relative position bias by buckets, each forward and backward,
for training batches and for streaming over a cache.

`run` makes the library's calls when `own` is true and otherwise computes the
same outputs in elementary torch operations in 32 bits.

Lengths are spread evenly between half and all of the padded length (a padded
batch of utterances), in an order drawn from the seed.
"""
import math

import numpy as np
import torch

own = False

F32, BF16 = "float32", "bfloat16"


def listed():
    return [
        # One streaming step's norm after a sublayer: 64 streams, chunks of 8 frames; latency counts.
        dict(name="norm_chunk_bf16", op="norm_fwd", dtype=BF16, B=64, T=8, C=256, residual=True, p=0.0, alpha=1.0),
        # Training: the macaron feed-forward's half-step residual with dropout, then the next sublayer's norm.
        dict(name="norm_train_bf16", op="norm_fwd", dtype=BF16, B=16, T=750, C=1024, residual=True, p=0.1, alpha=0.5),
        # Its gradient, with the gradient that flows along the residual.
        dict(name="norm_bwd_bf16", op="norm_bwd", dtype=BF16, B=16, T=750, C=1024, residual=True, p=0.1, alpha=0.5),
        # A small odd model in fp32: 200 channels, a plain norm without a residual.
        dict(name="norm_bwd_odd_f32", op="norm_bwd", dtype=F32, B=7, T=333, C=200, residual=False, p=0.0, alpha=1.0),
        # Dropout inside the feed-forward, after its activation: four times the model's width.
        dict(name="drop_inner_bf16", op="drop_fwd", dtype=BF16, B=16, T=750, C=4096, residual=False, p=0.1, alpha=1.0),
        # The gradient of a residual dropout in fp32.
        dict(name="drop_bwd_f32", op="drop_bwd", dtype=F32, B=32, T=1500, C=512, residual=False, p=0.1, alpha=1.0),
        # A chunk of 8 frames for 64 streams over caches of 512 frames, limited left context.
        dict(name="attn_chunk_bf16", op="attn_fwd", dtype=BF16, B=64, Tq=8, Tk=520, H=4, Hkv=4, D=64, stream=True,
             left=384, right=7, buckets=32, reach=128, lse=False),
        # A single frame for 4 streams over a long cache.
        dict(name="attn_step_bf16", op="attn_fwd", dtype=BF16, B=4, Tq=1, Tk=6000, H=8, Hkv=8, D=64, stream=True,
             left=-1, right=-1, buckets=32, reach=128, lse=False),
        # The training batch of the bf16 conv module: 1024 channels as 8 heads of 128, full context.
        dict(name="attn_train_bf16", op="attn_fwd", dtype=BF16, B=16, Tq=750, Tk=750, H=8, Hkv=8, D=128, stream=False,
             left=-1, right=-1, buckets=32, reach=128, lse=True),
        # The fp32 512-channel encoder, causal.
        dict(name="attn_causal_f32", op="attn_fwd", dtype=F32, B=8, Tq=1500, Tk=1500, H=8, Hkv=8, D=64, stream=False,
             left=-1, right=0, buckets=64, reach=800, lse=True),
        # The bf16 batch's backward pass: the largest case.
        dict(name="attn_bwd_bf16", op="attn_bwd", dtype=BF16, B=16, Tq=750, Tk=750, H=8, Hkv=8, D=128, stream=False,
             left=-1, right=-1, buckets=32, reach=128, lse=True),
        # 200 channels as 4 heads of 50, limited context, shared key heads, odd length, fp32.
        dict(name="attn_bwd_odd_f32", op="attn_bwd", dtype=F32, B=3, Tq=333, Tk=333, H=4, Hkv=2, D=50, stream=False,
             left=100, right=20, buckets=16, reach=64, lse=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "drop_fwd", "drop_bwd", "attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd"])
    dtype = rng.choice([F32, BF16])
    if not op.startswith("attn"):
        C = rng.choice([_log(rng, 8, 4096), 8 * _log(rng, 2, 512), rng.choice([200, 256, 512, 1024, 2048])])
        B, T = _log(rng, 1, 64), _log(rng, 1, 1500)
        while B * T * C > 12_000_000:
            B, T = _log(rng, 1, 64), _log(rng, 1, 1500)
        residual = op.startswith("norm") and rng.random() < 0.6
        p = rng.choice([0.05, 0.1, 0.3]) if op.startswith("drop") or (residual and rng.random() < 0.6) else 0.0
        return dict(op=op, dtype=dtype, B=B, T=T, C=C, residual=residual, p=p, alpha=rng.choice([1.0, 0.5]) if residual else 1.0)
    D = rng.choice([16, 32, 44, 50, 64, 64, 80, 96, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 1, 2, 4])
    buckets, reach = rng.choice([(16, 64), (32, 128), (32, 128), (64, 800)])
    if op == "attn_fwd" and rng.random() < 0.5:
        Tq, Tk, B = rng.choice([1, 1, _log(rng, 2, 40)]), _log(rng, 41, 20000), _log(rng, 1, 64)
        while B * Tk * Hkv * D > 40_000_000:
            Tk, B = _log(rng, 41, 20000), _log(rng, 1, 64)
        left = rng.choice([-1, _log(rng, 16, 4000)])
        return dict(op=op, dtype=dtype, B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, D=D, stream=True, left=left,
                    right=rng.choice([-1, 0, Tq - 1]), buckets=buckets, reach=reach, lse=False)
    B, T = _log(rng, 1, 32), _log(rng, 1, 3000)
    while B * H * T * T * D > (9_000_000_000 if dtype == BF16 else 3_000_000_000) or B * H * T * T > 72_000_000:
        B, T = _log(rng, 1, 32), _log(rng, 1, 3000)
    left, right = rng.choice([(-1, -1), (-1, -1), (-1, 0), (_log(rng, 8, 500), _log(rng, 1, 100))])
    return dict(op=op, dtype=dtype, B=B, Tq=T, Tk=T, H=H, Hkv=Hkv, D=D, stream=False, left=left, right=right,
                buckets=buckets, reach=reach, lse=True)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(B, T):
    """B lengths spread evenly from T down to about half of it (at least one frame)."""
    return np.array([max(1, T - (b * T) // (2 * B)) for b in range(B)], dtype=np.int64)


def _bucket_of(n, count, reach):
    """Bucket of a distance n >= 0 among `count`: the first half hold one distance each, the others grow by equal
    ratios up to `reach`.  In whole numbers: floor(log(n/e)/log(reach/e)*m) >= k where n^m e^k >= reach^k e^m."""
    e = count // 2
    if n < e:
        return n
    m = count - e
    k = 0
    while k + 1 < m and n ** m * e ** (k + 1) >= reach ** (k + 1) * e ** m:
        k += 1
    return e + k


def _bucket_map(buckets, reach):
    """Bucket of each key position relative to the query, -reach .. reach, both directions."""
    half = buckets // 2
    one = [_bucket_of(n, half, reach) for n in range(reach + 1)]
    return [one[n] for n in range(reach, 0, -1)] + [one[0]] + [half + one[n] for n in range(1, reach + 1)]


def _inputs(case, seed):
    """What both `run` and `exact` start from."""
    dev, dt = torch.device("cuda", 0), getattr(torch, case["dtype"])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 32))

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dt)

    s = dict(case=case)
    if not case["op"].startswith("attn"):
        B, T, C = case["B"], case["T"], case["C"]
        s["rng"] = torch.tensor([int(order.randint(0, 1 << 62)), int(order.randint(0, 1 << 40))], dtype=torch.int64, device=dev)
        s["lengths"] = torch.tensor(order.permutation(_lengths(B, T)), dtype=torch.int32, device=dev)
        s["x"] = normal(B, T, C)
        s["residual"] = normal(B, T, C, std=2.0) if case["residual"] else None
        s["gamma"], s["beta"] = normal(C, std=0.1, mean=1.0), normal(C, std=0.1)
        s["dy"] = normal(B, T, C)
        s["dsum"] = normal(B, T, C) if case["residual"] else None
        return s
    B, Tq, Tk, H, Hkv, D = (case[n] for n in ("B", "Tq", "Tk", "H", "Hkv", "D"))
    L = order.permutation(_lengths(B, Tk))
    if case["stream"]:
        L = np.maximum(L, Tq)
        s["q_lengths"] = None
        s["q_pos"] = torch.tensor(L - Tq, dtype=torch.int32, device=dev)
    else:
        s["q_lengths"], s["q_pos"] = torch.tensor(L, dtype=torch.int32, device=dev), None
    s["k_lengths"] = torch.tensor(L, dtype=torch.int32, device=dev)
    s["q"], s["k"], s["v"] = normal(B, Tq, H, D), normal(B, Tk, Hkv, D), normal(B, Tk, Hkv, D)
    s["table"] = normal(case["buckets"], H, std=0.5)
    s["buckets"] = torch.tensor(_bucket_map(case["buckets"], case["reach"]), dtype=torch.int32, device=dev)
    s["dout"] = normal(B, Tq, H, D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "norm_bwd":  # what the forward pass left
        v = _valid(s)
        x = _sum_plain(s)
        mean = x.mean(-1)
        var = (x - mean[..., None]).square().mean(-1)
        s["sum"] = (x * v[..., None]).to(s["x"].dtype)
        s["mean"], s["rstd"] = mean * v, (var + 1e-5).rsqrt() * v
    if case["op"] == "attn_bwd":
        s["out"], s["lse"] = _attn_fwd_plain(s)
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"norm_fwd": _norm_fwd_plain, "norm_bwd": _norm_bwd_plain, "drop_fwd": _drop_fwd_plain,
                "drop_bwd": _drop_bwd_plain, "attn_fwd": _attn_fwd_out_plain, "attn_bwd": _attn_bwd_plain}[op](s)
    import conv_subsampling_amd as dw
    rng = s["rng"] if c.get("p", 0.0) else None
    if op == "norm_fwd":
        y, total, mean, rstd = dw.dwnorm_fwd(s["x"], s["gamma"], s["beta"], s["lengths"], residual=s["residual"], rng=rng,
                                             p=c["p"], alpha=c["alpha"])
        return (y, total, mean, rstd) if c["residual"] else (y, mean, rstd)
    if op == "norm_bwd":
        dx, dres, dgamma, dbeta = dw.dwnorm_bwd(s["sum"], s["gamma"], s["lengths"], s["mean"], s["rstd"], s["dy"],
                                                dsum=s["dsum"], rng=rng, p=c["p"], alpha=c["alpha"],
                                                need=("dx", "dres", "dgamma", "dbeta") if c["residual"] else ("dx", "dgamma", "dbeta"))
        return (dx, dres, dgamma, dbeta) if c["residual"] else (dx, dgamma, dbeta)
    if op == "drop_fwd":
        return dw.dwdrop_fwd(s["x"], s["rng"], c["p"], alpha=c["alpha"])
    if op == "drop_bwd":
        return dw.dwdrop_bwd(s["dy"], s["rng"], c["p"], alpha=c["alpha"])
    kw = dict(q_lengths=s["q_lengths"], k_lengths=s["k_lengths"], q_pos=s["q_pos"], left=c["left"], right=c["right"])
    if op == "attn_fwd":
        out, lse = dw.dwattn_fwd(s["q"], s["k"], s["v"], s["table"], s["buckets"], need=("out", "lse") if c["lse"] else ("out",), **kw)
        return (out, lse) if c["lse"] else out
    return dw.dwattn_bwd(s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], s["table"], s["buckets"], **kw)


def work(case):
    op, e = case["op"], 2 if case["dtype"] == BF16 else 4
    if op.startswith("drop"):
        n = case["B"] * case["T"] * case["C"]
        return {"bytes": 2 * n * e, "flops": 3 * n}
    if op.startswith("norm"):
        rows, C = case["B"] * case["T"], case["C"]
        live = int(_lengths(case["B"], case["T"]).sum())
        reads, writes = (2, 2) if case["residual"] else (1, 1)
        if op == "norm_bwd":
            reads, writes = reads + 1, writes
        extra = 8 * rows + (2 * C * e if op == "norm_fwd" else C * e + 8 * C)
        return {"bytes": (reads * live + writes * rows) * C * e + extra, "flops": (8 if op == "norm_fwd" else 14) * live * C}
    B, Tq, Tk, H, Hkv, D = (case[n] for n in ("B", "Tq", "Tk", "H", "Hkv", "D"))
    L = _lengths(B, Tk)
    if case["stream"]:
        L = np.maximum(L, Tq)
    pairs = keys = 0
    for n in L:
        i = np.arange(Tq) + (n - Tq if case["stream"] else 0)
        i = i if case["stream"] else i[i < n]
        lo = np.maximum(0, i - case["left"]) if case["left"] >= 0 else np.zeros_like(i)
        hi = np.minimum(n - 1, i + case["right"]) if case["right"] >= 0 else np.full_like(i, n - 1)
        pairs += int(np.maximum(0, hi - lo + 1).sum())
        keys += int(hi.max() - lo.min() + 1)
    q = (B * Tq if case["stream"] else int(L.sum())) * H * D * e
    rows = B * Tq * H
    if op == "attn_fwd":
        return {"bytes": q + rows * D * e + 2 * keys * Hkv * D * e + (4 * rows if case["lse"] else 0), "flops": 4 * pairs * H * D}
    return {"bytes": 3 * q + rows * D * e + 2 * (keys + B * Tk) * Hkv * D * e + 4 * rows + 4 * case["buckets"] * H,
            "flops": 10 * pairs * H * D}


# ---------------------------------------------------------------------------
# Plain forms: elementary torch operations in 32 bits, rounded at the end
# ---------------------------------------------------------------------------
def _valid(s):
    T = s["x"].shape[1]
    return (torch.arange(T, device=s["x"].device)[None, :] < s["lengths"][:, None]).float()


def _threshold(p):
    return min(65535, int(math.floor(p * 65536 + 0.5)))


def _keep_plain(shape, rng, p):
    """1/(1-p) where the element stays and 0 where it is dropped: 16 bits of Philox4x32-10 for each element, one
    counter for each 8 elements of a row."""
    C = shape[-1]
    rows, groups = math.prod(shape[:-1]), -(-C // 8)
    low = 0xFFFFFFFF
    n = torch.arange(rows * groups, device=rng.device)
    c0, c1 = n & low, n >> 32
    c2, c3 = (rng[1] & low).expand_as(n), (rng[1] >> 32 & low).expand_as(n)
    k0, k1 = rng[0] & low, rng[0] >> 32 & low
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (b >> 32 & low) ^ c1 ^ k0, b & low, (a >> 32 & low) ^ c3 ^ k1, a & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    bits = torch.stack([h for c in (c0, c1, c2, c3) for h in (c & 0xFFFF, c >> 16)], dim=-1)
    thr = _threshold(p)
    return (bits >= thr).view(rows, groups * 8)[:, :C].reshape(shape).float() * (65536.0 / (65536 - thr))


def _sum_plain(s):
    c = s["case"]
    x = s["x"].float() * c["alpha"]
    if c["p"]:
        x = x * _keep_plain(x.shape, s["rng"], c["p"])
    return x if s["residual"] is None else x + s["residual"].float()


def _norm_fwd_plain(s):
    dt, v = s["x"].dtype, _valid(s)
    x = _sum_plain(s)
    mean = x.mean(-1)
    d = x - mean[..., None]
    rstd = (d.square().mean(-1) + 1e-5).rsqrt()
    y = d * rstd[..., None] * s["gamma"].float() + s["beta"].float()
    y, total, mean, rstd = (y * v[..., None]).to(dt), (x * v[..., None]).to(dt), mean * v, rstd * v
    return (y, mean, rstd) if s["residual"] is None else (y, total, mean, rstd)


def _norm_bwd_plain(s):
    c, dt, v = s["case"], s["x"].dtype, _valid(s)[..., None]
    xh = (s["sum"].float() - s["mean"][..., None]) * s["rstd"][..., None]
    dy = s["dy"].float() * v
    g = dy * s["gamma"].float()
    ds = s["rstd"][..., None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        ds = ds + s["dsum"].float() * v
    dx = ds * c["alpha"]
    if c["p"]:
        dx = dx * _keep_plain(dx.shape, s["rng"], c["p"])
    dgamma, dbeta = (dy * xh).sum((0, 1)), dy.sum((0, 1))
    return (dx.to(dt), dgamma, dbeta) if s["dsum"] is None else (dx.to(dt), ds.to(dt), dgamma, dbeta)


def _drop_fwd_plain(s):
    c, x = s["case"], s["x"]
    return (x.float() * c["alpha"] * _keep_plain(x.shape, s["rng"], c["p"])).to(x.dtype)


def _drop_bwd_plain(s):
    c, dy = s["case"], s["dy"]
    return (dy.float() * c["alpha"] * _keep_plain(dy.shape, s["rng"], c["p"])).to(dy.dtype)


def _heads_first(t, repeat=1):
    t = t.float().permute(0, 2, 1, 3)
    return t.repeat_interleave(repeat, 1) if repeat > 1 else t.contiguous()


def _places(s):
    """Bucket [B,1,Tq,Tk] of each pair, and whether it is allowed."""
    c, dev = s["case"], s["q"].device
    B, Tq, Tk, R = c["B"], c["Tq"], c["Tk"], c["reach"]
    i, j = torch.arange(Tq, device=dev)[None, :, None], torch.arange(Tk, device=dev)[None, None, :]
    rel = j - i - (0 if s["q_pos"] is None else s["q_pos"][:, None, None])
    allowed = j < s["k_lengths"][:, None, None]
    if s["q_lengths"] is not None:
        allowed = allowed & (i < s["q_lengths"][:, None, None])
    if c["left"] >= 0:
        allowed = allowed & (rel >= -c["left"])
    if c["right"] >= 0:
        allowed = allowed & (rel <= c["right"])
    return s["buckets"][rel.clamp(-R, R) + R].long()[:, None], allowed.expand(B, Tq, Tk)[:, None]


def _scores(s):
    """Scores [B,H,Tq,Tk], -inf where not allowed, and the bucket of each pair."""
    c = s["case"]
    bucket, allowed = _places(s)
    S = torch.matmul(_heads_first(s["q"]), _heads_first(s["k"], c["H"] // c["Hkv"]).transpose(-1, -2)) * c["D"] ** -0.5
    S += s["table"].float()[bucket[:, 0]].permute(0, 3, 1, 2)
    return S.masked_fill_(~allowed, -math.inf), bucket


def _attn_fwd_plain(s):
    c = s["case"]
    S, _ = _scores(s)
    m = S.amax(-1, keepdim=True).clamp_min(-1e30)
    P = S.sub_(m).exp_()
    total = P.sum(-1, keepdim=True)
    out = torch.matmul(P, _heads_first(s["v"], c["H"] // c["Hkv"])) / total.clamp_min(1e-30)
    lse = (m + total.log()).squeeze(-1)
    return out.permute(0, 2, 1, 3).contiguous().to(s["q"].dtype), lse


def _attn_fwd_out_plain(s):
    out, lse = _attn_fwd_plain(s)
    return (out, lse) if s["case"]["lse"] else out


def _attn_bwd_plain(s):
    c, dt = s["case"], s["q"].dtype
    G, scale = c["H"] // c["Hkv"], c["D"] ** -0.5
    S, bucket = _scores(s)
    lse = s["lse"][..., None]
    P = (S - torch.where(lse == -math.inf, 0.0, lse)).exp_()
    q, k, v = _heads_first(s["q"]), _heads_first(s["k"], G), _heads_first(s["v"], G)
    do, o = _heads_first(s["dout"]), _heads_first(s["out"])
    dS = (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * P
    back = lambda t: t.permute(0, 2, 1, 3)  # noqa: E731
    shared = lambda t: back(t.unflatten(1, (c["Hkv"], G)).sum(2))  # noqa: E731
    dq = back(torch.matmul(dS, k) * scale)
    dk = shared(torch.matmul(dS.transpose(-1, -2), q) * scale)
    dv = shared(torch.matmul(P.transpose(-1, -2), do))
    place = bucket.expand(c["B"], 1, c["Tq"], c["Tk"])
    dtable = torch.stack([(dS * (place == n)).sum((0, 2, 3)) for n in range(c["buckets"])])
    return dq.contiguous().to(dt), dk.contiguous().to(dt), dv.contiguous().to(dt), dtable


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _factor64(shape, rng, p):
    """The dropout factors, generated on the host."""
    C = shape[-1]
    groups = (C + 7) // 8
    rows = int(np.prod(shape[:-1]))
    seed, stream = (int(v) for v in rng.tolist())
    word = np.uint64(0xFFFFFFFF)
    at = np.arange(rows * groups, dtype=np.uint64)
    x = [at & word, at >> np.uint64(32), np.full_like(at, stream & 0xFFFFFFFF), np.full_like(at, stream >> 32)]
    key = [seed & 0xFFFFFFFF, seed >> 32]
    for r in range(10):
        p0, p1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        ka, kb = np.uint64((key[0] + r * 0x9E3779B9) & 0xFFFFFFFF), np.uint64((key[1] + r * 0xBB67AE85) & 0xFFFFFFFF)
        x = [(p1 >> np.uint64(32)) ^ x[1] ^ ka, p1 & word, (p0 >> np.uint64(32)) ^ x[3] ^ kb, p0 & word]
    halves = np.stack(x, 1).astype("<u4").view("<u2").reshape(rows, groups * 8)[:, :C]
    thr = _threshold(p)
    return torch.from_numpy((halves >= thr) * (65536.0 / (65536 - thr))).view(shape).cuda()


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if not op.startswith("attn"):
        B, T, C = case["B"], case["T"], case["C"]
        f = case["alpha"] * (_factor64((B, T, C), s["rng"], case["p"]) if case["p"] else 1.0)
        if op.startswith("drop"):
            return f * s["x" if op == "drop_fwd" else "dy"].double()
        live = torch.arange(T, device="cuda").view(1, T, 1) < s["lengths"].view(B, 1, 1)
        gamma, beta = s["gamma"].double(), s["beta"].double()
        if op == "norm_fwd":
            x = f * s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
            mean, sq = x.sum(-1, keepdim=True) / C, (x * x).sum(-1, keepdim=True) / C
            rstd = 1 / torch.sqrt(sq - mean * mean + 1e-5)
            y = (x - mean) * rstd * gamma + beta
            got = [torch.where(live, t, 0.0) for t in (y, x, mean, rstd)]
            got = got[:2] + [t[..., 0] for t in got[2:]]
            return tuple(got) if case["residual"] else (got[0], got[2], got[3])
        dy = torch.where(live, s["dy"].double(), 0.0)
        mean, rstd = s["mean"].double()[..., None], s["rstd"].double()[..., None]
        xh = (s["sum"].double() - mean) * rstd
        a, b = (dy * gamma).sum(-1, keepdim=True) / C, (dy * gamma * xh).sum(-1, keepdim=True) / C
        ds = rstd * (dy * gamma - a - xh * b)
        if case["residual"]:
            ds = ds + torch.where(live, s["dsum"].double(), 0.0)
            return f * ds, ds, (dy * xh).sum((0, 1)), dy.sum((0, 1))
        return f * ds, (dy * xh).sum((0, 1)), dy.sum((0, 1))
    B, Tq, Tk, H, Hkv, D = (case[n] for n in ("B", "Tq", "Tk", "H", "Hkv", "D"))
    R, NB, G = case["reach"], case["buckets"], H // Hkv
    where_to = torch.tensor(_bucket_map(NB, R), device="cuda")
    table = s["table"].double()
    out = torch.zeros((B, Tq, H, D), dtype=torch.float64, device="cuda")
    lse = torch.full((B, H, Tq), -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv, dtable = torch.zeros_like(out), s["k"].double() * 0, s["v"].double() * 0, torch.zeros_like(table)
    for b in range(B):  # one item at a time, over its valid frames alone
        nk = int(s["k_lengths"][b])
        nq = Tq if s["q_lengths"] is None else min(Tq, int(s["q_lengths"][b]))
        at = torch.arange(nq, device="cuda") + (0 if s["q_pos"] is None else int(s["q_pos"][b]))
        rel = torch.arange(nk, device="cuda")[None, :] - at[:, None]
        seen = torch.ones_like(rel, dtype=torch.bool)
        if case["left"] >= 0:
            seen &= rel + case["left"] >= 0
        if case["right"] >= 0:
            seen &= rel - case["right"] <= 0
        place = where_to[torch.clamp(rel, -R, R) + R]
        for h in range(H):
            q, k, v = s["q"][b, :nq, h].double(), s["k"][b, :nk, h // G].double(), s["v"][b, :nk, h // G].double()
            S = torch.where(seen, q @ k.T / math.sqrt(D) + table[:, h][place], -math.inf)
            if case["op"] == "attn_fwd":
                ls = torch.logsumexp(S, 1)
                lse[b, h, :nq] = ls
                out[b, :nq, h] = torch.where(ls[:, None] == -math.inf, 0.0, torch.exp(S - torch.clamp(ls, min=-1e300)[:, None])) @ v
                continue
            ls = s["lse"][b, h, :nq].double()
            P = torch.where(seen, torch.exp(S - torch.clamp(ls, min=-1e300)[:, None]), 0.0)
            do, o = s["dout"][b, :nq, h].double(), s["out"][b, :nq, h].double()
            dS = P * (do @ v.T - (do * o).sum(1, keepdim=True))
            dq[b, :nq, h] = dS @ k / math.sqrt(D)
            dk[b, :nk, h // G] += dS.T @ q / math.sqrt(D)
            dv[b, :nk, h // G] += P.T @ do
            dtable[:, h] += torch.zeros(NB, dtype=torch.float64, device="cuda").index_add_(0, place.reshape(-1), dS.reshape(-1))
    if case["op"] == "attn_fwd":
        return (out, lse) if case["lse"] else out
    return dq, dk, dv, dtable
