"""Performance cases of the recurrent block's operators: the gated linear
recurrence over the frames, the norm of the heads of queries and keys with the
rotation by their positions, and the conv module's activations with their
input kept in 8 bits for the backward pass.

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
SCALE = 8.0   # of the recurrence's decay
EPS = 1e-6    # of the heads' norm
GROUP = 32    # columns that share a scale, within each half of a GLU's input


def listed():
    return [
        # One frame for each of 64 streams through the recurrence, the state carried along; latency counts.
        dict(name="scan_step_bf16", op="scan_fwd", dtype=BF16, B=64, T=1, C=1024, state=True),
        # The bf16 training batch of the conv module, 1024 channels.
        dict(name="scan_train_bf16", op="scan_fwd", dtype=BF16, B=16, T=750, C=1024, state=False),
        # Two hour-long recordings after 8-fold subsampling, in fp32: few sequences, so that the frames have to be shared out.
        dict(name="scan_long_f32", op="scan_fwd", dtype=F32, B=2, T=6001, C=512, state=True),
        # The training batch's gradients.
        dict(name="scan_bwd_bf16", op="scan_bwd", dtype=BF16, B=16, T=750, C=1024, state=False),
        # 200 channels, odd lengths, fp32, with the gradient of the state at both ends.
        dict(name="scan_bwd_odd_f32", op="scan_bwd", dtype=F32, B=3, T=1333, C=200, state=True),
        # One frame for each of 64 streams: queries rotated, keys and values into caches of 512 frames.
        dict(name="rope_step_bf16", op="rope_fwd", dtype=BF16, B=64, T=1, H=8, Hkv=2, D=64, R=64, pairs="halves", cache=512),
        # The training batch as 8 heads of 128.
        dict(name="rope_train_bf16", op="rope_fwd", dtype=BF16, B=16, T=750, H=8, Hkv=8, D=128, R=128, pairs="halves", cache=0),
        # Its gradients.
        dict(name="rope_bwd_bf16", op="rope_bwd", dtype=BF16, B=16, T=750, H=8, Hkv=8, D=128, R=128, pairs="halves", cache=0),
        # 4 heads of 50 over 2 key heads, a rotation of neighbours over 32 of the 50, odd length, fp32.
        dict(name="rope_bwd_odd_f32", op="rope_bwd", dtype=F32, B=3, T=333, H=4, Hkv=2, D=50, R=32, pairs="neighbours", cache=0),
        # The conv module's GLU in training, forward and backward through the 8-bit checkpoint.
        dict(name="act_glu_bf16", op="act_pass", dtype=BF16, B=16, T=750, C=1024, kind="glu"),
        # SiLU of a small odd model in fp32, forward and backward.
        dict(name="act_silu_odd_f32", op="act_pass", dtype=F32, B=7, T=333, C=200, kind="silu"),
        # The backward pass of the SiLU inside the feed-forward, four times the model's width; the activation itself is computed
        # again for the weights' gradient of the projection behind it.
        dict(name="act_bwd_bf16", op="act_bwd", dtype=BF16, B=16, T=750, C=4096, kind="silu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["scan_fwd", "scan_fwd", "scan_bwd", "scan_bwd", "rope_fwd", "rope_bwd", "act_pass", "act_bwd"])
    dtype = rng.choice([F32, BF16])
    wide = 1 if dtype == BF16 else 2
    if op.startswith("scan"):
        size = lambda: (_log(rng, 1, 64), rng.choice([1, _log(rng, 2, 40), _log(rng, 41, 20000), _log(rng, 41, 20000)]),  # noqa: E731
                        rng.choice([_log(rng, 8, 4096), 8 * _log(rng, 2, 512), rng.choice([200, 256, 512, 1024])]))
        B, T, C = size()
        while B * T * C * wide > 12_000_000:
            B, T, C = size()
        return dict(op=op, dtype=dtype, B=B, T=T, C=C, state=T == 1 or rng.random() < 0.5)
    if op.startswith("act"):
        size = lambda: (_log(rng, 1, 64), _log(rng, 1, 1500), rng.choice([_log(rng, 8, 4096), 8 * _log(rng, 2, 512)]))  # noqa: E731
        kind = rng.choice(["silu", "glu"])
        B, T, C = size()
        while B * T * C * wide * (1 if kind == "silu" else 2) > 24_000_000:
            B, T, C = size()
        return dict(op=op, dtype=dtype, B=B, T=T, C=C, kind=kind)
    D = rng.choice([16, 32, 44, 50, 64, 64, 80, 96, 128, 128])
    R = D if rng.random() < 0.6 else 2 * rng.randint(1, D // 2)
    Hkv = rng.choice([1, 2, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 4])
    pairs = rng.choice(["halves", "halves", "neighbours"])
    if op == "rope_fwd" and rng.random() < 0.5:
        size = lambda: (_log(rng, 1, 64), rng.choice([1, _log(rng, 2, 40)]), _log(rng, 41, 4000))  # noqa: E731
        B, T, cache = size()
        while B * cache * Hkv * D > 8_000_000:
            B, T, cache = size()
        return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hkv=Hkv, D=D, R=R, pairs=pairs, cache=cache)
    B, T = _log(rng, 1, 64), _log(rng, 1, 1500)
    while B * T * (H + Hkv) * D * wide > 24_000_000:
        B, T = _log(rng, 1, 64), _log(rng, 1, 1500)
    return dict(op=op, dtype=dtype, B=B, T=T, H=H, Hkv=Hkv, D=D, R=R, pairs=pairs, cache=0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _lengths(B, T):
    """B lengths spread evenly from T down to about half of it (at least one frame)."""
    return np.array([max(1, T - (b * T) // (2 * B)) for b in range(B)], dtype=np.int64)


def _inputs(case, seed):
    """What both `run` and `exact` start from."""
    dev, dt = torch.device("cuda", 0), getattr(torch, case["dtype"])
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    order = np.random.RandomState(seed % (1 << 32))

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dt)

    s = dict(case=case)
    B, T = case["B"], case["T"]
    s["lengths"] = torch.tensor(order.permutation(_lengths(B, T)), dtype=torch.int32, device=dev)
    if case["op"].startswith("scan"):
        C = case["C"]
        s["x"], s["r"], s["g"], s["dy"] = (normal(B, T, C) for _ in range(4))
        # decays of 0.999 to 0.67 a frame where the gate is half open
        rate = torch.exp(torch.empty(C, device=dev).uniform_(math.log(2.5e-4), math.log(0.1), generator=g))
        s["decay"] = torch.log(torch.expm1(rate.double())).float()
        s["h0"] = torch.randn((B, C), generator=g, device=dev) if case["state"] else None
        s["dh_last"] = torch.randn((B, C), generator=g, device=dev) if case["state"] else None
        return s
    if case["op"].startswith("act"):
        C = case["C"]
        s["x"], s["dy"] = normal(B, T, C * (2 if case["kind"] == "glu" else 1), std=1.5), normal(B, T, C)
        return s
    H, Hkv, D, R = (case[n] for n in ("H", "Hkv", "D", "R"))
    # q, k and v as slices of one projection's output
    qkv = normal(B, T, H + 2 * Hkv, D, std=2.0)
    s["q"], s["k"], s["v"] = qkv.split([H, Hkv, Hkv], 2)
    s["q_gamma"], s["k_gamma"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1, mean=1.0)
    s["freq"] = torch.tensor([1e4 ** (-2.0 * j / R) for j in range(R // 2)], dtype=torch.float64, device=dev)
    s["dq"], s["dk"] = normal(B, T, H, D), normal(B, T, Hkv, D)
    s["pos"] = s["place"] = None
    if case["cache"]:  # streams of different ages; the cache of some has been cut from the front
        S = case["cache"]
        place = order.randint(0, max(1, S - T + 1), size=B)
        gone = order.choice([0, 0, 1000, 1_000_000], size=B)
        s["place"] = torch.tensor(place, dtype=torch.int32, device=dev)
        s["pos"] = torch.tensor(place + gone, dtype=torch.int32, device=dev)
        s["lengths"] = None
        s["k_cache"], s["v_cache"] = normal(B, S, Hkv, D), normal(B, S, Hkv, D)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "scan_bwd":  # what the forward pass left
        s["y"] = _scan_fwd_plain(s)[0]
    if case["op"] == "act_bwd":
        s["kept"] = _pack_plain(s["x"], case["kind"], s["lengths"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------
def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"scan_fwd": _scan_fwd_plain, "scan_bwd": _scan_bwd_plain, "rope_fwd": _rope_fwd_plain,
                "rope_bwd": _rope_bwd_plain, "act_pass": _act_pass_plain, "act_bwd": _act_bwd_plain}[op](s)
    import conv_subsampling_amd as dw
    if op == "scan_fwd":
        return dw.dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=s["h0"], scale=SCALE)
    if op == "scan_bwd":
        need = ("dx", "dr", "dg", "ddecay", "dh0") if c["state"] else ("dx", "dr", "dg", "ddecay")
        got = dw.dwscan_bwd(s["x"], s["r"], s["g"], s["decay"], s["y"], s["dy"], s["lengths"], h0=s["h0"],
                            dh_last=s["dh_last"], scale=SCALE, need=need)
        return got[:len(need)]
    if op == "act_pass":
        y, kept = dw.dwact_fwd(s["x"], c["kind"], s["lengths"])
        dx, _ = dw.dwact_bwd(kept, s["dy"], c["kind"], s["lengths"])
        return y, dx
    if op == "act_bwd":
        return dw.dwact_bwd(s["kept"], s["dy"], c["kind"], s["lengths"], need=("dx", "y"))
    kw = dict(pos=s["pos"], pairs=c["pairs"], eps=EPS)
    if op == "rope_bwd":
        return dw.dwrope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["q_gamma"], s["k_gamma"], s["freq"], s["lengths"], **kw)
    if c["cache"]:
        return dw.dwrope_fwd(s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["freq"], v=s["v"], k_out=s["k_cache"],
                             v_out=s["v_cache"], place=s["place"], **kw)
    return dw.dwrope_fwd(s["q"], s["k"], s["q_gamma"], s["k_gamma"], s["freq"], s["lengths"], **kw)[:2]


def work(case):
    op, e = case["op"], 2 if case["dtype"] == BF16 else 4
    B, T = case["B"], case["T"]
    rows, live = B * T, int(_lengths(B, T).sum())
    if op.startswith("scan"):
        C = case["C"]
        states = (2 if case["state"] else 1) * B * C * 4
        if op == "scan_fwd":
            return {"bytes": (3 * live + rows) * C * e + states + 4 * C, "flops": 20 * live * C}
        return {"bytes": (5 * live + 3 * rows) * C * e + (3 * B * C * 4 if case["state"] else 0) + 8 * C, "flops": 45 * live * C}
    if op.startswith("act"):
        C, wide = case["C"], 2 if case["kind"] == "glu" else 1
        kept = rows * wide * (C + -(-C // GROUP))
        fwd, bwd = live * wide * C * e + rows * C * e + kept, kept * live // rows + live * C * e + rows * wide * C * e
        if op == "act_pass":
            return {"bytes": fwd + bwd, "flops": 25 * live * C}
        return {"bytes": bwd + rows * C * e, "flops": 15 * live * C}
    H, Hkv, D, R = (case[n] for n in ("H", "Hkv", "D", "R"))
    if op == "rope_bwd":
        return {"bytes": (2 * live + rows) * (H + Hkv) * D * e + 2 * D * (e + 4) + 4 * R, "flops": 16 * live * (H + Hkv) * D}
    if case["cache"]:
        return {"bytes": 2 * rows * (H + 2 * Hkv) * D * e + 2 * D * e + 4 * R + 8 * B, "flops": 8 * rows * (H + Hkv) * D}
    return {"bytes": (live + rows) * (H + Hkv) * D * e + 2 * D * e + 4 * R, "flops": 8 * live * (H + Hkv) * D}


# ---------------------------------------------------------------------------
# Plain forms: elementary torch operations in 32 bits, rounded at the end
# ---------------------------------------------------------------------------
def _valid(s, T):
    if s["lengths"] is None:
        return None
    return (torch.arange(T, device=s["lengths"].device)[None, :] < s["lengths"][:, None])[..., None]


def _gates(s):
    """softplus(decay), the two gates, -log(a) and sqrt(1 - a^2), with a = 1 and an input of 0 past the lengths."""
    live = _valid(s, s["x"].shape[1])
    rate = torch.log1p(torch.exp(s["decay"]))
    si, ii = 1 / (1 + torch.exp(-s["r"].float())), 1 / (1 + torch.exp(-s["g"].float()))
    w = torch.where(live, SCALE * rate * si, 0.0)
    return rate, si, ii, w, torch.sqrt(-torch.expm1(-2 * w)), live


def _scan_plain(w, u, start):
    """h_t = exp(-w_t) h_{t-1} + u_t over axis 1 by doubling steps."""
    h, total = u.clone(), w.clone()
    if start is not None:
        h[:, 0] += torch.exp(-w[:, 0]) * start
    step = 1
    while step < h.shape[1]:
        add = torch.exp(-total[:, step:]) * h[:, :-step]
        h[:, step:] += add
        total[:, step:] += total[:, :-step].clone()
        step *= 2
    return h


def _scan_fwd_plain(s):
    _, _, i, w, m, live = _gates(s)
    h = _scan_plain(w, torch.where(live, m * i * s["x"].float(), 0.0), s["h0"])
    return torch.where(live, h, 0.0).to(s["x"].dtype), h[:, -1].contiguous()


def _scan_bwd_plain(s):
    dt = s["x"].dtype
    rate, si, i, w, m, live = _gates(s)
    x, y = torch.where(live, s["x"].float(), 0.0), s["y"].float()
    h0 = torch.zeros_like(y[:, 0]) if s["h0"] is None else s["h0"]
    before = torch.cat([h0[:, None], y[:, :-1]], 1)
    # backwards in time: G_t = dy_t + a_{t+1} G_{t+1}, the last frame's gradient in front of it
    after = torch.cat([w[:, 1:], torch.zeros_like(w[:, :1])], 1)
    G = _scan_plain(after.flip(1), torch.where(live, s["dy"].float(), 0.0).flip(1), s["dh_last"]).flip(1)
    a = torch.exp(-w)
    ratio = torch.where(m > 0, w / m, 0.0)
    q = torch.where(live, G * (i * x * a * a * ratio - w * a * before), 0.0)
    dx, dg, dr = G * m * i, G * m * x * i * (1 - i), q * (1 - si)
    ddecay = q.sum((0, 1)) * (1 / (1 + torch.exp(-s["decay"]))) / rate
    out = tuple(torch.where(live, t, 0.0).to(dt) for t in (dx, dr, dg)) + (ddecay,)
    return out + ((a[:, 0] * G[:, 0]).contiguous(),) if s["case"]["state"] else out


def _angles(s, T):
    """cos and sin [B or 1,T,1,R/2] of the angles in 64 bits, rounded."""
    t = torch.arange(T, device=s["q"].device)
    at = t[None] if s["pos"] is None else s["pos"].long()[:, None] + t
    ang = at.double()[:, :, None, None] * s["freq"]
    return torch.cos(ang).float(), torch.sin(ang).float()


def _split(x, c):
    """The two elements of each pair, and those that are not rotated."""
    R = c["R"]
    if c["pairs"] == "halves":
        return x[..., :R // 2], x[..., R // 2:R], x[..., R:]
    return x[..., 0:R:2], x[..., 1:R:2], x[..., R:]


def _merge(a, b, rest, c):
    return torch.cat([torch.cat([a, b], -1) if c["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2), rest], -1)


def _rotate(x, cos, sin, c):
    a, b, rest = _split(x, c)
    return _merge(a * cos - b * sin, b * cos + a * sin, rest, c)


def _rope_fwd_plain(s):
    c, dt, T = s["case"], s["q"].dtype, s["q"].shape[1]
    cos, sin = _angles(s, T)
    live = _valid(s, T)

    def one(x, gamma):
        x = x.float()
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()
        out = _rotate(n, cos, sin, c)
        return (out if live is None else torch.where(live[..., None], out, 0.0)).to(dt)

    q, k = one(s["q"], s["q_gamma"]), one(s["k"], s["k_gamma"])
    if not c["cache"]:
        return q, k
    at = s["place"].long()[:, None] + torch.arange(T, device=q.device)
    item = torch.arange(q.shape[0], device=q.device)[:, None].expand_as(at)
    fits = at < c["cache"]
    s["k_cache"][item[fits], at[fits]] = k[fits]
    s["v_cache"][item[fits], at[fits]] = s["v"][fits]
    return q, s["k_cache"], s["v_cache"]


def _rope_bwd_plain(s):
    c, dt, T = s["case"], s["q"].dtype, s["q"].shape[1]
    cos, sin = _angles(s, T)
    live = _valid(s, T)[..., None]

    def one(x, gamma, dout):
        x, d = x.float(), torch.where(live, _rotate(dout.float(), cos, -sin, c), 0.0)
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh, g = x * rstd, d * gamma.float()
        dx = rstd * (g - xh * (g * xh).mean(-1, keepdim=True))
        return dx.to(dt), (d * xh).sum((0, 1, 2))

    (dq, dgq), (dk, dgk) = one(s["q"], s["q_gamma"], s["dq"]), one(s["k"], s["k_gamma"], s["dk"])
    return dq, dk, dgq, dgk


def _pack_plain(x, kind, lengths):
    """8-bit values [B,T,W] and codes [B,T,parts*ceil(C/32)] of their scales, for each of the input's parts of C columns: scale
    2^(code-127), the smallest with which the group's largest is at most 127; what lies past the lengths is zero, as is its code."""
    B, T, W = x.shape
    parts = 2 if kind == "glu" else 1
    C = W // parts
    n = -(-C // GROUP)
    xg = torch.nn.functional.pad(x.float().view(B, T, parts, C), (0, n * GROUP - C)).view(B, T, parts * n, GROUP)
    top = xg.abs().amax(-1).contiguous()
    code = ((top.view(torch.int32) + 0x1FFFF >> 23) - 6).clamp_min(1)
    q = torch.round(xg * torch.exp2((127 - code).float())[..., None])
    live = torch.arange(T, device=x.device)[None, :] < lengths[:, None]
    q = torch.where(live[..., None, None], q, 0.0).view(B, T, parts, n * GROUP)[..., :C].reshape(B, T, W)
    return q.to(torch.int8), torch.where(live[..., None], code, 0).to(torch.uint8)


def _unpack_plain(kept, kind):
    q, code = kept
    parts = 2 if kind == "glu" else 1
    C = q.shape[-1] // parts
    scale = torch.exp2(code.float() - 127).unflatten(-1, (parts, -1)).repeat_interleave(GROUP, -1)[..., :C]
    return q.float() * scale.flatten(-2)


def _act_plain(x, kind):
    if kind == "silu":
        return x / (1 + torch.exp(-x))
    a, b = x.chunk(2, -1)
    return a / (1 + torch.exp(-b))


def _act_grad_plain(x, dy, kind):
    if kind == "silu":
        g = 1 / (1 + torch.exp(-x))
        return dy * (g * (1 + x * (1 - g)))
    a, b = x.chunk(2, -1)
    g = 1 / (1 + torch.exp(-b))
    return torch.cat([dy * g, dy * a * (g * (1 - g))], -1)


def _act_pass_plain(s):
    kind, dt = s["case"]["kind"], s["x"].dtype
    live = _valid(s, s["x"].shape[1])
    y = torch.where(live, _act_plain(s["x"].float(), kind), 0.0).to(dt)
    kept = _unpack_plain(_pack_plain(s["x"], kind, s["lengths"]), kind)
    return y, torch.where(live, _act_grad_plain(kept, s["dy"].float(), kind), 0.0).to(dt)


def _act_bwd_plain(s):
    kind, dt = s["case"]["kind"], s["x"].dtype
    live = _valid(s, s["x"].shape[1])
    kept = _unpack_plain(s["kept"], kind)
    dx = torch.where(live, _act_grad_plain(kept, s["dy"].float(), kind), 0.0).to(dt)
    return dx, torch.where(live, _act_plain(kept, kind), 0.0).to(dt)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    return (_exact_scan if op.startswith("scan") else _exact_act if op.startswith("act") else _exact_rope)(s)


def _exact_scan(s):
    """Frame by frame, as the recurrence is written."""
    op, T = s["case"]["op"], s["x"].shape[1]
    lam = torch.nn.functional.softplus(s["decay"].double(), threshold=60.0)
    L = s["lengths"][:, None]
    h = torch.zeros_like(s["x"][:, 0], dtype=torch.float64) if s["h0"] is None else s["h0"].double()

    def frame(t):
        x, si, i = s["x"][:, t].double(), torch.sigmoid(s["r"][:, t].double()), torch.sigmoid(s["g"][:, t].double())
        w = SCALE * lam * si
        return x, si, i, w, torch.exp(-w), torch.sqrt(-torch.expm1(-2 * w))

    if op == "scan_fwd":
        y = torch.zeros_like(s["x"], dtype=torch.float64)
        for t in range(T):
            x, _, i, _, a, m = frame(t)
            h = torch.where(t < L, a * h + m * i * x, h)
            y[:, t] = torch.where(t < L, h, 0.0)
        return y, h
    dx, dr, dg = (torch.zeros_like(s["x"], dtype=torch.float64) for _ in range(3))
    ddecay = torch.zeros_like(lam)
    G = torch.zeros_like(h) if s["dh_last"] is None else s["dh_last"].double()   # the gradient of h_t from the frames after it
    slope = SCALE * torch.sigmoid(s["decay"].double())
    for t in range(T - 1, -1, -1):
        x, si, i, w, a, m = frame(t)
        live = t < L
        full = G + s["dy"][:, t].double()
        prev = s["y"][:, t - 1].double() if t else h
        dm, da = full * i * x, full * prev
        dw = -a * da + dm * a * a / m
        dx[:, t], dg[:, t] = torch.where(live, full * m * i, 0.0), torch.where(live, full * m * x * i * (1 - i), 0.0)
        dr[:, t] = torch.where(live, dw * SCALE * lam * si * (1 - si), 0.0)
        ddecay += torch.where(live, dw * si, 0.0).sum(0) * slope
        G = torch.where(live, a * full, G)
    return (dx, dr, dg, ddecay, G) if s["case"]["state"] else (dx, dr, dg, ddecay)


def _exact_act(s):
    c = s["case"]
    B, T, W = s["x"].shape
    x = s["x"].double()
    live = (torch.arange(T, device=x.device) < s["lengths"][:, None]).unsqueeze(-1)
    C = c["C"]
    if c["op"] == "act_pass":
        scale = torch.ones((B, T, W), dtype=torch.float64, device=x.device)
        for j in [k for half in range(0, W, C) for k in range(half, half + C, GROUP)]:
            part = slice(j, min(j + GROUP, C if j < C else W))
            top = x[..., part].abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(top / 127))
            e = torch.where(top > 127 * torch.exp2(e), e + 1, torch.where(top <= 127 * torch.exp2(e - 1), e - 1, e))
            scale[..., part] = torch.exp2(e.clamp_min(-126))
        kept = torch.round(x / scale) * scale
    else:
        q, code = s["kept"]
        column = torch.arange(W, device=x.device)
        kept = q.double() * torch.exp2(code.double() - 127)[..., column // C * -(-C // GROUP) + column % C // GROUP]
    dy = s["dy"].double()

    def act(z):
        if c["kind"] == "silu":
            return z * torch.sigmoid(z)
        return z[..., :W // 2] * torch.sigmoid(z[..., W // 2:])

    if c["kind"] == "silu":
        g = torch.sigmoid(kept)
        dx = dy * (g + kept * g * torch.sigmoid(-kept))
    else:
        a, b = kept[..., :W // 2], kept[..., W // 2:]
        dx = torch.cat([dy * torch.sigmoid(b), dy * a * torch.sigmoid(b) * torch.sigmoid(-b)], -1)
    dx = torch.where(live, dx, 0.0)
    if c["op"] == "act_pass":
        return torch.where(live, act(x), 0.0), dx
    return dx, torch.where(live, act(kept), 0.0)


def _exact_rope(s):
    """Head by head, each pair as a complex number turned by its angle."""
    c = s["case"]
    B, T = c["B"], c["T"]
    R, D = c["R"], c["D"]
    first = torch.arange(R // 2, device="cuda") * (1 if c["pairs"] == "halves" else 2)
    second = first + (R // 2 if c["pairs"] == "halves" else 1)
    at = torch.arange(T, device="cuda").expand(B, T) + (0 if s["pos"] is None else s["pos"][:, None].long())
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), at[..., None].double() * s["freq"])
    live = None if s["lengths"] is None else (torch.arange(T, device="cuda") < s["lengths"][:, None])[..., None]

    def turned(z, by):
        out = z.clone()
        p = torch.complex(z[..., first], z[..., second]) * by
        out[..., first], out[..., second] = p.real, p.imag
        return out

    def forward(x, gamma):
        out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
        for h in range(x.shape[2]):
            z = x[:, :, h].double()
            z = z / torch.sqrt((z * z).sum(-1, keepdim=True) / D + EPS) * gamma.double()
            z = turned(z, turn)
            out[:, :, h] = z if live is None else torch.where(live, z, 0.0)
        return out

    def backward(x, gamma, dout):
        dx, dgamma = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
        for h in range(x.shape[2]):
            z, d = x[:, :, h].double(), torch.where(live, turned(dout[:, :, h].double(), turn.conj()), 0.0)
            norm = torch.sqrt((z * z).sum(-1, keepdim=True) / D + EPS)
            dgamma += (d * z / norm).sum((0, 1))
            g = d * gamma.double()
            dx[:, :, h] = g / norm - z * (g * z).sum(-1, keepdim=True) / (D * norm ** 3)
        return dx, dgamma

    if c["op"] == "rope_bwd":
        dq, dgq = backward(s["q"], s["q_gamma"], s["dq"])
        dk, dgk = backward(s["k"], s["k_gamma"], s["dk"])
        return dq, dk, dgq, dgk
    q, k = forward(s["q"], s["q_gamma"]), forward(s["k"], s["k_gamma"])
    if not c["cache"]:
        return q, k
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for b in range(B):
        p = int(s["place"][b])
        n = min(T, c["cache"] - p)
        kc[b, p:p + n], vc[b, p:p + n] = k[b, :n], s["v"][b, :n].double()
    return q, kc, vc
