"""The recurrence, the rotated heads and the kept activations in 64 bits, as
plainly as they are defined: NumPy on the host, sharing nothing with the
library.  Beside the values stand the sums of absolute terms that the tests'
tolerances count roundings in."""
import numpy as np

from block_ref import U16, U32  # noqa: F401


def sigmoid(v):
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def softplus(v):
    return np.where(v > 30, v, np.log1p(np.exp(np.minimum(v, 30))))


def clip(lengths, B, T):
    return np.full(B, T) if lengths is None else np.clip(np.asarray(lengths, dtype=np.int64), 0, T)


def gates(r, g, decay, scale):
    s, i = sigmoid(r), sigmoid(g)
    w = scale * softplus(decay) * s
    return s, i, w, np.exp(-w), np.sqrt(-np.expm1(-2 * w))


# The state moves by the float nearest to 1 - a, so a step loses up to 2 roundings of the state before it however small a is.  The
# sums of absolute terms, of which at least 80 roundings are allowed, keep a 32nd of it.
KEPT = 1 / 32


def scan_fwd(x, r, g, decay, lengths=None, h0=None, scale=8.0):
    """(y, h_last), then for both the sum of absolute terms and that sum weighted by each term's -log of its decay."""
    B, T, C = x.shape
    L = clip(lengths, B, T)[:, None]
    h = np.zeros((B, C)) if h0 is None else h0.astype(np.float64)
    size, bent = np.abs(h), np.zeros((B, C))
    y, ysize, ybent = (np.zeros((B, T, C)) for _ in range(3))
    for t in range(T):
        live = t < L
        _, i, w, a, m = gates(r[:, t], g[:, t], decay, scale)
        with np.errstate(invalid="ignore"):
            u = m * i * x[:, t]
            h = np.where(live, a * h + u, h)
            bent = np.where(live, a * (bent + w * size), bent)
            size = np.where(live, np.maximum(a, KEPT) * size + np.abs(u), size)
        for into, value in ((y, h), (ysize, size), (ybent, bent)):
            into[:, t] = np.where(live, value, 0.0)
    return y, h, ysize, size, ybent, bent


def scan_bwd(x, r, g, decay, y, dy, lengths=None, h0=None, dh_last=None, scale=8.0):
    """dict of the gradients and, under name + "_size" and "_bent", of what their errors are counted in."""
    B, T, C = x.shape
    L = clip(lengths, B, T)[:, None]
    G = np.zeros((B, C)) if dh_last is None else dh_last.astype(np.float64)
    size, bent = np.abs(G), np.zeros((B, C))
    h0 = np.zeros((B, C)) if h0 is None else h0
    o = {n + k: np.zeros((B, T, C)) for n in ("dx", "dr", "dg") for k in ("", "_size", "_bent")}
    o |= {"ddecay" + k: np.zeros(C) for k in ("", "_size", "_bent")}
    slope = np.where(decay < -30, 1.0, sigmoid(decay) / np.maximum(softplus(decay), 1e-300))
    for t in range(T - 1, -1, -1):
        live = t < L
        with np.errstate(invalid="ignore", divide="ignore"):
            s, i, w, a, m = gates(r[:, t], g[:, t], decay, scale)
            ratio = np.where(m > 0, w / m, 0.0)
            prev = y[:, t - 1] if t else h0
            full, fsize = G + dy[:, t], size + np.abs(dy[:, t])
            ix = i * x[:, t]
            q, qa = full * (ix * a * a * ratio - w * a * prev), np.abs(ix) * ratio + w * np.abs(prev)
            for n, v, c in (("dx", full * m * i, m * i), ("dg", full * m * ix * (1 - i), m * np.abs(ix)), ("dr", q * (1 - s), qa)):
                o[n][:, t] = np.where(live, v, 0.0)
                o[n + "_size"][:, t] = np.where(live, c * fsize, 0.0)
                o[n + "_bent"][:, t] = np.where(live, c * bent, 0.0)
            o["ddecay"] += np.where(live, q, 0.0).sum(0) * slope
            o["ddecay_size"] += np.where(live, qa * fsize, 0.0).sum(0) * slope
            o["ddecay_bent"] += np.where(live, qa * bent, 0.0).sum(0) * slope
            G = np.where(live, a * full, G)
            bent = np.where(live, a * (bent + w * fsize), bent)
            size = np.where(live, np.maximum(a, KEPT) * fsize, size)
    o["dh0"], o["dh0_size"], o["dh0_bent"] = G, size, bent
    return o


def pairs_of(R, D, kind):
    first = np.arange(R // 2) * (1 if kind == "halves" else 2)
    return first, first + (R // 2 if kind == "halves" else 1)


def rope_fwd(x, gamma, freq, lengths, pos, kind, eps):
    """One tensor [B,T,H,D]: (out, sum of the absolute terms of each element)."""
    B, T, H, D = x.shape
    gamma = np.ones(D) if gamma is None else gamma
    freq = np.zeros(0) if freq is None else freq
    out, size = np.zeros(x.shape), np.zeros(x.shape)
    L = clip(lengths, B, T)
    i, j = pairs_of(2 * len(freq), D, kind)
    for b in range(B):
        n = L[b]
        z = x[b, :n]
        with np.errstate(invalid="ignore", divide="ignore"):
            z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps) * gamma
        f = ((0 if pos is None else int(pos[b])) + np.arange(n))[:, None, None] * freq
        o, s = z.copy(), np.abs(z)
        o[..., i], o[..., j] = z[..., i] * np.cos(f) - z[..., j] * np.sin(f), z[..., j] * np.cos(f) + z[..., i] * np.sin(f)
        s[..., i] = s[..., j] = np.abs(z[..., i]) + np.abs(z[..., j])
        out[b, :n], size[b, :n] = o, s
    return out, size


def rope_bwd(x, gamma, freq, lengths, pos, kind, eps, dout):
    """One tensor: (dx, its sums of absolute terms, dgamma, its)."""
    B, T, H, D = x.shape
    gamma = np.ones(D) if gamma is None else gamma
    freq = np.zeros(0) if freq is None else freq
    dx, dsize, dg, gsize = np.zeros(x.shape), np.zeros(x.shape), np.zeros(D), np.zeros(D)
    L = clip(lengths, B, T)
    i, j = pairs_of(2 * len(freq), D, kind)
    for b in range(B):
        n = L[b]
        z, d = x[b, :n], dout[b, :n]
        f = ((0 if pos is None else int(pos[b])) + np.arange(n))[:, None, None] * freq
        u, s = d.copy(), np.abs(d)
        u[..., i], u[..., j] = d[..., i] * np.cos(f) + d[..., j] * np.sin(f), d[..., j] * np.cos(f) - d[..., i] * np.sin(f)
        s[..., i] = s[..., j] = np.abs(d[..., i]) + np.abs(d[..., j])
        rstd = 1 / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
        xh, e, es = z * rstd, u * gamma, s * np.abs(gamma)
        dx[b, :n] = rstd * (e - xh * (e * xh).mean(-1, keepdims=True))
        dsize[b, :n] = rstd * (es + np.abs(xh) * (es * np.abs(xh)).mean(-1, keepdims=True))
        dg += (u * xh).sum((0, 1))
        gsize += (s * np.abs(xh)).sum((0, 1))
    return dx, dsize, dg, gsize


def pack(x, parts):
    """(kept int8, codes uint8) of x [rows, parts * C]: one group at a time, in whole powers of two."""
    rows, W = x.shape
    C = W // parts
    n = -(-C // 32)
    kept, codes = np.zeros((rows, W), np.int8), np.zeros((rows, parts * n), np.uint8)
    for p in range(parts):
        for k in range(n):
            at = slice(p * C + 32 * k, p * C + min(C, 32 * (k + 1)))
            part = x[:, at]
            bad = ~np.isfinite(part).all(1)
            top = np.where(bad, 0.0, np.abs(np.where(np.isfinite(part), part, 0.0)).max(1))
            e = np.full(rows, -126)
            with np.errstate(divide="ignore"):
                guess = np.where(top > 0, np.floor(np.log2(np.where(top > 0, top, 1.0))) - 8, -200).astype(int)
            for step in range(4):  # the smallest of guess .. guess + 3 that holds the largest
                e = np.where((top > 127 * np.exp2(guess + step - 1.0)) & (guess + step > e), guess + step, e)
            e = np.minimum(e, 121)  # 128 times the next scale would be no finite float32
            codes[:, p * n + k] = np.where(bad, 255, e + 127)
            kept[:, at] = np.clip(np.rint(np.where(bad[:, None], 0.0, part) * np.exp2(-e.astype(np.float64))[:, None]), -127, 127)
    return kept, codes


def unpack(kept, codes, parts):
    rows, W = kept.shape
    C, n = W // parts, codes.shape[1] // parts
    column = np.arange(W)
    code = codes[:, column // C * n + column % C // 32].astype(np.float64)
    return np.where(code == 255, np.nan, kept * np.exp2(code - 127))


def act(x, kind):
    if kind == "none":
        return x.copy()
    if kind == "silu":
        return x * sigmoid(x)
    C = x.shape[-1] // 2
    return x[..., :C] * sigmoid(x[..., C:])


def act_grad(x, dy, kind):
    """(dx, its sums of absolute terms)."""
    if kind == "none":
        return dy.copy(), np.abs(dy)
    if kind == "silu":
        s = sigmoid(x)
        return dy * (s + x * s * sigmoid(-x)), np.abs(dy) * (s + np.abs(x) * s)
    C = x.shape[-1] // 2
    a, s = x[..., :C], sigmoid(x[..., C:])
    return (np.concatenate([dy * s, dy * a * s * sigmoid(-x[..., C:])], -1),
            np.concatenate([np.abs(dy) * s, np.abs(dy * a) * s], -1))
