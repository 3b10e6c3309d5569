"""The recurrence and the kept activations' gradients in 64 bits, with sums of
absolute terms that decay and vanish as the terms themselves do: every factor
of a term, a, a^2 and both halves of a gate, is in its sum, so that an error in
it counts in units of what is left of the term."""
import numpy as np

from recur_ref import clip, sigmoid, softplus


def gates(r, g, decay, scale):
    w = scale * softplus(decay) * sigmoid(r)
    return sigmoid(g), w, np.exp(-w), np.sqrt(-np.expm1(-2 * w))


def scan_fwd(x, r, g, decay, lengths=None, h0=None, scale=8.0):
    """(y, h_last), then for both the sum of absolute terms and that sum weighted by each term's -log of its decay."""
    B, T, C = x.shape
    L = clip(lengths, B, T)[:, None]
    h = np.zeros((B, C)) if h0 is None else h0.astype(np.float64)
    size, bent = np.abs(h), np.zeros((B, C))
    y, ysize, ybent = (np.zeros((B, T, C)) for _ in range(3))
    for t in range(T):
        live = t < L
        i, w, a, m = gates(r[:, t], g[:, t], decay, scale)
        u = m * i * x[:, t]
        h = np.where(live, a * h + u, h)
        bent = np.where(live, a * (bent + w * size), bent)
        size = np.where(live, a * size + np.abs(u), size)
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
    slope = sigmoid(decay) / softplus(decay)
    for t in range(T - 1, -1, -1):
        live = t < L
        i, w, a, m = gates(r[:, t], g[:, t], decay, scale)
        prev = y[:, t - 1] if t else h0
        full, fsize = G + dy[:, t], size + np.abs(dy[:, t])
        ix, ratio = i * x[:, t], a * a * w / m
        q, qa = full * (ix * ratio - w * a * prev), np.abs(ix) * ratio + w * a * np.abs(prev)
        shut, closed = sigmoid(-r[:, t]), sigmoid(-g[:, t])
        turned = bent + 2 * w * fsize  # a and a^2 themselves are bent by their own w
        for n, v, c, k in (("dx", full * m * i, m * i, bent), ("dg", full * m * ix * closed, m * np.abs(ix) * closed, bent),
                           ("dr", q * shut, qa * shut, turned)):
            o[n][:, t] = np.where(live, v, 0.0)
            o[n + "_size"][:, t] = np.where(live, c * fsize, 0.0)
            o[n + "_bent"][:, t] = np.where(live, c * k, 0.0)
        o["ddecay"] += np.where(live, q, 0.0).sum(0) * slope
        o["ddecay_size"] += np.where(live, qa * fsize, 0.0).sum(0) * slope
        o["ddecay_bent"] += np.where(live, qa * turned, 0.0).sum(0) * slope
        G = np.where(live, a * full, G)
        bent = np.where(live, a * (bent + w * fsize), bent)
        size = np.where(live, a * fsize, size)
    o["dh0"], o["dh0_size"], o["dh0_bent"] = G, size, bent
    return o


def act_grad(x, dy, kind):
    """(dx, its sums of absolute terms)."""
    if kind == "silu":
        s, o = sigmoid(x), sigmoid(-x)
        return dy * (s + x * s * o), np.abs(dy) * (s + np.abs(x) * s * o)
    C = x.shape[-1] // 2
    a, s, o = x[..., :C], sigmoid(x[..., C:]), sigmoid(-x[..., C:])
    dx = np.concatenate([dy * s, dy * a * s * o], -1)
    return dx, np.abs(dx)
