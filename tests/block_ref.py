"""The encoder block's operators in 64 bits, as plainly as they are defined:
NumPy on the host, sharing nothing with the library."""
import numpy as np

U32 = 2.0 ** -24   # unit roundoff of float32
U16 = 2.0 ** -8    # largest relative distance of a bfloat16 rounding


def philox4x32(counter, key):
    """Philox4x32-10 of one 4-word counter and 2-word key, in whole numbers."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & 0xFFFFFFFF, (a >> 32) ^ c[3] ^ k[1], a & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return c


def drop_factor(rows, C, seed, stream, p):
    """[rows, C]: 0 where the element is dropped, else the scale."""
    n = min(65535, int(np.floor(p * 65536 + 0.5)))
    G = -(-C // 8)
    word = np.uint64(0xFFFFFFFF)
    g = np.arange(rows * G, dtype=np.uint64)
    c = [g & word, g >> np.uint64(32), np.full_like(g, stream & 0xFFFFFFFF), np.full_like(g, stream >> 32)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & word, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & word]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    u = np.stack([h for w in c for h in (w & np.uint64(0xFFFF), w >> np.uint64(16))], 1).reshape(rows, G * 8)[:, :C]
    return np.where(u >= n, 65536.0 / (65536 - n), 0.0)


def norm_fwd(x, gamma, beta, lengths, residual, factor, alpha, eps=1e-5):
    """(y, s, mean, rstd); frames past the lengths are zero and their inputs unused."""
    B, T, C = x.shape
    y, s, mean, rstd = np.zeros((B, T, C)), np.zeros((B, T, C)), np.zeros((B, T)), np.zeros((B, T))
    for b in range(B):
        for t in range(int(np.clip(lengths[b], 0, T))):
            r = alpha * x[b, t] * factor[b, t] + (0.0 if residual is None else residual[b, t])
            m = r.mean()
            q = 1.0 / np.sqrt(((r - m) ** 2).mean() + eps)
            y[b, t] = (r - m) * q * gamma + beta
            s[b, t], mean[b, t], rstd[b, t] = r, m, q
    return y, s, mean, rstd


def norm_bwd(s, gamma, lengths, mean, rstd, dy, dsum, factor, alpha):
    """(dx, dres, dgamma, dbeta) and the sums of the absolute terms of the last two."""
    B, T, C = s.shape
    dx, dres = np.zeros((B, T, C)), np.zeros((B, T, C))
    dg, db, ag, ab = np.zeros(C), np.zeros(C), np.zeros(C), np.zeros(C)
    for b in range(B):
        for t in range(int(np.clip(lengths[b], 0, T))):
            xh = (s[b, t] - mean[b, t]) * rstd[b, t]
            g = dy[b, t] * gamma
            d = rstd[b, t] * (g - g.mean() - xh * (g * xh).mean()) + (0.0 if dsum is None else dsum[b, t])
            dres[b, t], dx[b, t] = d, alpha * factor[b, t] * d
            dg += dy[b, t] * xh
            db += dy[b, t]
            ag += np.abs(dy[b, t] * xh)
            ab += np.abs(dy[b, t])
    return dx, dres, dg, db, ag, ab


def bucket(rel, buckets, reach, bidirectional):
    """The bucket of one distance, in whole numbers."""
    per = buckets // 2 if bidirectional else buckets
    n = abs(rel) if bidirectional else max(0, -rel)
    n, e = min(n, reach), per // 2
    b = n
    if n >= e:
        m, k = per - e, 0
        while k + 1 < m and n ** m * e ** (k + 1) >= reach ** (k + 1) * e ** m:
            k += 1
        b = e + k
    return b + (per if bidirectional and rel > 0 else 0)


def attn(q, k, v, table, buckets, q_len, k_len, pos, left, right, scale, dout=None, out=None, lse=None):
    """Attention of [B,T,H,D] arrays.  Returns (out, lse), or with dout (dq, dk, dv, dtable) and the sums of the
    absolute terms of dtable; there out and lse are the forward's as given."""
    B, Tq, H, D = q.shape
    Tk, G = k.shape[1], H // k.shape[2]
    R = 0 if buckets is None else len(buckets) // 2
    bwd = dout is not None
    if not bwd:
        out, lse = np.zeros_like(q), np.full((B, H, Tq), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    dt = None if table is None else np.zeros_like(table)
    at = None if table is None else np.zeros_like(table)
    for b in range(B):
        nq, nk = int(np.clip(q_len[b], 0, Tq)), int(np.clip(k_len[b], 0, Tk))
        if not nq or not nk:
            continue
        rel = np.arange(nk)[None, :] - np.arange(nq)[:, None] - int(pos[b])
        seen = np.ones((nq, nk), bool)
        if left >= 0:
            seen &= rel >= -left
        if right >= 0:
            seen &= rel <= right
        place = None if buckets is None else np.asarray(buckets)[np.clip(rel, -R, R) + R]
        for h in range(H):
            kk, vv = k[b, :nk, h // G], v[b, :nk, h // G]
            S = scale * (q[b, :nq, h] @ kk.T) + (0.0 if table is None else table[place, h])
            S = np.where(seen, S, -np.inf)
            if not bwd:
                m = S.max(1, keepdims=True)
                m = np.where(np.isinf(m), 0.0, m)
                P = np.exp(S - m)
                total = P.sum(1, keepdims=True)
                out[b, :nq, h] = np.where(total > 0, P @ vv / np.where(total > 0, total, 1), 0.0)
                with np.errstate(divide="ignore"):
                    lse[b, h, :nq] = (m + np.log(total))[:, 0]
                continue
            ls = lse[b, h, :nq, None]
            P = np.where(np.isinf(ls) | ~seen, 0.0, np.exp(S - np.where(np.isinf(ls), 0.0, ls)))
            do, o = dout[b, :nq, h], out[b, :nq, h]
            dS = P * (do @ vv.T - (do * o).sum(1, keepdims=True))
            dq[b, :nq, h] = scale * dS @ kk
            dk[b, :nk, h // G] += scale * dS.T @ q[b, :nq, h]
            dv[b, :nk, h // G] += P.T @ do
            if table is not None:
                np.add.at(dt[:, h], place, dS)
                np.add.at(at[:, h], place, np.abs(dS))
    return (dq, dk, dv, dt, at) if bwd else (out, lse)
