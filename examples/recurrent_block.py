"""A recurrent block and an attention block with rotated heads from this
library's operators: one training step (forward and gradients), whose
activations wait for the backward pass in 8 bits, and the same blocks run as a
stream, chunk by chunk, over their caches.

    python examples/recurrent_block.py

Per frame: x -> norm -> attention whose queries and keys are normed head by
head and turned by their positions -> residual add and the next norm in one
pass -> pointwise to twice the width, GLU, causal depthwise conv -> gated
linear recurrence -> pointwise -> residual add.  Everything is causal, so the
stream gives what the whole utterance gives.  The projections are plain matrix
products.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv_subsampling_amd as dw  # noqa: E402

K = 4            # taps of the depthwise conv


def parameters(C, H, Hkv, seed=0, dtype=torch.float32, device="cuda"):
    """Random weights of a block of C channels, H query heads and Hkv key heads."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def r(*shape, std):
        return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

    D = C // H
    return dict(
        g1=1 + r(C, std=0.1), b1=r(C, std=0.1), wqkv=r(C, (H + 2 * Hkv) * D, std=C ** -0.5), qg=1 + r(D, std=0.1),
        kg=1 + r(D, std=0.1), wo=r(C, C, std=C ** -0.5), g2=1 + r(C, std=0.1), b2=r(C, std=0.1),
        wglu=r(C, 2 * C, std=C ** -0.5), wdw=r(K, C, std=K ** -0.5), bdw=r(C, std=0.1),
        wgate=r(C, 2 * C, std=C ** -0.5), decay=-4 + r(C, std=1.0).float(), wp=r(C, C, std=C ** -0.5))


def _heads(w, y, H):
    """Queries, keys and values as slices of one projection's output."""
    D = w["qg"].shape[0]
    Hkv = (w["wqkv"].shape[1] // D - H) // 2
    return (y @ w["wqkv"]).view(*y.shape[:2], H + 2 * Hkv, D).split([H, Hkv, Hkv], 2)


def _gates(w, c):
    """The recurrence's two gates, slices of one projection's output."""
    return (c @ w["wgate"]).chunk(2, -1)


def forward(w, x, lengths, freq):
    """The block over whole utterances x [B,T,C]; returns the output and what `backward` takes.  Of the two wide
    activations (the GLU's input and the conv's output) 8 bits are kept."""
    B, T, C = x.shape
    y1, _, m1, i1 = dw.dwnorm_fwd(x, w["g1"], w["b1"], lengths)
    q, k, v = _heads(w, y1, C // w["qg"].shape[0])
    qr, kr, _ = dw.dwrope_fwd(q, k, w["qg"], w["kg"], freq, lengths)
    a, lse = dw.dwattn_fwd(qr, kr, v, q_lengths=lengths, k_lengths=lengths, right=0)
    y2, s2, m2, i2 = dw.dwnorm_fwd(a.view(B, T, C) @ w["wo"], w["g2"], w["b2"], lengths, residual=x)
    e, glu8 = dw.dwact_fwd(y2 @ w["wglu"], "glu", lengths)
    c = dw.dwconv1d_fwd(e, w["wdw"], w["bdw"], lengths, causal=True)
    _, c8 = dw.dwact_fwd(c, "none", lengths, need=("kept",))
    r, g = _gates(w, c)
    h, _ = dw.dwscan_fwd(c, r, g, w["decay"], lengths)
    out = h @ w["wp"] + s2
    return out, (x, y1, m1, i1, q, k, v, qr, kr, a, lse, y2, s2, m2, i2, glu8, c8, h)


def backward(w, kept, lengths, freq, dout):
    """(dx, gradients of the parameters) given dout.  Frames past the lengths carry no gradient."""
    x, y1, m1, i1, q, k, v, qr, kr, a, lse, y2, s2, m2, i2, glu8, c8, h = kept
    B, T, C = x.shape
    dt = x.dtype
    flat = lambda t: t.reshape(B * T, -1)  # noqa: E731
    grads = {"wp": flat(h).T @ flat(dout)}
    _, c = dw.dwact_bwd(c8, None, "none", lengths, dtype=dt, need=("y",))  # the conv's output, from its 8 bits
    r, g = _gates(w, c)
    dgates = torch.empty((B, T, 2 * C), dtype=dt, device=x.device)
    dr, dg = dgates.chunk(2, -1)  # the recurrence writes its gates' gradients into slices of the projection's
    dc, _, _, grads["decay"], _ = dw.dwscan_bwd(c, r, g, w["decay"], h, dout @ w["wp"].T, lengths, dr=dr, dg=dg,
                                                need=("dx", "ddecay"))
    grads["wgate"] = flat(c).T @ flat(dgates)
    dc = dc + dgates @ w["wgate"].T
    _, e = dw.dwact_bwd(glu8, None, "glu", lengths, dtype=dt, need=("y",))
    de, grads["wdw"], grads["bdw"] = dw.dwconv1d_bwd(e, w["wdw"], lengths, dc, causal=True)
    dglu, _ = dw.dwact_bwd(glu8, de, "glu", lengths)
    grads["wglu"] = flat(y2).T @ flat(dglu)
    do, dres, grads["g2"], grads["b2"] = dw.dwnorm_bwd(s2, w["g2"], lengths, m2, i2, dglu @ w["wglu"].T, dsum=dout)
    grads["wo"] = flat(a).T @ flat(do)
    dqkv = torch.empty((B, T, q.shape[2] + 2 * k.shape[2], q.shape[3]), dtype=dt, device=x.device)
    dq, dk, dv = dqkv.split([q.shape[2], k.shape[2], k.shape[2]], 2)
    dw.dwattn_bwd(qr, kr, v, a, lse, (do @ w["wo"].T).view(a.shape), q_lengths=lengths, k_lengths=lengths, right=0, dq=dq, dk=dk,
                  dv=dv)
    _, _, grads["qg"], grads["kg"] = dw.dwrope_bwd(q, k, dq, dk, w["qg"], w["kg"], freq, lengths, dq=dq, dk=dk)  # in place
    dqkv = dqkv.view(B, T, -1)
    grads["wqkv"] = flat(y1).T @ flat(dqkv)
    dx, _, grads["g1"], grads["b1"] = dw.dwnorm_bwd(x, w["g1"], lengths, m1, i1, dqkv @ w["wqkv"].T, dsum=dres,
                                                    need=("dx", "dgamma", "dbeta"))
    return dx, grads


class Stream:
    """The block over chunks of frames: caches of keys and values that the rotation writes and the attention reads in
    place, the conv's cache of K - 1 frames and the recurrence's state.  Streams may pause (a length of 0)."""

    def __init__(self, w, streams, frames, freq):
        C, D = w["wo"].shape[0], w["qg"].shape[0]
        H = C // D
        Hkv = (w["wqkv"].shape[1] // D - H) // 2
        like = dict(dtype=w["wo"].dtype, device=w["wo"].device)
        self.w, self.H, self.freq = w, H, freq
        self.k, self.v = torch.zeros((2, streams, frames, Hkv, D), **like).unbind(0)
        self.conv = torch.zeros((streams, K - 1, C), **like)
        self.state = torch.zeros((streams, C), dtype=torch.float32, device=w["wo"].device)
        self.filled = torch.zeros(streams, dtype=torch.int32, device=w["wo"].device)

    def step(self, x, lengths):
        w, (B, T, C) = self.w, x.shape
        y1, _, _, _ = dw.dwnorm_fwd(x, w["g1"], w["b1"], lengths, need=("y",))
        q, k, v = _heads(w, y1, self.H)
        q, _, _ = dw.dwrope_fwd(q, k, w["qg"], w["kg"], self.freq, lengths, pos=self.filled, v=v, place=self.filled, k_out=self.k,
                                v_out=self.v)
        after = self.filled + lengths
        a, _ = dw.dwattn_fwd(q, self.k, self.v, q_lengths=lengths, k_lengths=after, q_pos=self.filled, right=0, need=("out",))
        y2, s2, _, _ = dw.dwnorm_fwd(a.view(B, T, C) @ w["wo"], w["g2"], w["b2"], lengths, residual=x, need=("y", "sum"))
        e, _ = dw.dwact_fwd(y2 @ w["wglu"], "glu", lengths, need=("y",))
        c, self.conv = dw.dwconv1d_stream_fwd(e, w["wdw"], w["bdw"], lengths, self.conv)
        r, g = _gates(w, c)
        h, _ = dw.dwscan_fwd(c, r, g, w["decay"], lengths, h0=self.state, h_last=self.state)
        self.filled = after
        return h @ w["wp"] + s2


def main():
    B, T, C, H, Hkv = 4, 200, 256, 4, 2
    w = parameters(C, H, Hkv)
    freq = dw.rope_frequencies(C // H)
    x = torch.randn((B, T, C), device="cuda")
    lengths = torch.tensor([T, 150, 77, T], dtype=torch.int32, device="cuda")
    out, kept = forward(w, x, lengths, freq)
    dx, grads = backward(w, kept, lengths, freq, torch.randn_like(out))
    print("training step: out", tuple(out.shape), "gradients", {k: tuple(v.shape) for k, v in grads.items()})
    whole, _ = forward(w, x, None, freq)
    stream = Stream(w, B, T, freq)
    parts = torch.cat([stream.step(c.contiguous(), torch.full((B,), c.shape[1], dtype=torch.int32, device="cuda"))
                       for c in x.split([8, 1, 40, 1, 150], 1)], 1)
    print("stream against the whole utterance: largest difference", float((parts - whole).abs().max()))


if __name__ == "__main__":
    main()
