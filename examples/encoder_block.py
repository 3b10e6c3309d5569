"""A Conformer encoder block's attention and convolution modules from this
library's operators: one training step (forward and gradients) and the same
block run as a stream, chunk by chunk, over its caches.

    python examples/encoder_block.py

Per frame: x -> norm -> attention with a bucketed relative position bias ->
dropout, residual add and the next norm in one pass -> pointwise, depthwise
conv, SiLU, pointwise -> dropout and residual add.  The block is causal, so
the stream gives what the whole utterance gives.  The projections are plain
matrix products.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import conv_subsampling_amd as dw  # noqa: E402

K = 9            # taps of the depthwise conv
BUCKETS, REACH = 32, 128


def parameters(C, H, seed=0, dtype=torch.float32, device="cuda"):
    """Random weights of a block of C channels with H heads."""
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def r(*shape, std):
        return (torch.randn(shape, generator=g, device=device) * std).to(dtype)

    return dict(
        g1=1 + r(C, std=0.1), b1=r(C, std=0.1), wqkv=r(C, 3 * C, std=C ** -0.5), table=r(BUCKETS, H, std=0.5),
        wo=r(C, C, std=C ** -0.5), g2=1 + r(C, std=0.1), b2=r(C, std=0.1), wp1=r(C, C, std=C ** -0.5),
        wdw=r(K, C, std=1 / K), bdw=r(C, std=0.1), wp2=r(C, C, std=C ** -0.5))


def forward(w, x, lengths, buckets, left=-1, rng=None, p=0.0):
    """The block over whole utterances x [B,T,C]; returns the output and what `backward` takes.  rng: two generator
    states (int64 [2] each), for the two dropouts."""
    B, T, C = x.shape
    H = w["table"].shape[1]
    r1, r2 = rng if rng is not None else (None, None)
    y1, _, m1, i1 = dw.dwnorm_fwd(x, w["g1"], w["b1"], lengths)
    q, k, v = (y1 @ w["wqkv"]).view(B, T, 3, H, C // H).unbind(2)
    a, lse = dw.dwattn_fwd(q, k, v, w["table"], buckets, lengths, lengths, left=left, right=0)
    y2, s2, m2, i2 = dw.dwnorm_fwd(a.view(B, T, C) @ w["wo"], w["g2"], w["b2"], lengths, residual=x, rng=r1, p=p)
    h = y2 @ w["wp1"]
    c = dw.dwconv1d_fwd(h, w["wdw"], w["bdw"], lengths, causal=True)
    e = torch.nn.functional.silu(c)
    out = dw.dwdrop_fwd(e @ w["wp2"], r2, p, residual=s2)
    return out, (x, y1, m1, i1, q, k, v, a, lse, y2, s2, m2, i2, h, c, e)


def backward(w, kept, lengths, buckets, dout, left=-1, rng=None, p=0.0):
    """(dx, gradients of the parameters) given dout.  Frames past the lengths carry no gradient."""
    x, y1, m1, i1, q, k, v, a, lse, y2, s2, m2, i2, h, c, e = kept
    B, T, C = x.shape
    r1, r2 = rng if rng is not None else (None, None)
    flat = lambda t: t.reshape(B * T, -1)  # noqa: E731
    g = {}
    de2 = dw.dwdrop_bwd(dout, r2, p)
    g["wp2"] = flat(e).T @ flat(de2)
    de = de2 @ w["wp2"].T
    s = torch.sigmoid(c)
    dh, g["wdw"], g["bdw"] = dw.dwconv1d_bwd(h, w["wdw"], lengths, (de * (s * (1 + c * (1 - s)))).contiguous(), causal=True)
    g["wp1"] = flat(y2).T @ flat(dh)
    do, dres, g["g2"], g["b2"] = dw.dwnorm_bwd(s2, w["g2"], lengths, m2, i2, dh @ w["wp1"].T, dsum=dout, rng=r1, p=p)
    g["wo"] = flat(a).T @ flat(do)
    dqkv = torch.empty((B, T, 3) + tuple(q.shape[2:]), dtype=x.dtype, device=x.device)
    dq, dk, dv = dqkv.unbind(2)   # the attention writes its gradients into slices of the projection's
    _, _, _, g["table"] = dw.dwattn_bwd(q, k, v, a, lse, (do @ w["wo"].T).view(a.shape), w["table"], buckets, lengths, lengths,
                                        left=left, right=0, dq=dq, dk=dk, dv=dv)
    dqkv = dqkv.view(B, T, 3 * C)
    g["wqkv"] = flat(y1).T @ flat(dqkv)
    dx, _, g["g1"], g["b1"] = dw.dwnorm_bwd(x, w["g1"], lengths, m1, i1, dqkv @ w["wqkv"].T, dsum=dres, need=("dx", "dgamma", "dbeta"))
    return dx, g


class Stream:
    """The block over chunks of frames: a cache of keys and values that the attention reads in place, and the conv's
    cache of K - 1 frames."""

    def __init__(self, w, streams, frames, buckets, left=-1):
        C, H = w["wo"].shape[0], w["table"].shape[1]
        like = dict(dtype=w["wo"].dtype, device=w["wo"].device)
        self.w, self.buckets, self.left = w, buckets, left
        self.kv = torch.zeros((streams, frames, 2, H, C // H), **like)
        self.conv = torch.zeros((streams, K - 1, C), **like)
        self.filled = 0
        self.count = torch.zeros((2, streams), dtype=torch.int32, device=w["wo"].device)   # frames cached, and with the chunk

    def step(self, x):
        w, (B, T, C), n = self.w, x.shape, self.filled
        H = w["table"].shape[1]
        y1, _, _, _ = dw.dwnorm_fwd(x, w["g1"], w["b1"], need=("y",))
        qkv = (y1 @ w["wqkv"]).view(B, T, 3, H, C // H)
        self.kv[:, n:n + T] = qkv[:, :, 1:]
        self.count[0].fill_(n)
        self.count[1].fill_(n + T)
        k, v = self.kv.unbind(2)
        a, _ = dw.dwattn_fwd(qkv[:, :, 0], k, v, w["table"], self.buckets, None, self.count[1], self.count[0],
                             left=self.left, right=0, need=("out",))
        y2, s2, _, _ = dw.dwnorm_fwd(a.view(B, T, C) @ w["wo"], w["g2"], w["b2"], residual=x, need=("y", "sum"))
        c, self.conv = dw.dwconv1d_stream_fwd(y2 @ w["wp1"], w["wdw"], w["bdw"], None, self.conv)
        self.filled = n + T
        return dw.dwdrop_fwd(torch.nn.functional.silu(c) @ w["wp2"], None, 0.0, residual=s2)


def main():
    B, T, C, H = 4, 200, 256, 4
    w = parameters(C, H)
    buckets = dw.rel_buckets(BUCKETS, REACH, bidirectional=False)
    x = torch.randn((B, T, C), device="cuda")
    lengths = torch.tensor([T, 150, 77, T], dtype=torch.int32, device="cuda")
    rng = [torch.tensor([1234, site], dtype=torch.int64, device="cuda") for site in (0, 1)]
    out, kept = forward(w, x, lengths, buckets, rng=rng, p=0.1)
    dx, grads = backward(w, kept, lengths, buckets, torch.randn_like(out), rng=rng, p=0.1)
    print("training step: out", tuple(out.shape), "gradients", {k: tuple(v.shape) for k, v in grads.items()})
    whole, _ = forward(w, x, None, buckets, left=96)
    stream = Stream(w, B, T, buckets, left=96)
    parts = torch.cat([stream.step(c.contiguous()) for c in x.split([8, 1, 40, 1, 150], 1)], 1)
    print("stream against the whole utterance: largest difference", float((parts - whole).abs().max()))


if __name__ == "__main__":
    main()
