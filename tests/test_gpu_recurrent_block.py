"""The recurrent example block: its gradients against the same block in 64 bits
and against differences, and its stream against the whole utterance."""
import importlib.util
import os

import pytest
import torch

import datagen

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def block():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "recurrent_block.py")
    spec = importlib.util.spec_from_file_location("recurrent_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def setup(T=40, C=64):
    m = block()
    w = m.parameters(C, 4, 2, seed=3)
    freq = m.dw.rope_frequencies(C // 4)
    lengths = torch.tensor([T, 25, 33], dtype=torch.int32, device=DEV)
    x = datagen.normal((3, T, C), 1.0, "recur/x", device=DEV)
    valid = (torch.arange(T, device=DEV)[None] < lengths[:, None]).float()[..., None]
    return m, w, freq, lengths, x, datagen.normal((3, T, C), 1.0, "recur/dout", device=DEV) * valid, valid


def in_64_bits(m, w, x, lengths, freq):
    """The block's output from its formulas, on the host, for torch's own gradients."""
    w = {k: v.double() for k, v in w.items()}
    B, T, C = x.shape
    D = w["qg"].shape[0]
    H, live = C // D, (torch.arange(T)[None] < lengths[:, None])[..., None]

    def norm(s, g, b):
        d = s - s.mean(-1, keepdim=True)
        return d / (d.square().mean(-1, keepdim=True) + 1e-5).sqrt() * g + b
    y1 = norm(x, w["g1"], w["b1"])
    Hkv = (w["wqkv"].shape[1] // D - H) // 2
    q, k, v = (y1 @ w["wqkv"]).view(B, T, -1, D).split([H, Hkv, Hkv], 2)
    ang = torch.arange(T, dtype=torch.float64)[:, None, None] * freq

    def turn(t, g):
        t = t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * g
        a, b = t.chunk(2, -1)
        return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    q, k = turn(q, w["qg"]), turn(k, w["kg"])
    k, v = (t.repeat_interleave(H // Hkv, 2) for t in (k, v))
    S = torch.einsum("bihd,bjhd->bhij", q, k) * D ** -0.5
    seen = torch.tril(torch.ones(T, T, dtype=torch.bool)) & live[:, None, None, :, 0]
    a = torch.einsum("bhij,bjhd->bihd", S.masked_fill(~seen, -torch.inf).softmax(-1), v).reshape(B, T, C)
    s2 = x + a @ w["wo"]
    u = norm(s2, w["g2"], w["b2"]) @ w["wglu"]
    e = torch.where(live, u[..., :C] * torch.sigmoid(u[..., C:]), 0.0)
    pad = torch.nn.functional.pad(e, (0, 0, m.K - 1, 0))
    c = torch.where(live, sum(pad[:, t:t + T] * w["wdw"][t] for t in range(m.K)) + w["bdw"], 0.0)
    r, g = (c @ w["wgate"]).chunk(2, -1)
    z = 8 * torch.nn.functional.softplus(w["decay"]) * torch.sigmoid(r)
    h, ys = torch.zeros(B, C, dtype=torch.float64), []
    for t in range(T):
        h = torch.exp(-z[:, t]) * h + (-torch.expm1(-2 * z[:, t])).sqrt() * torch.sigmoid(g[:, t]) * c[:, t]
        ys.append(h)
    return torch.where(live, torch.stack(ys, 1) @ w["wp"] + s2, 0.0)


def test_forward_and_gradients_against_64_bits():
    """The forward within 1e-4 (ten sums of at most 128 float32 terms of unit scale, twice over).  In the gradients, the kept
    activations are off by half a step of 8 bits: up to 1/127 of their group's largest, some 2% of a typical value and of either sign.
    Each gradient sums hundreds of such terms, so a relative difference (norm to norm) of 3% allows for what each of the two checkpoints
    adds and for nothing of the size of a missing or doubled path."""
    m, w, freq, lengths, x, dout, valid = setup()
    out, kept = m.forward(w, x, lengths, freq)
    dx, grads = m.backward(w, kept, lengths, freq, dout)
    torch.cuda.synchronize()
    assert set(grads) == set(w)
    leaves = {k: v.double().cpu().requires_grad_() for k, v in w.items()}
    at = x.double().cpu().requires_grad_()
    want = in_64_bits(m, leaves, at, lengths.cpu(), freq.cpu())
    assert float((out * valid - want.to(DEV)).detach().abs().max()) <= 1e-4
    (want * dout.double().cpu()).sum().backward()
    for name, got, ref in [("x", dx * valid, at.grad), *((k, grads[k], leaves[k].grad) for k in w)]:
        off = float((got.double().cpu() - ref).norm() / ref.norm())
        assert off <= 3e-2, (name, off)


def test_parameters_behind_the_checkpoints_against_differences():
    """wp's and decay's gradients pass through one kept activation at most; their directional differences agree within the same 3%."""
    m, w, freq, lengths, x, dout, _ = setup()
    _, g = m.backward(w, m.forward(w, x, lengths, freq)[1], lengths, freq, dout)
    loss = lambda w: float((m.forward(w, x, lengths, freq)[0].double() * dout.double()).sum())  # noqa: E731
    for name in ("wp", "decay"):
        v = g[name] / g[name].norm()
        e = 1e-2
        diff = (loss({**w, name: w[name] + e * v}) - loss({**w, name: w[name] - e * v})) / (2 * e)
        exact = float((g[name].double() * v.double()).sum())
        assert abs(diff - exact) <= 3e-2 * max(1.0, abs(exact)), (name, diff, exact)


def test_stream_equals_the_whole_utterance_with_pauses():
    """Chunks of 1 to 64 frames, streams pausing in turn: each output passes through about ten sums of at most 150 float32 terms of unit
    scale, and 1e-4 is over ten times their rounding."""
    m = block()
    w = m.parameters(128, 4, 2, seed=5)
    freq = m.dw.rope_frequencies(32)
    B, T = 3, 150
    x = datagen.normal((B, T, 128), 1.0, "recur/stream", device=DEV)
    whole, _ = m.forward(w, x, None, freq)
    s = m.Stream(w, B, T, freq)
    done = [0] * B
    for n, chunk in enumerate((1, 8, 64, 1, 7, 69, 60, 64, 150)):
        take = [0 if (n + b) % 4 == 3 and n < 7 else min(chunk, T - done[b]) for b in range(B)]
        part = torch.zeros((B, max(1, *take), 128), device=DEV)
        for b in range(B):
            part[b, :take[b]] = x[b, done[b]:done[b] + take[b]]
        out = s.step(part, torch.tensor(take, dtype=torch.int32, device=DEV))
        for b in range(B):
            if take[b]:
                off = float((out[b, :take[b]] - whole[b, done[b]:done[b] + take[b]]).abs().max())
                assert off <= 1e-4, (n, b, off)
            done[b] += take[b]
    assert done == [T] * B


def test_the_example_runs(capsys):
    block().main()
    assert "largest difference" in capsys.readouterr().out
