"""Attention with a bucketed relative position bias and its gradients in 64
bits over whole batches: plain torch on the tensors' device, for the sizes that
the loops of block_ref would take long over."""
import math

import torch


def _heads(t, repeat=1):
    return t.double().permute(0, 2, 1, 3).repeat_interleave(repeat, 1).contiguous()


def _back(t):
    return t.permute(0, 2, 1, 3)


def scores(s):
    """Scores [B,H,Tq,Tk] with -inf where a pair is not allowed, and each pair's bucket [B,Tq,Tk] (or None)."""
    B, Tq, Tk, G = s["B"], s["Tq"], s["Tk"], s["H"] // s["Hkv"]
    i = torch.arange(Tq, device=s["q"].device)[None, :, None]
    j = torch.arange(Tk, device=s["q"].device)[None, None, :]
    r = j - i - (0 if s["q_pos"] is None else s["q_pos"].long()[:, None, None])
    seen = torch.ones((B, Tq, Tk), dtype=torch.bool, device=r.device)
    if s["q_lengths"] is not None:
        seen &= i < s["q_lengths"][:, None, None]
    if s["k_lengths"] is not None:
        seen &= j < s["k_lengths"][:, None, None]
    if s["left"] >= 0:
        seen &= r >= -s["left"]
    if s["right"] >= 0:
        seen &= r <= s["right"]
    S = torch.matmul(_heads(s["q"]), _heads(s["k"], G).transpose(-1, -2).contiguous()) * s["D"] ** -0.5
    place = None
    if s["table"] is not None:
        R = len(s["buckets"]) // 2
        place = s["buckets"].long()[r.clamp(-R, R) + R].expand(B, Tq, Tk)
        S = S + s["table"].double()[place].permute(0, 3, 1, 2)
    return torch.where(seen[:, None], S, -math.inf), place


def forward(s):
    S, _ = scores(s)
    lse = torch.logsumexp(S, -1)
    P = torch.exp(S - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    return _back(torch.matmul(P, _heads(s["v"], s["H"] // s["Hkv"]))), lse


def backward(s, out, lse):
    """(dq, dk, dv, dtable) given the forward's out and lse, and for each the sum of its terms' sizes."""
    S, place = scores(s)
    G, scale, shape = s["H"] // s["Hkv"], s["D"] ** -0.5, (s["B"], s["Hkv"], s["H"] // s["Hkv"])
    lse = lse.double()[..., None]
    P = torch.exp(S - torch.where(lse == -math.inf, 0.0, lse))
    del S
    q, k, v, do, o = _heads(s["q"]), _heads(s["k"], G), _heads(s["v"], G), _heads(s["dout"]), _heads(out)

    def all_of(f, minus):
        dS = P * (torch.matmul(f(do), f(v).transpose(-1, -2).contiguous()) + minus * (f(do) * f(o)).sum(-1, keepdim=True))
        shared = lambda t: _back(t.unflatten(1, (s["Hkv"], G)).sum(2))  # noqa: E731
        turned = dS.transpose(-1, -2).contiguous()
        table = None
        if place is not None:
            table = torch.stack([(dS * (place == n)[:, None]).sum((0, 2, 3)) for n in range(len(s["table"]))])
        return (_back(torch.matmul(dS, f(k)) * scale), shared(torch.matmul(turned, f(q)) * scale),
                shared(torch.matmul(P.transpose(-1, -2).contiguous(), f(do))), table)

    return all_of(lambda t: t, -1), all_of(torch.abs, 1)
