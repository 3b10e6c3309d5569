"""Every form of the attention's kernels, forward and gradients, over the shapes
of tests/attn_forms.py, against the definition in 64 bits.  The tolerances are
those of test_gpu_dwattn.py and test_gpu_dwattn_bwd.py: scores stay below 32 in
units of log2 here too."""
import math

import pytest
import torch

import attn_forms
import attn_ref64
import block_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F32, BF16 = torch.float32, torch.bfloat16


def lib():
    import conv_subsampling_amd as dw
    return dw


def make(c):
    B, Tq, Tk, H, Hkv, D = (c[n] for n in ("B", "Tq", "Tk", "H", "Hkv", "D"))
    dt, pad = BF16 if c["elem"] == 2 else F32, c.get("pad", 0)
    g = torch.Generator(device=DEV)
    g.manual_seed(B * 1000003 + Tk * 1009 + D * 31 + c["elem"])

    def normal(T, heads, more):
        t = torch.randn((B, T, heads * D + more), generator=g, device=DEV).to(dt)
        return t[..., :heads * D].unflatten(2, (heads, D))

    i32 = lambda n: torch.tensor(c[n], dtype=torch.int32, device=DEV) if n in c else None  # noqa: E731
    s = dict(B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, D=D, dt=dt, left=c.get("left", -1), right=c.get("right", -1),
             q=normal(Tq, H, pad), k=normal(Tk, Hkv, pad), v=normal(Tk, Hkv, pad), dout=normal(Tq, H, 0).contiguous(),
             q_lengths=i32("q_len"), k_lengths=i32("k_len"), q_pos=i32("pos"), table=None, buckets=None)
    if c.get("bias", True):
        s["table"] = torch.randn((16, H), generator=g, device=DEV).to(dt)
        s["buckets"] = lib().rel_buckets(16, c.get("reach", 40), device=DEV)
        if c.get("special"):
            s["table"][0], s["table"][5] = -math.inf, torch.finfo(dt).min
    return s


def arguments(s):
    return s["table"], s["buckets"], s["q_lengths"], s["k_lengths"], s["q_pos"], s["left"], s["right"]


def check_forward(s):
    out, lse = lib().dwattn_fwd(s["q"], s["k"], s["v"], *arguments(s))
    torch.cuda.synchronize()
    want, wlse = attn_ref64.forward(s)
    assert torch.isfinite(out).all()
    tol = 2e-5 + (ref.U16 * float(s["v"].float().abs().max()) if s["dt"] == BF16 else 0)
    off = (out.double() - want).abs()
    assert float(off.max()) <= tol, f"out off by {float(off.max()):.3e} of {tol:.3e} at {int(off.argmax())}"
    empty = wlse == -math.inf
    assert torch.equal(empty, lse == -math.inf)
    far = (lse.double() - wlse)[~empty].abs().max()
    assert float(far) <= 1e-5 * (1 + float(wlse[~empty].abs().max())), f"lse off by {float(far):.3e}"
    assert not out[empty.transpose(1, 2)].any()
    again = lib().dwattn_fwd(s["q"], s["k"], s["v"], *arguments(s))
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    return out, lse


@pytest.mark.parametrize("case", attn_forms.self_attention() + attn_forms.few_queries(), ids=attn_forms.name)
def test_forward(case):
    say("attention forward", case)
    check_forward(make(case))


@pytest.mark.parametrize("case", attn_forms.self_attention(), ids=attn_forms.name)
def test_gradients(case):
    say("attention gradients", case)
    s = make(case)
    out, lse = check_forward(s)
    calls = [lib().dwattn_bwd(s["q"], s["k"], s["v"], out, lse, s["dout"], *arguments(s)) for _ in range(2)]
    torch.cuda.synchronize()
    want, bound = attn_ref64.backward(s, out, lse)
    for name, g, g2, w, b in zip(("dq", "dk", "dv", "dtable"), *calls, want, bound):
        if w is None:
            assert g is None
            continue
        assert torch.equal(g, g2), f"{name} differs from call to call"
        assert torch.isfinite(g).all(), name
        tol = 2e-5 * (b + 1e-6)
        if s["dt"] == BF16 and name != "dtable":
            tol = tol + ref.U16 * b + ref.U16 * w.abs()
        off = (g.double() - w).abs()
        assert bool((off <= tol).all()), f"{name}: {float(off.max()):.3e}, {int((off > tol).sum())} past their bound"
        assert name == "dtable" or not g[b == 0].any(), f"{name}: not zero where nothing flows"
