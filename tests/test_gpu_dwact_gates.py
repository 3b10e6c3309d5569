"""Gradients of kept activations whose gates are open or shut: sigmoid(-b) of
down to 1e-38 against the definition in 64 bits.  16 roundings of 2^-24 (U) of a term as in
test_gpu_dwact.py, where 1 - sigmoid is a factor of the term; bf16 gates add |b| of them."""
import pytest
import torch

import datagen
import recur_exact as exact
import recur_ref as ref
from test_gpu_dwact import BF16, DEV, F32, host64, lib, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16], ids=["f32", "bf16"])
@pytest.mark.parametrize("kind", ["silu", "glu"])
@pytest.mark.parametrize("lo,hi", [(0.0, 4.0), (8.0, 12.0), (12.0, 20.0), (20.0, 60.0), (60.0, 87.0)])
@pytest.mark.parametrize("C", [64, 50])
def test_gates_far_from_zero(C, lo, hi, kind, dt):
    W = C * (2 if kind == "glu" else 1)
    n = f"far/{C}/{lo}/{kind}"
    x = datagen.uniform((2, 9, W), lo, hi, n, device=DEV) * torch.sign(datagen.normal((2, 9, W), 1.0, n + "/sign", device=DEV))
    x, dy = x.to(dt), datagen.normal((2, 9, C), 1.0, n + "/dy", device=DEV).to(dt)
    _, kept = lib().dwact_fwd(x, kind)
    dx, y = lib().dwact_bwd(kept, dy, kind, need=("dx", "y"))
    torch.cuda.synchronize()
    parts = W // C
    xk = ref.unpack(host64(kept[0]).reshape(18, W), kept[1].cpu().numpy().reshape(18, -1), parts).reshape(x.shape)
    want, size = exact.act_grad(xk, host64(dy), kind)
    near(dx, want, size, xk, dt, "dx")
    act = ref.act(xk, kind)
    near(y, act, abs(act), xk, dt, "y")
