"""Launch plans of the recurrence and of the heads' gradients that only many
sequences or many frames reach, against the definitions in 64 bits: chains of
more than four tiles in turn, and teams that take several frames in turn.
The tolerances are those of test_gpu_dwscan.py and test_gpu_dwrope.py, which
count frames, tiles and rows."""
import pytest
import torch

import test_gpu_dwrope as heads
import test_gpu_dwscan as scan

pytestmark = pytest.mark.gpu
TYPES = pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])


@TYPES
@pytest.mark.parametrize("B,T,C", [(512, 330, 2), (512, 1100, 3), (256, 400, 66), (256, 1090, 65), (64, 321, 512), (520, 64 * 5, 1)])
def test_five_and_more_tiles_in_turn(B, T, C, dt):
    """512 chains and more; one item of each length at its tile's ends and around, some empty, one past the last frame."""
    edges = [0, 1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 319, 320, 321, T - 1, T, T + 9]
    L = [min(edges[b % len(edges)], T + 9) if b % 3 else max(1, T - (b * T) // (2 * B)) for b in range(B)]
    s = scan.make(B, T, C, dt, L, tag="turns")
    scan.say("scan in turn", B, T, C, dt)
    assert B * -(-C // 64) >= 512 and scan.lib().dwscan_fwd_workspace_bytes(B, T, C) == 0
    got = scan.check_fwd(s)
    back = scan.check_bwd(s, got[0])
    state = s["h0"].clone()  # again, with the states in place
    again = scan.lib().dwscan_fwd(s["x"], s["r"], s["g"], s["decay"], s["lengths"], h0=state, h_last=state)
    assert torch.equal(again[0], got[0]) and torch.equal(state, got[1])
    dh = s["dh_last"].clone()
    for a, b in zip(scan.grads(s | {"dh_last": dh}, got[0], dh0=dh), back):
        assert torch.equal(a, b)


@TYPES
@pytest.mark.parametrize("D,R,pairs,B,T", [(128, 128, "halves", 3, 6001), (100, 36, "neighbours", 3, 6001), (50, 50, "halves", 5, 6700),
                                           (64, 64, "neighbours", 5, 6700), (32, 32, "halves", 7, 9500), (128, 64, "halves", 17, 2900)])
def test_frames_in_several_turns(D, R, pairs, B, T, dt):
    """More frames than workgroups have teams (1024 of 16, 32 or 64): each adds the gammas' gradients of two frames or more."""
    lanes = 4 if D <= 32 else 8 if D <= 64 else 16
    assert B * T > 1024 * 256 // lanes
    L = [T - (b * T) // (2 * B) for b in range(B - 1)] + [0]
    s = heads.make(B, T, 1, 1, D, R, dt, pairs, L, [3 * b for b in range(B)], seed=7)
    heads.say("rope in turns", B, T, D, R, dt)
    heads.check_bwd(s)
