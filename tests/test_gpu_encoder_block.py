"""The example block: its gradients against differences of its forward, and its
stream against the whole utterance."""
import importlib.util
import os

import pytest
import torch

import datagen

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def block():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "encoder_block.py")
    spec = importlib.util.spec_from_file_location("encoder_block", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_gradients_against_differences():
    """<dL, v> of the hand-chained gradients against (L(+h) - L(-h)) / 2h, L = <out, w> over the valid frames in fp64 of
    fp32 outputs.  N = 3 * 40 * 64 outputs of unit scale leave about sqrt(N) * 1e-6 / h of rounding and a curvature of
    about h^2 times a few: at h = 1e-2 both stay under 2e-2 of gradients whose projections are of unit size."""
    m = block()
    C, H, T = 64, 2, 40
    w = m.parameters(C, H, seed=3)
    buckets = m.dw.rel_buckets(m.BUCKETS, m.REACH, bidirectional=False)
    lengths = torch.tensor([T, 25, 33], dtype=torch.int32, device=DEV)
    x = datagen.normal((3, T, C), 1.0, "block/x", device=DEV)
    valid = (torch.arange(T, device=DEV)[None] < lengths[:, None]).float()[..., None]
    dout = datagen.normal((3, T, C), 1.0, "block/dout", device=DEV) * valid
    rng = [torch.tensor([99, site], dtype=torch.int64, device=DEV) for site in (0, 1)]
    kw = dict(rng=rng, p=0.1, left=20)

    def loss(w, x):
        return float((m.forward(w, x, lengths, buckets, **kw)[0].double() * dout.double()).sum())

    dx, g = m.backward(w, m.forward(w, x, lengths, buckets, **kw)[1], lengths, buckets, dout, **kw)
    assert set(g) == set(w)
    for name, grad in [("x", dx), *g.items()]:
        at = x if name == "x" else w[name]
        v = datagen.normal(tuple(at.shape), 1.0, f"block/dir/{name}", device=DEV)
        v /= v.norm()
        h = 1e-2
        up, down = ((({**w}, x + s * v) if name == "x" else ({**w, name: at + s * v}, x)) for s in (h, -h))
        diff = (loss(*up) - loss(*down)) / (2 * h)
        exact = float((grad.double() * v.double()).sum())
        assert abs(diff - exact) <= 2e-2 * max(1.0, abs(exact)), (name, diff, exact)


@pytest.mark.parametrize("left", [-1, 50])
def test_stream_equals_the_whole_utterance(left):
    """Chunks of 1 to 64 frames.  Each output passes through about ten sums of at most 150 float32 terms of unit scale:
    1e-4 is over ten times their rounding."""
    m = block()
    w = m.parameters(128, 4, seed=5)
    buckets = m.dw.rel_buckets(m.BUCKETS, m.REACH, bidirectional=False)
    x = datagen.normal((2, 150, 128), 1.0, "block/stream", device=DEV)
    whole, _ = m.forward(w, x, None, buckets, left=left)
    s = m.Stream(w, 2, 150, buckets, left=left)
    parts = torch.cat([s.step(c.contiguous()) for c in x.split([1, 8, 64, 1, 7, 69], 1)], 1)
    assert float((parts - whole).abs().max()) <= 1e-4


def test_the_example_runs(capsys):
    block().main()
    assert "largest difference" in capsys.readouterr().out
