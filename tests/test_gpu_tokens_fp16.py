"""A captured training step of tokens.step in fp16 with finite gradients."""
import pytest
import torch

from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300 import tokens
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().flatten().clone().view(torch.uint8)


@pytest.mark.parametrize("n,V,D", [(700, 300, 512), (200, 40, 257)])
def test_captured_fp16_step_of_a_full_batch(n, V, D):
    """Without padded rows (whose gradients, r = 1000 at each norm, overflow
    fp16) every gradient is finite; a replay gives the eager step's bits."""
    ensure_built()
    ids, table, weights, stand_ins = tokens.make_inputs(n, V, D, 2, "fp16")
    gy = draw("act", (n, D), seed_for("tokens", "gy16", n, D), "fp16", "cuda") * 0.125
    args = (gy, ids, table, weights, stand_ins, 0.5, 8.0, 1e-6)
    graph, out = tokens.capture_step(*args)
    seen = []
    for r in range(3):
        ids.copy_(torch.roll(ids, 17 * r))
        gy.mul_(1.0 if r == 0 else 0.5)
        y, grads, norm = tokens.step(*args)
        graph.replay()
        torch.cuda.synchronize()
        assert 0.5 < float(norm) < float("inf")  # and the clipping takes part
        for t in (y, *grads):
            assert bool(torch.isfinite(t).all())
        assert all(bool(t.any()) for t in grads)
        for a, b in zip([out[0], out[2], *out[1]], [y, norm, *grads]):
            assert torch.equal(bits(a), bits(b))
        seen.append(float(norm))
    assert len(set(seen)) == 3
