"""Calls around attention whose inputs other than the rows -- weights, angles, scales of an E4M3 cache -- have just been
written by the call before, which may still run when the next one starts."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("chains", tag, *shape), dtype, "cuda")


@pytest.mark.parametrize("D", [128, 34])
def test_weights_written_by_the_call_before(D):
    """Both weights are turned in place, a step each time, between the norms and their gradients."""
    L, Hq, Hk = 600, 6, 2
    q, k, gq, gk = (act(L, h, D, tag=n) for n, h in (("q", Hq), ("k", Hk), ("gq", Hq), ("gk", Hk)))
    cos, sin = dit.rotary_table(torch.arange(L, device="cuda"), dit.rotary_frequencies(D // 2))
    one_cos, one_sin = cos[7:8].contiguous(), sin[7:8].contiguous()

    def chain(wait):
        w = act(2, 1, D, tag="w")
        wq, wk = w[0, 0], w[1, 0]
        outs = []
        for _ in range(8):
            outs += dit.rmsnorm_rope(q, k, wq, wk, cos, sin)
            wait()
            dit.rope(w[:1], w[1:], one_cos, one_sin, out_q=w[:1], out_k=w[1:])
            wait()
            outs += dit.rmsnorm_rope(q, k, wq, wk, cos, sin)
            wait()
            dit.rope(w[:1], w[1:], one_cos, one_sin, out_q=w[:1], out_k=w[1:])
            wait()
            outs += dit.rmsnorm_rope_backward(gq, gk, q, k, wq, wk, cos, sin)
            wait()
        return outs + [w]

    got = chain(lambda: None)
    want = chain(torch.cuda.synchronize)
    assert len(got) == len(want) == 8 * 8 + 1
    for n, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), n
    assert not torch.equal(want[0], want[2]) and not torch.equal(want[0], want[8])
