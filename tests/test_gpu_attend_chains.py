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


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [128, 34])
def test_e4m3_rows_written_by_the_call_before(D, dtype):
    """The same places get rows of other sizes each time, so that codes and scales differ from step to step: in place from
    the packed projection into an E4M3 cache, back, and attention over it."""
    L, size = 500, 8
    w = act(D, tag="w", dtype=dtype)
    qkv = act(L, 6, D, tag="qkv", dtype=dtype)
    slots = torch.arange(L, device="cuda")
    pages = torch.arange(-(-L // size), device="cuda").int()[None].expand(L, -1)
    lengths = slots + 1

    def chain(wait):
        cache = dit.KVCache.empty(-(-L // size), 1, size, D, torch.float8_e4m3fn)
        for t in (cache.k.view(torch.uint8), cache.v.view(torch.uint8), cache.k_scales, cache.v_scales):
            t.zero_()
        outs = []
        for i in range(10):
            x = qkv * float(2.0 ** (i % 4) * (1 + 0.25 * i))
            q, k, v = x[:, :4], x[:, 4:5], x[:, 5:]
            cos, sin = dit.rotary_table(slots + 17 * i, freqs)
            wait()
            dit.rmsnorm_rope(q, k, w, w, cos, sin, weight_offset=float(i), out_q=q, out_k=k)
            wait()
            dit.cache_write(cache, k, v, slots)
            wait()
            outs += dit.paged_attention(q, cache, pages, lengths, need_lse=True)
            wait()
            outs += dit.cache_read(cache, slots, dtype=x.dtype)
            wait()
        return outs

    freqs = dit.rotary_frequencies(D // 2)
    got = chain(lambda: None)
    want = chain(torch.cuda.synchronize)
    for n, (a, b) in enumerate(zip(got, want, strict=True)):
        assert torch.equal(a, b), n
    assert not torch.equal(want[3], want[7])  # (the scales do differ)
