"""Decoding steps of the token transformer (tokens.decode_attending) held tightly against 64 bits: the reference takes the
old tokens' keys and values as the cache holds them, so that what is compared is one step's arithmetic and not what
earlier roundings have become."""
import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300 import tokens as tk
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for
from test_gpu_tokens_attend import B, D, HEADS, SIZE, V, rms, setup, turned

pytestmark = pytest.mark.gpu

# Both sides round every stored tensor to the dtype (or to E4M3), so an element differs by one step where it lies next to the
# middle of two, and by no more than the fp32 arithmetic's error elsewhere.  If all elements of the at most five
# tensors of each of the four sites differed by one step, independently, the root mean square of x's difference
# would be sqrt(20) steps of 2^-8 (bf16), 2^-11 (fp16) of its own.  fp32: the operators' own errors, each within 2^-18 (norm and
# rotation) and some 2^-17 (attention over logits of ten and less), over four sites: 2^-14.
TOL = {"bf16": 20 ** 0.5 * 2.0 ** -8, "fp16": 20 ** 0.5 * 2.0 ** -11, "fp32": 2.0 ** -14}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rel(got, want):
    return float((got - want).square().mean().sqrt() / want.square().mean().sqrt())


def held(cache, pages, n):
    """The rows of a sequence's first n tokens in 64 bits."""
    t = torch.arange(n, device="cuda")
    slots = pages.long()[t // SIZE] * SIZE + t % SIZE
    t = torch.float32 if cache.k_scales is not None else None
    return (x.double() for x in dit.cache_read(cache, slots, dtype=t))


@pytest.mark.parametrize("dtype", list(TOL))
@pytest.mark.parametrize("fp8", [False, True])
def test_steps(dtype, fp8):
    table, weights, stand_ins, sites, caches, pages, freqs = setup(dtype, fp8)
    rnd = lambda v: v.to(table.dtype).double()
    steps, tol = 11, TOL[dtype]
    tokens = ((draw("gate", (B, steps), seed_for("decode", B), "fp32", "cuda") + 1) * 0.5 * V).long().clamp_(0, V - 1)
    Hq, Hk, d = HEADS
    for n in range(1, steps + 1):
        ids, lengths = tokens[:, n - 1].contiguous(), torch.full((B,), n, dtype=torch.int32, device="cuda")
        x, codes, scales = tk.decode_attending(ids, table, weights, stand_ins, sites, HEADS, caches, pages, lengths, freqs)
        angle = (n - 1) * freqs
        cos, sin = angle.cos().float().double(), angle.sin().float().double()
        for b in range(B):
            r = rnd(table[ids[b]].double())
            y = rnd(rms(r, weights[0].double()))
            for k, w in enumerate(weights[1:]):
                if k % 2 == 0:
                    wq, wk, a = sites[k // 2]
                    qkv = rnd(y.repeat(2)[:(Hq + 2 * Hk) * d].view(-1, d) * a.double())
                    q, own = (rnd(turned(rms(z, u.double()), cos, sin)) for z, u in ((qkv[:Hq], wq), (qkv[Hq:Hq + Hk], wk)))
                    kk, vv = held(caches[k // 2], pages[b], n)
                    # the new token's rows: E4M3 takes half a step, 2^-4, of an element
                    for got, want in ((kk[-1], own), (vv[-1], qkv[Hq + Hk:])):
                        assert rel(got, want) <= tol + (2.0 ** -4 if fp8 else 0), (n, b, k)
                    kk, vv = (z.repeat_interleave(Hq // Hk, 1) for z in (kk, vv))
                    s = torch.einsum("hd,thd->ht", q, kk) * d ** -0.5
                    u = rnd(torch.einsum("ht,thd->hd", s.softmax(-1), vv)).flatten()
                else:
                    u = rnd(y * stand_ins[k][b].double())
                r = rnd(r + u)
                y = rms(r, w.double())
                if k + 2 < len(weights):
                    y = rnd(y)
            assert rel(x[b].double(), r) <= tol, (n, b, rel(x[b].double(), r))
            # E4M3 of the norm: half a step of each code on top
            got, scale = codes[b].double(), scales[b].double()
            _, e = np.frexp((y / scale).abs().cpu().numpy())
            half = torch.from_numpy(np.ldexp(0.5, np.maximum(e - 4, -9))).cuda() * scale
            over = ((got * scale - y).abs() - half).clamp_min(0)
            assert float(over.square().mean().sqrt()) <= 2 * tol * float(y.square().mean().sqrt()), (n, b)
