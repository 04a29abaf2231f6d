"""Infinities and the largest numbers among the values that attention reads, at equal logits: an infinite value makes its
column infinite (or NaN, over E4M3 where its code is 0 or another token's infinity has the other sign), and no other."""
import math

import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import f64
from _gpu import ensure_built
from _token_ref import check_close

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def outputs(cache, n, dtype, D, Hq):
    table = torch.arange(cache.pages, device="cuda").int()[None]
    q = torch.zeros(1, Hq, D, dtype=T[dtype], device="cuda")
    out, lse = dit.paged_attention(q, cache, table, torch.tensor([n], device="cuda"), need_lse=True)
    assert torch.allclose(lse, torch.full_like(lse, math.log(n)), rtol=1e-6, atol=0)
    return out[0]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 5, 40, 3000])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 12), (256, 1), (33, 2)])
def test_infinite_values(D, Hq, n, dtype):
    g = torch.Generator().manual_seed(D + n)
    pages = -(-n // 16)
    k, v = torch.zeros(pages, 1, 16, D), torch.randn(pages, 1, 16, D, generator=g)
    rows = v.transpose(1, 2).reshape(pages * 16, D)
    rows[n // 2, 3], rows[0, 5], rows[n - 1, 7] = math.inf, -math.inf, math.nan
    if n > 1:
        rows[0, 9], rows[n - 1, 9] = math.inf, -math.inf
    v = rows.view(pages, 16, 1, D).transpose(1, 2).contiguous()
    cache = dit.KVCache(k.to(T[dtype]).cuda(), v.to(T[dtype]).cuda())
    held = f64(rows[:n].to(T[dtype]))
    with np.errstate(invalid="ignore"):
        want = held.mean(0)
    # equal weights, exact in any type; the sum of n products in any order, the quotient, and the output's rounding
    tol = (n + 8) * 2.0 ** -23 * np.abs(np.where(np.isfinite(held), held, 0.0)).mean(0) + torch.finfo(T[dtype]).eps / 2 * np.abs(want)
    out = outputs(cache, n, dtype, D, Hq)
    for h in range(Hq):
        check_close(out[h], want, np.where(np.isfinite(want), tol, 0.0), f"{h}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 40, 3000])
@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 12), (256, 1), (33, 2)])
@pytest.mark.parametrize("scale", [math.inf, -math.inf, math.nan, 0.0, -0.0, 1e-44, 2.0 ** -126, 2.0 ** -100])
def test_scales_at_the_ends(scale, D, Hq, n, dtype):
    """One token's scale at an end of fp32's range beside ordinary ones (of 1, and where n is 1 none)."""
    g = torch.Generator().manual_seed(D + n)
    pages = -(-n // 16)
    kc = torch.zeros(pages, 1, 16, D).to(torch.float8_e4m3fn)
    vc = torch.randint(-4, 5, (pages, 1, 16, D), generator=g).float().to(torch.float8_e4m3fn)
    ks, vs = torch.ones(pages, 1, 16), torch.ones(pages, 1, 16)
    at = n // 2
    vs[at // 16, 0, at % 16] = scale
    cache = dit.KVCache(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda())
    codes = f64(vc.float().transpose(1, 2).reshape(pages * 16, D)[:n])
    with np.errstate(invalid="ignore"):
        held = codes * f64(vs.transpose(1, 2).reshape(pages * 16, 1)[:n])
        want = held.mean(0)
    # as above, the weights' rounding to fp16 (half a step) and the smallest numbers of fp32 and of the output's type
    size = np.abs(np.where(np.isfinite(held), held, 0.0)).mean(0)
    tol = ((n + 8) * 2.0 ** -23 + 2.0 ** -11) * size + torch.finfo(T[dtype]).eps / 2 * np.abs(want)
    tol = tol + (2.0 ** -24 if dtype == "fp16" else 2.0 ** -110)
    out = outputs(cache, n, dtype, D, Hq)
    for h in range(Hq):
        check_close(out[h], want, np.where(np.isfinite(want), tol, 0.0), f"{h}")


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 12), (33, 2)])
@pytest.mark.parametrize("n", [1, 40])
def test_largest_scales(D, Hq, n):
    """Values up to 2^127: the weights' units stay within fp32's range, and so does the output."""
    vc = torch.zeros(3, 1, 16, D)
    vc[..., ::2] = 1.0
    ks, vs = torch.ones(3, 1, 16), torch.full((3, 1, 16), 1.75 * 2.0 ** 127)
    cache = dit.KVCache(torch.zeros(3, 1, 16, D).to(torch.float8_e4m3fn).cuda(), vc.to(torch.float8_e4m3fn).cuda(),
                        ks.cuda(), (vs / n).cuda())
    out = outputs(cache, n, "bf16", D, Hq)
    assert (out[:, 1::2] == 0).all()
    got = f64(out[:, ::2])
    want = float(vs[0, 0, 0]) / n
    assert (np.abs(got / want - 1.0) <= 2.0 ** -8 + 2.0 ** -11).all()
