"""E4M3 caches that others have filled: attention where the rows' scales have either sign, against
64 bits.  A value is code * scale, whatever the scale's sign."""
import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import attend, f64, weight_error
from _gpu import ensure_built
from _token_ref import U, check_close, rounding
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def check(out, lse, q, k, v, scale, what):
    """out [D], lse of a head q [D] over rows k, v [tokens, D], all fp64.  With S = |scale| sum |q k| a logit is
    off by (D + 8) u S and the sum's cut 2^-22 S; the output by twice that and the exponential's 2^-21
    (its own and the sum's), by its weights' rounding, and by what fp16 cannot hold of a weight below 2^-14 of the
    largest: 2^-25 of the largest value for each of these few hundred tokens."""
    D = len(q)
    want, wl, size = attend(q, k, v, scale)
    S = float((np.abs(k) @ np.abs(q)).max() * abs(scale))
    logit = (D + 8) * U * S + 2.0 ** -22 * S
    tol = (2 * (logit + 2.0 ** -20) + weight_error(out.dtype, True)) * size + rounding(want, out.dtype)
    check_close(out, want, tol + len(k) * 2.0 ** -25 * np.abs(v).max(), what + " out")
    check_close(lse.reshape(()), np.float64(wl), logit + 2.0 ** -20 * (1 + abs(wl)), what + " lse")


@pytest.mark.parametrize("which", ["values", "keys", "both"])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D,Hq,Hk", [(64, 4, 2), (128, 8, 1), (256, 4, 1), (128, 24, 2), (33, 4, 2), (320, 3, 1)])
def test_signed_scales(D, Hq, Hk, dtype, which):
    lengths, size, pages = [200, 1, 77], 16, 40
    codes = [draw("act", (pages, Hk, size, D), seed_for("signed", n, D), "fp32", "cuda").clamp_(-4, 4)
             .to(torch.float8_e4m3fn) for n in "kv"]
    scales = []
    for n in "kv":
        s = draw("act", (pages, Hk, size), seed_for("signed", "s", n), "fp32", "cuda")
        s = s.abs() * 0.5 + 0.25
        if which in ("both", "keys" if n == "k" else "values"):
            s[(torch.arange(s.numel(), device="cuda") % 3 == 1).view(s.shape)] *= -1.0
        scales.append(s)
    cache = dit.KVCache(*codes, *scales)
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(7))[:3 * 13].view(3, 13).int().cuda()
    q = draw("act", (3, Hq, D), seed_for("signed", "q"), dtype, "cuda")
    out, lse = dit.paged_attention(q, cache, table, torch.tensor(lengths, device="cuda"),
                                   scale=0.25 * D ** -0.5, need_lse=True)
    k, v = (f64(c.float()) * f64(s)[..., None] for c, s in zip(codes, scales))
    scale = float(np.float32(0.25 * D ** -0.5))
    for b, n in enumerate(lengths):
        at = [(int(table[b, t // size]), t % size) for t in range(n)]
        for h in range(Hq):
            rows = [np.stack([x[p, h // (Hq // Hk), i] for p, i in at]) for x in (k, v)]
            check(out[b, h], lse[b, h], f64(q[b, h]), *rows, scale, f"{b} {h}")
    # what reads the rows back takes the same values
    slots = torch.tensor([p * size + i for p, i in at], device="cuda")
    got = dit.cache_read(cache, slots, dtype=torch.float32)
    for y, x in zip(got, (k, v)):
        check_close(y, np.stack([x[p, :, i] for p, i in at]), U * np.abs(np.stack([x[p, :, i] for p, i in at])), "read")
