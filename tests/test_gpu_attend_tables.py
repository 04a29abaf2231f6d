"""Page tables and batches of attention beside the usual ones: a row that all sequences share, and batches of more
sequences than a CTA has threads, some of them long."""
import numpy as np
import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import attend, f64, weight_error
from _gpu import ensure_built
from _token_ref import U, check_close, rounding
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("tables", tag, *shape), dtype, "cuda")


@pytest.mark.parametrize("D,fp8", [(64, False), (128, True), (33, False), (320, True)])
def test_one_row_for_all(D, fp8):
    """An expanded page table gives what its copy gives."""
    cache = dit.KVCache.empty(9, 2, 16, D, torch.float8_e4m3fn if fp8 else torch.bfloat16)
    x = act(9 * 16, 2, D, tag="rows")
    dit.cache_write(cache, x, -x, torch.arange(9 * 16, device="cuda"))
    q = act(5, 4, D, tag="q")
    lengths = torch.tensor([100, 0, 16, 1, 77], dtype=torch.int32, device="cuda")
    row = torch.tensor([[3, 8, 0, 1, 5, 7, 2]], dtype=torch.int32, device="cuda")
    out, lse = dit.paged_attention(q, cache, row.expand(5, -1), lengths, need_lse=True)
    want, wl = dit.paged_attention(q, cache, row.repeat(5, 1), lengths, need_lse=True)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("B", [700, 1200])
@pytest.mark.parametrize("dtype,fp8,D,Hq,Hk", [("bf16", False, 64, 2, 1), ("bf16", True, 64, 4, 2), ("fp32", False, 128, 2, 1),
                                              ("fp16", True, 128, 16, 1), ("bf16", False, 33, 2, 1)])
def test_many_sequences_some_of_them_long(dtype, fp8, D, Hq, Hk, B):
    """More sequences than threads, so that a part's place is looked for in several steps, and long ones among short
    and empty ones, so that CTAs begin within one, at its end and between two.  The long ones and their neighbours are held
    against 64 bits: tolerances as for any attention (the sum of D products in any order, the exponential, the weights'
    rounding; all rows are of like size, so what fp16 cannot hold is below 2^-37 a token)."""
    long = {3: 9000, 255: 4000, 256: 5000, 383: 2500, 511: 3000, 600: 7000, B - 2: 8000, B - 1: 33}
    lengths = [long.get(b, 0 if b % 5 == 0 else b * 7 % 90) for b in range(B)]
    size, pages = 32, 700
    cache = dit.KVCache.empty(pages, Hk, size, D, torch.float8_e4m3fn if fp8 else
                              {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}[dtype])
    slots = torch.arange(pages * size, device="cuda")
    x = act(pages * size, Hk, D, tag="k", dtype=dtype), act(pages * size, Hk, D, tag="v", dtype=dtype)
    dit.cache_write(cache, *x, slots)
    k, v = (f64(y) for y in dit.cache_read(cache, slots, dtype=torch.float32 if fp8 else None))
    width = 9000 // size + 1
    g = torch.Generator().manual_seed(B)
    table = torch.randint(0, pages, (B, width), generator=g, dtype=torch.int32)
    q = act(B, Hq, D, tag="q", dtype=dtype)
    out, lse = dit.paged_attention(q, cache, table.cuda(), torch.tensor(lengths, device="cuda"), need_lse=True)
    empty = torch.tensor([n == 0 for n in lengths], device="cuda")
    assert (out[empty] == 0).all() and (lse[empty] == -float("inf")).all() and torch.isfinite(lse[~empty]).all()
    for b in sorted({c for a in long for c in range(a - 2, a + 3) if 0 <= c < B}):
        n = lengths[b]
        if n == 0:
            continue
        t = np.arange(n)
        at = table[b].numpy()[t // size].astype(np.int64) * size + t % size
        for h in (0, Hq - 1):
            kk, vv, qq = k[at, h // (Hq // Hk)], v[at, h // (Hq // Hk)], f64(q[b, h])
            want, wl, sizes = attend(qq, kk, vv, D ** -0.5)
            S = float((np.abs(kk) @ np.abs(qq)).max() * D ** -0.5)
            logit = (D + 8) * U * S + 2.0 ** -22 * S
            tol = (2 * (logit + 2.0 ** -20) + weight_error(q.dtype, fp8)) * sizes + rounding(want, q.dtype)
            check_close(out[b, h], want, tol + n * 2.0 ** -37 * np.abs(vv).max(), f"out {b} {h}")
            check_close(lse[b, h].reshape(()), np.float64(wl), logit + 2.0 ** -20 * (1 + abs(wl)), f"lse {b} {h}")
