"""Page tables and batches of attention beside the usual ones: a row that all sequences share, and batches of more
sequences than a CTA has threads, some of them long."""
import numpy as np
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
