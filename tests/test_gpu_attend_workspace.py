"""Attention writes nothing outside the workspace that its size function asks for: every kernel's heads, between guards."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D", [32, 64, 80, 128, 192, 256, 272, 512, 99, 300])
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (8, 1), (24, 1)])
def test_guards(D, Hq, Hk, dtype, fp8):
    size, pages = 16, 700
    cache = dit.KVCache.empty(pages, Hk, size, D, torch.float8_e4m3fn if fp8 else T[dtype])
    x = draw("act", (pages * size, Hk, D), seed_for("guards", D, Hk), dtype, "cuda")
    dit.cache_write(cache, x, -x, torch.arange(pages * size, device="cuda"))
    table = torch.arange(pages, device="cuda").int()[None].expand(3, -1)
    # every segment is split, over warps and over CTAs
    lengths = torch.tensor([pages * size, 5000, 3001], device="cuda")
    q = draw("act", (3, Hq, D), seed_for("guards", "q"), dtype, "cuda")
    want, wl = dit.paged_attention(q, cache, table, lengths, need_lse=True)
    need = dit.library().dit_paged_attention_workspace_bytes(Hq, Hk, D)
    room = torch.full((need + (8 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[4 << 20:(4 << 20) + need]
    for fill in (0, 0xFF):
        ws.fill_(fill)
        out, lse = dit.paged_attention(q, cache, table, lengths, need_lse=True, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, wl)
    assert bool((room[:4 << 20] == 0xA5).all()) and bool((room[(4 << 20) + need:] == 0xA5).all())
