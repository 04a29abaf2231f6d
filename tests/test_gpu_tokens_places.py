"""Decoding steps of a padded batch (tokens.py): rows of empty sequences, and of sequences longer than their page tables,
write to no cache, whatever their rows of the page table hold."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300 import tokens as tk

pytestmark = pytest.mark.gpu
HEADS = (4, 2, 32)
V, D, SIZE, B = 50, 128, 4, 4


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_without_a_place(fp8, captured):
    ids, table, weights, stand_ins = tk.make_inputs(B, V, D, blocks=1)
    sites = tk.make_attention(D, HEADS, 1)
    # row 0 is idle and its page table full of zeros, row 1 too long for its table, row 2 without a page for its token
    pages = torch.tensor([[0, 0], [0, 1], [2, -1], [3, 4]], dtype=torch.int32, device="cuda")
    lengths = torch.tensor([0, 9, 6, 5], dtype=torch.int32, device="cuda")
    cache = dit.KVCache.empty(6, HEADS[1], SIZE, HEADS[2], torch.float8_e4m3fn if fp8 else torch.bfloat16)
    held = [cache.k, cache.v] + ([cache.k_scales, cache.v_scales] if fp8 else [])
    for n, t in enumerate(held):
        t.copy_(torch.linspace(-1, 1, t.numel(), device="cuda").view(t.shape) + n)
    before = [t.clone() for t in held]
    freqs = dit.rotary_frequencies(HEADS[2] // 2)
    run = lambda: tk.decode_attending(ids, table, weights, stand_ins, sites, HEADS, [cache], pages, lengths, freqs)
    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        for t, b in zip(held, before):
            t.copy_(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            x, codes, scales = run()
        graph.replay()
    else:
        x, codes, scales = run()
    assert torch.isfinite(x.float()).all() and torch.isfinite(codes.float()).all() and torch.isfinite(scales).all()
    for now, was in zip(held, before):
        now, was = (t.view(torch.uint8) if t.dtype is torch.float8_e4m3fn else t for t in (now, was))
        changed = (now != was).flatten(3).any(-1) if now.dim() == 4 else now != was
        # token 4 of row 3 lies at the first place of page 4, in every head; nothing else has changed
        assert changed[4, :, 0].all()
        changed[4, :, 0] = False
        assert not changed.any()
