"""The cache's places of new tokens (tokens.places): of tokens that have none, because their sequence is empty, longer than
its page table, or without a page there, no other token's."""
import torch

from diffusion_transformer_elementwise_gb300 import tokens as tk


def test_places():
    pages = torch.tensor([[0, 1], [5, 3], [4, -1]], dtype=torch.int32)
    for dtype in (torch.int32, torch.int64):
        at = lambda *p: tk.places(pages, torch.tensor(p, dtype=dtype), 4)
        assert at(0, 3, 1).tolist() == [0, 23, 17]
        assert at(7, 4, 3).tolist() == [7, 12, 19]
        assert at(-1, -1, -1).tolist() == [-1, -1, -1]      # empty sequences
        assert at(8, 9, 8).tolist() == [-1, -1, -1]         # behind the table
        assert at(2 ** 30, -7, 5).tolist() == [-1, -1, -1]  # far away; before the start; no page there
    assert at(0, 0, 0).dtype == torch.int64
    assert tk.places(pages[:, :0], torch.tensor([0, -1, 3]), 4).tolist() == [-1, -1, -1]
    assert tk.places(pages[:0], torch.tensor([], dtype=torch.int64), 4).tolist() == []
