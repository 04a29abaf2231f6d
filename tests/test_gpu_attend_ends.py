"""Arguments of the calls around attention at the ends of their ranges."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def test_windows_past_64_bits():
    """A window of more tokens than there are is none, whatever its size; a negative one is refused."""
    cache = dit.KVCache.empty(4, 1, 16, 64)
    x = draw("act", (64, 1, 64), seed_for("ends"), "bf16", "cuda")
    dit.cache_write(cache, x, -x, torch.arange(64, device="cuda"))
    args = (x[:2], cache, torch.tensor([[0, 1, 2, 3], [3, 2, 1, 0]], dtype=torch.int32, device="cuda"),
            torch.tensor([64, 40], device="cuda"))
    want, wl = dit.paged_attention(*args, need_lse=True)
    for window in (2 ** 63 - 1, 2 ** 63, 2 ** 64, 2 ** 64 + 3, 2 ** 200):
        out, lse = dit.paged_attention(*args, window=window, need_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, wl), window
    for window in (-1, -2 ** 63, -2 ** 64 + 3, -2 ** 200):
        with pytest.raises(dit.DitError):
            dit.paged_attention(*args, window=window)
