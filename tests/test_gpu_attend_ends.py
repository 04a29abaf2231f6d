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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", [(3, 2, 16, 0), (3, 0, 16, 64), (0, 2, 16, 64), (3, 2, 1, 1), (1, 1, 1, 1)])
def test_caches_of_nothing(shape, fp8):
    """A cache without pages, heads or columns takes rows of that size, as the C entry points do."""
    t = torch.float8_e4m3fn if fp8 else torch.bfloat16
    cache = dit.KVCache.empty(*shape, dtype=t)
    pages, heads, size, D = shape
    x = torch.ones(2, heads, D, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([0, pages * size], device="cuda")
    dit.cache_write(cache, x, x, slots)
    k, v = dit.cache_read(cache, slots, dtype=torch.bfloat16)
    want = x.clone()
    want[1] = 0
    if pages == 0:
        want[0] = 0
    assert torch.equal(k, want) and torch.equal(v, want)
