"""Sizes of a paged cache at the ends of their ranges, without a GPU: what no kernel could count is refused on
the host.  Pointers are plain integers that are never dereferenced."""
import ctypes

import pytest
import torch

from diffusion_transformer_elementwise_gb300 import library
from diffusion_transformer_elementwise_gb300._attend import Cache
from diffusion_transformer_elementwise_gb300.build import build

SHAPE, NODEV = 2, 9
BF16, E4M3 = 0, 3
A = 1 << 24

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="the pointers are not real: a valid call would launch")


@pytest.fixture(scope="module")
def lib():
    build()
    return library()


def cache(pages, page_size, D=16, heads=1, format=BF16):
    n = heads * page_size * D
    return Cache(A, 2 * A, 3 * A, 4 * A, pages, heads, page_size, D, n, heads * page_size, format)


def heads(p):
    return (ctypes.c_int64 * 4)(p, 0, 16, 16)


@pytest.mark.parametrize("format", [BF16, E4M3])
def test_page_size(lib, format):
    """A page size of more than 31 bits, in a cache without pages, whose number of places is 0."""
    k, v = heads(5 * A), heads(6 * A)
    rows = [ctypes.addressof(k), ctypes.addressof(v), 3, 7 * A, 1, BF16, None]
    need = lib.dit_paged_attention_workspace_bytes(1, 1, 16)
    for size in (1 << 31, 1 << 32, 3 << 32, (1 << 32) + 1, 1 << 36):
        c = cache(0, size, format=format)
        at = ctypes.addressof(c)
        assert lib.dit_cache_read(at, *rows) == SHAPE and lib.dit_cache_write(at, *rows) == SHAPE, size
        assert lib.dit_paged_attention(ctypes.addressof(k), None, ctypes.addressof(v), at, 8 * A, 0, 0, 9 * A, 1, 1, 1.0,
                                       0, 0, BF16, 10 * A, need, None) == SHAPE, size
    for size in (1, (1 << 31) - 1):
        assert lib.dit_cache_read(ctypes.addressof(cache(0, size, format=format)), *rows) == NODEV


def test_page_table_strides(lib):
    """A page table is read alone: rows apart, or one row for all sequences."""
    q, out, c = heads(5 * A), heads(6 * A), cache(3, 16)
    need = lib.dit_paged_attention_workspace_bytes(1, 1, 16)
    call = lambda B, stride, width: lib.dit_paged_attention(
        ctypes.addressof(out), None, ctypes.addressof(q), ctypes.addressof(c), 8 * A, stride, width, 9 * A, B, 1, 1.0, 0,
        0, BF16, 10 * A, need, None)
    for B, stride, width in ((5, 0, 4), (5, 4, 4), (5, 7, 4), (1, 0, 4), (5, 0, 0)):
        assert call(B, stride, width) == NODEV, (B, stride, width)
    for B, stride, width in ((5, 1, 4), (5, 3, 4), (5, -4, 4), (1, -1, 4), (5, -1, 0)):
        assert call(B, stride, width) == SHAPE, (B, stride, width)


def test_attention_workspace(lib):
    """Room for the parts that the kernels for heads of D columns have, and no more: 160 CTAs and the warps of each, at most
    16, 12 or 8 of them, or 608 CTAs; two parts each, of up to 16 rows of D + 2 numbers."""
    need = lib.dit_paged_attention_workspace_bytes
    up = lambda n: -(-n // 256) * 256
    for D, parts in ((1, 160 * 17), (64, 160 * 17), (65, 160 * 13), (128, 160 * 13), (129, 160 * 9), (256, 160 * 9),
                     (257, 608), (512, 608)):
        for Hq, Hk, rows in ((1, 1, 1), (8, 2, 4), (16, 1, 16), (80, 2, 16)):
            assert need(Hq, Hk, D) == up(608 * 2 * 8) + up(parts * 2 * rows * (D + 2) * 4), (D, Hq, Hk)
