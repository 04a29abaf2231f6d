"""The paged cache: rows written in their dtype or in E4M3, and read back,
against 64 bits (tests/_attend_ref.py)."""
import math

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import check_rows_e4m3
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("cache", tag, *shape), dtype, "cuda")


def filled(pages, heads, size, D, dtype, fp8, joined=False):
    """A cache that holds a known pattern everywhere, and copies of its tensors."""
    t = torch.uint8 if fp8 else T[dtype]
    if joined:  # keys and values of a page side by side in one allocation
        kv = torch.full((pages, 2, heads, size, D), 77, dtype=t, device="cuda")
        k, v = kv[:, 0], kv[:, 1]
        sc = torch.full((pages, 2, heads, size), 5.0, device="cuda")
        ks, vs = sc[:, 0], sc[:, 1]
    else:
        k, v = (torch.full((pages, heads, size, D), 77, dtype=t, device="cuda") for _ in "kv")
        ks, vs = (torch.full((pages, heads, size), 5.0, device="cuda") for _ in "kv")
    return dit.KVCache(k, v, *((ks, vs) if fp8 else ()))


def by_slot(x):
    """[pages, heads, size, ...] as [slots, heads, ...]."""
    return x.transpose(1, 2).reshape(x.shape[0] * x.shape[2], x.shape[1], *x.shape[3:])


CASES = [  # tokens, heads, D, page size, pages
    (1, 1, 1, 1, 1), (1, 8, 128, 16, 3), (64, 8, 128, 16, 9), (130, 2, 80, 13, 17), (33, 3, 96, 1, 40),
    (517, 4, 64, 64, 12), (100, 1, 256, 8, 20), (50, 2, 33, 16, 6), (9, 1, 1024, 4, 3), (70, 2, 200, 16, 8),
    (3000, 2, 128, 128, 30)]


@pytest.mark.parametrize("kind", ["plain", "packed", "joined", "shifted"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("tokens,heads,D,size,pages", CASES)
def test_write_and_read(tokens, heads, D, size, pages, dtype, fp8, kind):
    x = act(tokens, 3 * heads, D, tag="x", dtype=dtype)
    k, v = x[:, :heads], x[:, 2 * heads:]
    if kind == "plain":
        k, v = k.contiguous(), v.contiguous()
    elif kind == "shifted":
        flat = torch.empty(tokens * heads * D + 1, dtype=T[dtype], device="cuda")
        flat[1:] = k.reshape(-1)
        k = flat[1:].view(tokens, heads, D)
    cache = filled(pages, heads, size, D, dtype, fp8, kind == "joined")
    order = torch.randperm(pages * size, generator=torch.Generator().manual_seed(tokens)).cuda()
    slots = order[:tokens].clone()
    if tokens > 4:  # some are not written
        slots[1], slots[2], slots[-1] = -1, pages * size, -2 ** 40
    inside = (slots >= 0) & (slots < pages * size)
    before = [t.clone() for t in (cache.k, cache.v)]
    dit.cache_write(cache, k, v, slots)
    if tokens > 4:
        slots[-1] = -5
    dit.cache_write(cache, k, v, slots.to(torch.int32))  # the same again, by 32-bit slots
    torch.cuda.synchronize()
    at = slots[inside]
    for now, was, scales, rows in ((cache.k, before[0], cache.k_scales, k), (cache.v, before[1], cache.v_scales, v)):
        got = by_slot(now)
        if fp8:
            check_rows_e4m3(got[at], by_slot(scales)[at], rows[inside], f"{kind}")
            rest = by_slot(scales).clone()
            rest[at] = 5.0
            assert (rest == 5.0).all()
        else:
            assert torch.equal(got[at], rows[inside])
        keep = got.clone()
        keep[at] = 77
        assert torch.equal(keep, by_slot(was))  # nothing else has changed
    rk, rv = dit.cache_read(cache, slots, dtype=T[dtype])
    for got, now, scales in ((rk, cache.k, cache.k_scales), (rv, cache.v, cache.v_scales)):
        assert got.dtype is T[dtype] and (got[~inside] == 0).all()
        want = by_slot(now)[at]
        if fp8:
            want = (want.view(torch.float8_e4m3fn).float() * by_slot(scales)[at][..., None]).to(T[dtype])
        assert torch.equal(got[inside], want)


@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D", [128, 33])
def test_rows_out_of_the_ordinary(D, dtype):
    """Zeros, subnormals, the largest values, infinities, NaN and exact ties."""
    big = torch.finfo(T[dtype]).max
    tiny = torch.finfo(T[dtype]).smallest_normal
    x = act(10, 1, D, tag="odd", dtype="fp32").clamp_(-2, 2)
    x[0] = 0
    x[1] *= tiny / 4
    x[2] = x[2] / x[2].abs().max() * big
    x[3, 0, 5] = math.inf
    x[4, 0, 7] = math.nan
    x[5, 0, 1:] = 0
    x[6] *= 1e-30 if dtype != "fp16" else 1e-6
    x[7, 0] = torch.arange(D, device="cuda") % 32 + 0.5
    x[7, 0, 0] = 448.0
    x[8] = -0.0
    x[9] *= 1e-38 if dtype != "fp16" else 1e-7
    x = x.to(T[dtype])
    cache = filled(2, 1, 16, D, dtype, True)
    slots = torch.arange(10, device="cuda") + 3
    dit.cache_write(cache, x, x, slots)
    check_rows_e4m3(by_slot(cache.k)[slots], by_slot(cache.k_scales)[slots], x)
    assert torch.equal(cache.k, cache.v)
    rk, _ = dit.cache_read(cache, slots, dtype=T[dtype])
    assert torch.isnan(rk[3:5]).all() and (rk[0] == 0).all() and torch.isfinite(rk[2]).all()


def test_other_types_into_e4m3():
    """An E4M3 cache takes and gives rows of any type."""
    x = act(20, 2, 64, tag="any", dtype="fp32")
    cache = dit.KVCache.empty(2, 2, 16, 64, dtype=torch.float8_e4m3fn)
    slots = torch.arange(20, device="cuda")
    dit.cache_write(cache, x, x * 2, slots)
    got = {t: dit.cache_read(cache, slots, dtype=t) for t in T.values()}
    for t in T.values():
        assert torch.equal(got[t][1], got[torch.float32][1].to(t))
    assert dit.cache_read(cache, slots)[0].dtype is torch.bfloat16
    assert dit.cache_read(cache, slots[:0])[0].shape == (0, 2, 64)


def test_read_outputs_may_be_views():
    x = act(40, 2, 128, tag="view")
    cache = dit.KVCache.empty(5, 2, 8, 128)
    slots = torch.arange(40, device="cuda").flip(0).contiguous()
    dit.cache_write(cache, x, -x, slots)
    room = torch.full((40, 6, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    dit.cache_read(cache, slots, k=room[:, :2], v=room[:, 4:])
    assert torch.equal(room[:, :2], x) and torch.equal(room[:, 4:], -x) and (room[:, 2:4] == 3).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(fp8):
    """Offsets past 32 bits: pages a stride of 2^26 elements apart (2^32 and more in all)."""
    pages, heads, size, D = 70, 1, 4, 64
    t = torch.uint8 if fp8 else torch.bfloat16
    room = torch.zeros(pages * 2 ** 26, dtype=t, device="cuda")
    kv = room.view(pages, 2 ** 26)
    k = kv[:, :size * D].view(pages, heads, size, D)
    v = kv[:, 2 ** 20:2 ** 20 + size * D].view(pages, heads, size, D)
    scales = [torch.zeros(pages, heads, size, device="cuda") for _ in "kv"] if fp8 else []
    cache = dit.KVCache(k, v, *scales)
    x = act(6, 1, D, tag="far")
    slots = torch.tensor([0, 1, 65 * 4, 69 * 4 + 3, 33 * 4 + 2, 68 * 4], device="cuda")
    dit.cache_write(cache, x, 2 * x, slots)
    rk, rv = dit.cache_read(cache, slots, dtype=torch.bfloat16)
    if fp8:
        assert torch.allclose(rk.float(), x.float(), atol=0.07 * float(x.abs().max()))
        assert torch.equal(rv, 2 * rk)
    else:
        assert torch.equal(rk, x) and torch.equal(rv, 2 * x)
    assert int((kv[:, :2 ** 19] != 0).sum()) <= 6 * D
