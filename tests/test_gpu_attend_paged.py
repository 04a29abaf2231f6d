"""Attention of one new token over a paged cache, against 64 bits
(tests/_attend_ref.py)."""
import math

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import check_attention, f64
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("paged", tag, *shape), dtype, "cuda")


class Setup:
    """Sequences of the given lengths in a cache whose every other place holds NaN."""

    def __init__(self, lengths, Hq, Hk, D, size, dtype="bf16", fp8=False, joined=False, rows=None):
        self.lengths, self.size, self.fp8 = lengths, size, fp8
        counts = [-(-max(0, n) // size) for n in lengths]
        width, total = max(1, max(counts, default=0)), sum(counts) + 2
        t = torch.uint8 if fp8 else T[dtype]
        lead = (total, 2) if joined else (2, total)
        kv = torch.full((*lead, Hk, size, D), 0x7F if fp8 else math.nan, dtype=t, device="cuda")
        sc = torch.full((*lead, Hk, size), math.nan, device="cuda")
        k, v = (kv[:, 0], kv[:, 1]) if joined else (kv[0], kv[1])
        ks, vs = (sc[:, 0], sc[:, 1]) if joined else (sc[0], sc[1])
        self.cache = dit.KVCache(k, v, *((ks, vs) if fp8 else ()))
        order = torch.randperm(total, generator=torch.Generator().manual_seed(total)).tolist()
        self.pages = torch.full((len(lengths), width), -1, dtype=torch.int32)
        at, slots = 0, []
        for b, c in enumerate(counts):
            mine = order[at:at + c]
            at += c
            self.pages[b, :c] = torch.tensor(mine, dtype=torch.int32)
            slots += [mine[i // size] * size + i % size for i in range(max(0, lengths[b]))]
        self.pages = self.pages.cuda()
        self.starts = [sum(max(0, x) for x in lengths[:b]) for b in range(len(lengths) + 1)]
        n = len(slots)
        x = rows if rows is not None else (act(n, Hk, D, tag="k", dtype=dtype), act(n, Hk, D, tag="v", dtype=dtype))
        slots = torch.tensor(slots, dtype=torch.int64, device="cuda")
        dit.cache_write(self.cache, x[0], x[1], slots)
        self.k, self.v = (f64(y) for y in dit.cache_read(self.cache, slots, dtype=torch.float32 if fp8 else None))
        self.q = act(len(lengths), Hq, D, tag="q", dtype=dtype)
        self.group, self.window = Hq // Hk, 0
        self.seen = None  # tokens of a sequence that count, where a page is missing

    def ids(self, dtype=torch.int32):
        return torch.tensor(self.lengths, dtype=dtype, device="cuda")

    def rows(self, which):
        def of(b, h):
            n = max(0, self.lengths[b])
            lo = max(0, n - self.window) if self.window else 0
            x = which[self.starts[b] + lo:self.starts[b] + n, h // self.group]
            return x if self.seen is None else x[self.seen(b, n)[lo:n]]
        return of

    def check(self, out, lse, scale=None, what=""):
        D = self.q.shape[-1]
        check_attention(out, lse, self.q, self.rows(self.k), self.rows(self.v), self.lengths,
                        D ** -0.5 if scale is None else float(torch.tensor(scale, dtype=torch.float32)),
                        self.fp8, what)

    def run(self, **kw):
        kw.setdefault("need_lse", True)
        return dit.paged_attention(self.q, self.cache, self.pages, self.ids(), window=self.window, **kw)


LENGTHS = [[1], [0], [0, 0, 3], [16], [17, 15, 1], [100, 0, 1, 33], [700, 5, 64, 128, 127], [5000],
           [300] * 9]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("lengths", LENGTHS, ids=str)
def test_lengths(lengths, dtype, fp8):
    s = Setup(lengths, 8, 2, 128, 16, dtype, fp8)
    s.check(*s.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D", [1, 8, 16, 33, 64, 72, 80, 96, 112, 128, 136, 192, 256, 264, 512])
def test_head_sizes(D, dtype, fp8):
    s = Setup([77, 300, 1], 4, 2, D, 16, dtype, fp8)
    s.check(*s.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 3), (2, 1), (5, 1), (8, 1), (9, 1), (16, 2), (17, 1), (40, 2),
                                   (64, 1)])
def test_groups(Hq, Hk, dtype, fp8):
    s = Setup([130, 9], Hq, Hk, 64, 16, dtype, fp8)
    s.check(*s.run())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [1, 3, 8, 13, 16, 32, 64, 100, 256])
def test_page_sizes(size, fp8):
    s = Setup([1, 129, 400, 31], 4, 1, 128, size, "bf16", fp8, joined=True)
    s.check(*s.run())


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("fp16", True), ("fp32", False)])
@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 64, 100, 1000, 2 ** 40])
def test_windows(window, dtype, fp8):
    s = Setup([5, 700, 0, 64, 101], 4, 2, 64, 16, dtype, fp8)
    s.window = window
    s.check(*s.run())


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("bf16", True), ("fp16", False), ("fp32", True)])
def test_pages_that_are_not_there(dtype, fp8):
    """Page numbers outside the cache leave their tokens out; a length is cut to the table's width."""
    s = Setup([70, 40, 33, 8], 4, 2, 64, 8, dtype, fp8)
    total = s.cache.pages
    s.pages[0, 2] = -1
    s.pages[0, 8] = total
    s.pages[1, 0] = 2 ** 31 - 1
    s.pages[3, 0] = -2 ** 31

    def seen(b, n):
        keep = torch.ones(n, dtype=torch.bool)
        for page in {0: (2, 8), 1: (0,), 3: (0,)}.get(b, ()):
            keep[8 * page:8 * page + 8] = False
        return keep.numpy()

    s.seen = seen
    out, lse = s.run()
    s.check(out, lse)
    assert (out[3] == 0).all() and (lse[3] == -math.inf).all()
    s.seen = None
    s.pages[:, 0] = s.pages[2, 0]
    long = torch.tensor([2 ** 40, -3, 33, -2 ** 62], device="cuda")
    got, lse = dit.paged_attention(s.q, s.cache, s.pages[:, :4], long, need_lse=True)
    want = dit.paged_attention(s.q, s.cache, s.pages[:, :4], torch.tensor([32, 0, 32, 0], device="cuda"))
    assert torch.equal(got, want[0]) and (got[1] == 0).all() and (got[3] == 0).all()


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("fp16", False), ("fp32", False), ("bf16", True), ("fp16", True)])
def test_sharp_and_flat(dtype, fp8):
    """Logits of hundreds (one token has all the weight), and none at all."""
    s = Setup([200, 31], 4, 2, 64, 16, dtype, fp8)
    for scale in (0.0, 20.0, -3.0, 1e-30):
        s.check(*s.run(scale=scale), scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_values_of_different_sizes(fp8):
    """Rows of values that differ by powers of ten: scales of E4M3 far from each other, and zeros."""
    n, Hk, D = 150, 2, 64
    k, v = act(n, Hk, D, tag="ka"), act(n, Hk, D, tag="va")
    size = torch.logspace(-12, 12, n, device="cuda")[torch.randperm(n, generator=torch.Generator().manual_seed(3)).cuda()]
    v = (v.float() * size[:, None, None]).bfloat16()
    v[5] = 0
    s = Setup([100, 50], 4, Hk, D, 16, "bf16", fp8, rows=(k, v))
    s.check(*s.run())


def test_nan_reaches_its_sequence_alone():
    s = Setup([40, 40, 40], 4, 2, 64, 16)
    clean, _ = s.run()
    s.cache.k[int(s.pages[1, 1]), 0, 3, 7] = math.nan
    s.cache.v[int(s.pages[2, 0]), 1, 3, 9] = math.inf
    out, lse = s.run()
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1, :2]).all() and torch.equal(out[1, 2:], clean[1, 2:])
    assert torch.isnan(lse[1, :2]).all() and torch.isfinite(lse[2]).all()
    assert torch.isinf(out[2, 2:, 9]).all() and torch.isfinite(out[2, :2]).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_views_and_outputs(fp8):
    """Queries as a view of the packed projection, an output within a larger tensor, 64-bit lengths, a
    page table that is a view."""
    s = Setup([50, 300, 7], 8, 2, 128, 16, "bf16", fp8)
    want, wl = s.run()
    packed = torch.full((3, 12, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    packed[:, :8] = s.q
    room = torch.full((3, 10, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    table = torch.full((3, s.pages.shape[1] + 5), 7, dtype=torch.int32, device="cuda")
    table[:, 2:2 + s.pages.shape[1]] = s.pages
    lse = torch.empty(3, 8, device="cuda")
    out, l2 = dit.paged_attention(packed[:, :8], s.cache, table[:, 2:2 + s.pages.shape[1]],
                                  s.ids(torch.int64), out=room[:, 1:9], lse=lse)
    assert torch.equal(out, want) and l2 is lse and torch.equal(lse, wl)
    assert (room[:, 0] == 9).all() and (room[:, 9] == 9).all()
    none, no = dit.paged_attention(s.q[:0], s.cache, s.pages[:0], s.ids()[:0])
    assert none.shape == (0, 8, 128) and no is None


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lengths,Hq,Hk,D", [([9000, 3, 0, 700], 8, 2, 128), ([20000], 4, 1, 64), ([33] * 50, 4, 4, 80)])
def test_workspace_and_repeats(lengths, Hq, Hk, D, fp8):
    s = Setup(lengths, Hq, Hk, D, 64, "bf16", fp8)
    want, wl = s.run()
    need = dit.library().dit_paged_attention_workspace_bytes(Hq, Hk, D)
    buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[4096:4096 + need]
    for fill in (0, 0xFF):
        ws.fill_(fill)
        for _ in range(2):
            got, gl = s.run(workspace=ws)
            assert torch.equal(got, want) and torch.equal(gl, wl)
        assert bool((buf[:4096] == 0xA5).all()) and bool((buf[4096 + need:] == 0xA5).all())


@pytest.mark.parametrize("dtype,fp8,Hq,Hk,D", [("bf16", False, 8, 2, 128), ("bf16", True, 8, 8, 64), ("fp32", False, 2, 1, 64),
                                              ("fp16", False, 4, 1, 256)])
def test_long(dtype, fp8, Hq, Hk, D):
    s = Setup([40000, 1, 9999, 0, 20], Hq, Hk, D, 64, dtype, fp8)
    s.check(*s.run())


def test_many_sequences():
    """More sequences than threads of a CTA, most of them empty or short."""
    lengths = [(7 * i) % 40 if i % 3 else 0 for i in range(700)]
    s = Setup(lengths, 2, 1, 64, 8)
    s.check(*s.run())


@pytest.mark.parametrize("fp8", [False, True])
def test_far_pages(fp8):
    """Offsets past 32 bits."""
    pages, size, D = 70, 16, 64
    room = torch.zeros(pages * 2 ** 26, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda").view(pages, 2 ** 26)
    k = room[:, :size * D].view(pages, 1, size, D)
    v = room[:, 2 ** 20:2 ** 20 + size * D].view(pages, 1, size, D)
    scales = [torch.zeros(pages, 1, size, device="cuda") for _ in "kv"] if fp8 else []
    cache = dit.KVCache(k, v, *scales)
    x, y = act(48, 1, D, tag="fk"), act(48, 1, D, tag="fv")
    table = torch.tensor([[69, 1, 66]], dtype=torch.int32, device="cuda")
    t = torch.arange(48, device="cuda")
    slots = table[0].long()[t // 16] * 16 + t % 16
    dit.cache_write(cache, x, y, slots)
    rk, rv = (f64(z) for z in dit.cache_read(cache, slots, dtype=torch.float32 if fp8 else None))
    q = act(1, 4, D, tag="fq")
    out, lse = dit.paged_attention(q, cache, table, torch.tensor([45], dtype=torch.int32, device="cuda"),
                                   need_lse=True)
    check_attention(out, lse, q, lambda b, h: rk[:45, 0], lambda b, h: rv[:45, 0], [45], D ** -0.5, fp8)


# Caches that the kernel for any alignment takes: odd heads, heads of more than 256 columns, views off 16 bytes.
ANY = [(5, 6, 1), (33, 5, 1), (99, 4, 2), (99, 8, 1), (99, 17, 1), (70, 40, 2), (129, 3, 3), (264, 9, 1), (320, 4, 1),
       (511, 40, 2)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D,Hq,Hk", ANY)
def test_any_alignment(D, Hq, Hk, dtype, fp8):
    """Groups in one block and in several, sequences of several parts, windows, empty rows."""
    s = Setup([3000, 9, 0, 130, 64], Hq, Hk, D, 13, dtype, fp8)
    out, lse = s.run()
    s.check(out, lse)
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()
    again, l2 = s.run()
    assert torch.equal(out, again) and torch.equal(lse, l2)
    for s.window in (1, 65, 2990):
        s.check(*s.run(), what=s.window)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hk", [(99, 4, 2), (99, 8, 1), (320, 2, 1)])
def test_any_alignment_missing_pages_and_sharp_logits(D, Hq, Hk, fp8):
    s = Setup([200, 40, 33, 8], Hq, Hk, D, 8, "bf16", fp8)
    for scale in (0.0, 20.0, -3.0, 1e-30):
        s.check(*s.run(scale=scale), scale=scale)
    s.pages[0, 2] = s.pages[0, 3] = -1
    s.pages[0, 20] = s.cache.pages
    s.pages[1, :] = -7
    gone = {0: (2, 3, 20), 1: range(5)}

    def seen(b, n):
        keep = torch.ones(n, dtype=torch.bool)
        for page in gone.get(b, ()):
            keep[8 * page:8 * page + 8] = False
        return keep.numpy()

    s.seen = seen
    out, lse = s.run()
    s.check(out, lse)
    assert (out[1] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("D", [99, 320])
def test_any_alignment_nan_reaches_its_sequence_alone(D):
    s = Setup([40, 100, 40], 4, 2, D, 16)
    clean, _ = s.run()
    s.cache.k[int(s.pages[1, 1]), 0, 3, 7] = math.nan
    s.cache.v[int(s.pages[2, 0]), 1, 3, 9] = math.inf
    out, lse = s.run()
    assert torch.equal(out[0], clean[0]) and torch.isnan(out[1, :2]).all() and torch.equal(out[1, 2:], clean[1, 2:])
    assert torch.isnan(lse[1, :2]).all() and torch.isfinite(lse[2]).all()
    assert torch.isinf(out[2, 2:, 9]).all() and torch.isfinite(out[2, :2]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("D,Hq,Hk", [(99, 8, 2), (320, 4, 1)])
def test_any_alignment_long(D, Hq, Hk, fp8):
    s = Setup([20000, 1, 9999, 0, 20], Hq, Hk, D, 64, "bf16", fp8)
    s.check(*s.run())
