"""The embedding lookup and its gradient on the GPU: the lookup bit for bit,
the gradient against the 64-bit sums of tests/_token_ref.py."""
import numpy as np
import pytest
import torch

import _token_ref as ref
import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built, guarded, offset_copy
from diffusion_transformer_elementwise_gb300.synth import seed_for

pytestmark = pytest.mark.gpu
IDS = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
dtypes = pytest.mark.parametrize("dtype", ref.TYPES, ids=IDS.get)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(shape, dtype, *seed):
    rng = np.random.default_rng(seed_for(*seed))
    return torch.from_numpy(rng.standard_normal(shape)).to(dtype)


def tokens(n, V, kind, *seed):
    """ids of a batch: text-like frequencies, all alike, all different, with
    ids outside the table."""
    rng = np.random.default_rng(seed_for("ids", n, V, kind, *seed))
    if kind == "same":
        ids = np.full(n, V - 1)
    elif kind == "distinct":
        ids = rng.permutation(max(n, V))[:n] % V
    else:
        ids = (np.exp(rng.uniform(size=n) * np.log(V)) - 1).astype(np.int64) % V
    if kind == "padded":
        ids[rng.uniform(size=n) < 0.3] = -1
        ids[:1] = V
        ids[-1:] = np.iinfo(np.int64).min
    return torch.from_numpy(ids.astype(np.int64))


def bits(t):
    return t.cpu().flatten().clone().view(torch.uint8) if t.numel() else torch.empty(0)


def looked_up(ids, table, scale):
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table[ids.clamp(0, table.shape[0] - 1)].float() * float(np.float32(scale))
    return torch.where(ok[..., None], rows, torch.zeros(())).to(table.dtype)


@pytest.mark.parametrize("D", [1, 7, 8, 64, 129, 2048, 3077, 4096, 8200])
@pytest.mark.parametrize("n", [1, 5, 130])
@dtypes
def test_lookup(dtype, n, D):
    V = 37
    table, ids = make((V, D), dtype, "table", D), tokens(n, V, "padded")
    out, fresh = guarded((n, D), dtype, "cuda")
    got = dit.embedding(ids.cuda(), table.cuda(), 45.25, out=out)
    torch.cuda.synchronize()
    assert got is out and fresh()
    assert torch.equal(bits(out), bits(looked_up(ids, table, 45.25)))
    ids32 = torch.where(ids < -1, torch.tensor(-7), ids).to(torch.int32)
    out2 = dit.embedding(ids32.cuda(), table.cuda(), 45.25)
    assert torch.equal(bits(out), bits(out2))


@dtypes
def test_lookup_shapes_offsets_and_values(dtype):
    table = make((50, 96), dtype, "shape")
    table[3, 5], table[3, 6], table[4, 0] = float("inf"), float("nan"), -0.0
    ids = tokens(12, 50, "text").view(3, 4)
    ids[0, 0], ids[2, 1] = 3, 4
    out = dit.embedding(ids.cuda(), table.cuda())
    assert out.shape == (3, 4, 96)
    torch.testing.assert_close(out.cpu(), table[ids], rtol=0, atol=0, equal_nan=True)
    # the same from tensors off a 16-byte boundary
    t1, o1 = offset_copy(table, 1), offset_copy(torch.zeros((3, 4, 96), dtype=dtype), 3)
    dit.embedding(ids.cuda(), t1, out=o1)
    torch.testing.assert_close(o1.cpu(), table[ids], rtol=0, atol=0, equal_nan=True)
    assert dit.embedding(ids.cuda()[:0], table.cuda()).shape == (0, 4, 96)
    empty = dit.embedding(ids.cuda(), table.cuda()[:0])
    assert empty.shape == (3, 4, 96) and not empty.any()


@pytest.mark.parametrize("kind", ["text", "same", "distinct", "padded"])
@pytest.mark.parametrize("n,V,D", [(1, 1, 8), (1, 1000, 64), (31, 40, 7), (32, 40, 8), (33, 3, 129),
                                   (126, 3000, 256), (255, 30, 4100), (256, 500, 33),
                                   (257, 500, 33), (1000, 50, 1), (4096, 700, 24),
                                   (4097, 5000, 72), (6000, 130000, 8), (9000, 17, 40),
                                   (300, 300, 4100)])
@dtypes
def test_gradient(dtype, n, V, D, kind):
    ids, g = tokens(n, V, kind), make((n, D), dtype, "grad", n, D)
    out, fresh = guarded((V, D), dtype, "cuda")
    got = dit.embedding_backward(g.cuda(), ids.cuda(), V, 3.3, out=out)
    again = dit.embedding_backward(g.cuda(), ids.cuda(), V, 3.3)
    torch.cuda.synchronize()
    assert got is out and fresh()
    ref.check_embedding_grad(out, g, ids, V, 3.3, f"{kind} {n} {V} {D}")
    assert torch.equal(bits(out), bits(again))


@pytest.mark.parametrize("lengths", [
    [32, 32, 64, 32, 96, 32], [31, 33, 32, 65, 63, 64, 1, 97, 95, 128], [1, 64, 31, 64, 64, 200],
    [20, 44, 64, 20, 45, 63], [30, 500], [300, 1, 31, 2], list(range(1, 70)),
    list(range(69, 0, -1))], ids=lambda v: "-".join(map(str, v[:6])))
@pytest.mark.parametrize("D", [8, 77, 512])
@dtypes
def test_gradient_of_runs(dtype, D, lengths):
    """Ids that stand a given number of times: runs that start, end and fill
    blocks of 32 sorted tokens in every way."""
    V, out_of_range = 2 * len(lengths) + 1, 37
    ids = torch.cat([torch.full((n,), 2 * k + 1) for k, n in enumerate(lengths)]
                    + [torch.full((out_of_range,), -1)])
    ids = torch.cat([ids, torch.full((max(0, 257 - ids.numel()),), V)])
    order = np.random.default_rng(seed_for("runs", *lengths)).permutation(ids.numel())
    ids, g = ids[torch.from_numpy(order)].contiguous(), make((ids.numel(), D), dtype, "runs", D)
    out, fresh = guarded((V, D), dtype, "cuda")
    dit.embedding_backward(g.cuda(), ids.cuda(), V, 0.7, out=out)
    torch.cuda.synchronize()
    assert fresh()
    ref.check_embedding_grad(out, g, ids, V, 0.7)


@pytest.mark.parametrize("n", [70_000, 300_000])
def test_gradient_of_many_tokens(n):
    """Several rounds of every warp of the sort, long runs, int32 ids, an id
    range of three digits."""
    V, D = 300_000, 8
    ids, g = tokens(n, V, "padded"), make((n, D), torch.bfloat16, "many", n)
    ids32 = ids.clamp(-1, V).to(torch.int32)
    out = dit.embedding_backward(g.cuda(), ids32.cuda(), V)
    torch.cuda.synchronize()
    ref.check_embedding_grad(out, g, ids, V, 1.0)


@dtypes
def test_gradient_off_a_16_byte_boundary(dtype):
    n, V, D = 200, 90, 104
    ids, g = tokens(n, V, "text"), make((n, D), dtype, "off")
    out = offset_copy(torch.full((V, D), 5.0, dtype=dtype), 3)
    dit.embedding_backward(offset_copy(g, 1), ids.cuda(), V, out=out)
    torch.cuda.synchronize()
    ref.check_embedding_grad(out, g, ids, V, 1.0)


def test_gradient_edges():
    g, ids = torch.ones((4, 16), device="cuda"), torch.full((4,), -1, device="cuda")
    out = dit.embedding_backward(g, ids, 5, out=torch.full((5, 16), 9.0, device="cuda"))
    assert not out.any()                                     # nothing but padding
    out = dit.embedding_backward(g[:0], ids[:0], 5, out=torch.full((5, 16), 9.0, device="cuda"))
    assert not out.any()                                     # no tokens
    assert dit.embedding_backward(g, ids, 0).shape == (0, 16)
    # NaN and infinity stay with their ids
    g[1, 2], g[2, 3] = float("nan"), float("inf")
    out = dit.embedding_backward(g, torch.tensor([0, 1, 2, 3], device="cuda"), 5).cpu()
    assert torch.isnan(out[1, 2]) and torch.isinf(out[2, 3]) and torch.isfinite(out).sum() == 78


def test_refusals():
    g, ids = torch.ones((4, 16), device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(TypeError):
        dit.embedding(ids.float(), g)
    with pytest.raises(TypeError):
        dit.embedding(ids.to(torch.int16), g)
    with pytest.raises(ValueError):
        dit.embedding(ids, g[0])
    with pytest.raises(ValueError):
        dit.embedding(ids, g, out=torch.empty((4, 8), device="cuda"))
    with pytest.raises(ValueError):
        dit.embedding_backward(g, ids[:3], 5)
    with pytest.raises(ValueError):
        dit.embedding_backward(g, ids, 5, out=torch.empty((4, 16), device="cuda"))
    with pytest.raises(dit.DitError):
        dit.embedding(ids, g, float("nan"))
    with pytest.raises(dit.DitError):
        dit.embedding_backward(g, ids, 4, out=g)
    with pytest.raises(dit.DitError):
        dit.embedding_backward(torch.ones((300, 16), device="cuda"),
                               torch.zeros(300, dtype=torch.int64, device="cuda"), 5,
                               workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_streams_and_graphs():
    V, D = 500, 256
    table = make((V, D), torch.bfloat16, "t").cuda()
    ids = [tokens(700, V, k).cuda() for k in ("text", "padded", "same")]
    now = ids[0].clone()

    def step(stream=None):
        o = dit.embedding(now, table, 2.0, stream=stream)
        return [o, dit.embedding_backward(o, now, V, 2.0, stream=stream)]

    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = step(side)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in ids:
        now.copy_(k)
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(outs, want))


def test_offsets_past_32_bits():
    """A table whose last rows lie past 2^32 bytes, and its gradient."""
    V, D = 600_000, 4096
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    tail = make((2, D), torch.bfloat16, "far")
    table[-2:] = tail.cuda()
    ids = torch.tensor([V - 1, 0, V - 2], device="cuda")
    out = dit.embedding(ids, table)
    assert torch.equal(out.cpu(), torch.stack([tail[1], torch.zeros(D, dtype=torch.bfloat16), tail[0]]))
    dit.embedding_backward(out, ids, V, out=table.fill_(1.0))
    torch.cuda.synchronize()
    assert torch.equal(table[-2:].cpu(), tail) and not table[:-2].any()


@pytest.mark.parametrize("D", [8_000_000, 8_000_003])
def test_gradient_of_rows_past_32_bits(D):
    """Tokens whose rows lie past 2^32 bytes, through the sort, runs of two
    and of more segments: rows of zeros and ones, whose sums are exact."""
    n, V = 300, 4
    t = torch.arange(n)
    ids = torch.where(t % 3 > 0, 0, torch.where(t % 2 > 0, 2, 3))
    value = (t * 7 % 5 < 2).to(torch.bfloat16)
    g = value.cuda()[:, None].expand(n, D).contiguous()
    out = dit.embedding_backward(g, ids.cuda(), V)
    want = torch.zeros(V).index_add_(0, ids, value.float())
    assert want.max() <= 256
    assert bool((out == want.to(torch.bfloat16).cuda()[:, None]).all())
