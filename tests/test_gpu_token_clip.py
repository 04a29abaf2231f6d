"""The global gradient norm and clipping on the GPU, against 64-bit sums."""
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


def make(n, dtype, *seed, std=1.0):
    rng = np.random.default_rng(seed_for("clip", n, *seed))
    return torch.from_numpy(rng.standard_normal(n) * std).to(dtype)


def bits(t):
    return t.cpu().flatten().clone().view(torch.uint8) if t.numel() else torch.empty(0)


@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [0, 5, 0], [16384], [16385, 16383], [100_003, 3],
                                   [1] * 100, list(range(0, 2100))])
@dtypes
def test_clip(dtype, sizes):
    gs = [make(n, dtype, i) for i, n in enumerate(sizes)]
    gd = [g.cuda() for g in gs]
    total = float(np.sqrt(sum((ref.f64(g) ** 2).sum() for g in gs)))
    for m in (0.5 * total, 2.0 * total, 0.0):
        outs, norm = dit.clip_grads(gd, m)
        only = dit.grad_norm(gd)
        torch.cuda.synchronize()
        ref.check_clip(norm, outs, gs, m, what=f"max {m}")
        assert torch.equal(bits(norm), bits(only)) and norm.shape == ()
        if m > total:
            assert all(torch.equal(bits(o), bits(g)) for o, g in zip(outs, gs))
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(gd, gs))


def test_mixed_types_offsets_in_place_and_lists():
    gs = [make(n, ref.TYPES[i % 3], "mixed", i, std=10.0 ** (i % 4 - 2))
          for i, n in enumerate([5, 40_000, 17, 16_384 * 3 + 5, 1, 1000, 0, 333])]
    gd = [offset_copy(g, i % 4) for i, g in enumerate(gs)]
    pairs = [guarded(tuple(g.shape), g.dtype, "cuda", pad=61 + i) for i, g in enumerate(gs)]
    outs = [p[0] for p in pairs]
    lst = dit.TensorList(gd, out=outs)
    for _ in range(2):
        got, norm = dit.clip_grads(lst, 1.0)
        torch.cuda.synchronize()
        assert got == lst.out and all(a is b for a, b in zip(got, outs))
        ref.check_clip(norm, outs, gs, 1.0)
    assert all(p[1]() for p in pairs if p[0].numel())
    keep = [o.clone() for o in outs]
    back, n2 = dit.clip_grads(gd, 1.0, out=gd)
    torch.cuda.synchronize()
    assert all(a is b for a, b in zip(back, gd)) and torch.equal(bits(norm), bits(n2))
    for a, b in zip(gd, keep):
        assert torch.equal(bits(a), bits(b))


@pytest.mark.parametrize("std", [2.0 ** 66, 2.0 ** -75, 2.0 ** -120, 0.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=IDS.get)
def test_squares_outside_fp32(dtype, std):
    """Squares that overflow fp32, or fall below its normal range."""
    gs = [make(n, dtype, "range", std=std) for n in (3, 20_001, 16)]
    outs, norm = dit.clip_grads([g.cuda() for g in gs], 1.0)
    torch.cuda.synchronize()
    ref.check_clip(norm, outs, gs, 1.0)


@dtypes
def test_not_finite(dtype):
    g = make(5000, dtype, "nan")
    for v in (float("nan"), float("inf")):
        for at in (0, 1, 4999, 2500):
            h = g.clone()
            h[at] = v
            (out,), norm = dit.clip_grads([h.cuda()], 1.0)
            o, n = out.cpu().float(), float(norm)
            if v != v:
                assert n != n and bool(torch.isnan(o).all())
            else:
                assert n == v and torch.isnan(o[at]) and int((o == 0).sum()) == 4999


def test_refusals():
    g = [torch.ones(8, device="cuda"), torch.ones(9, device="cuda")]
    with pytest.raises(ValueError):
        dit.clip_grads(g, 1.0, out=g[:1])
    with pytest.raises(ValueError):
        dit.clip_grads(g, 1.0, out=[g[1], g[0]])
    with pytest.raises(ValueError):
        dit.grad_norm([])
    with pytest.raises(ValueError):
        dit.clip_grads(dit.TensorList(g), 1.0)
    with pytest.raises(ValueError):
        dit.clip_grads(dit.TensorList(g, g), 1.0, out=g)
    with pytest.raises(TypeError):
        dit.grad_norm([g[0].double()])
    with pytest.raises(TypeError):
        dit.clip_grads([g[0]], 1.0, out=[g[0].half()])
    with pytest.raises(ValueError):
        dit.grad_norm([torch.ones((4, 4), device="cuda").t()])
    for m in (-1.0, float("nan"), float("inf")):
        with pytest.raises(dit.DitError):
            dit.clip_grads(g, m)
    same = torch.ones(20, device="cuda")
    with pytest.raises(dit.DitError):
        dit.clip_grads([same[:8], same[8:16]], 1.0, out=[same[4:12], same[12:20]])
    with pytest.raises(dit.DitError):
        dit.grad_norm(g, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_streams_and_two_graphs():
    """Two captured calls replayed side by side, each with its own workspace."""
    a = [make(n, torch.bfloat16, "a", i).cuda() for i, n in enumerate((100, 70_000, 3))]
    b = [make(n, torch.float32, "b", i).cuda() for i, n in enumerate((5000, 1, 90_000))]
    la, lb = dit.TensorList(a, [torch.empty_like(t) for t in a]), dit.TensorList(b, [torch.empty_like(t) for t in b])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    (wa, na), (wb, nb) = dit.clip_grads(a, 1.0), dit.clip_grads(b, 1.0, stream=side)
    torch.cuda.synchronize()
    graphs, norms = [], []
    for lst in (la, lb):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norms.append(dit.clip_grads(lst, 1.0)[1])
        graphs.append(graph)
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    for lst, want, n, m in ((la, wa, na, norms[0]), (lb, wb, nb, norms[1])):
        assert torch.equal(bits(n), bits(m))
        assert all(torch.equal(bits(x), bits(y)) for x, y in zip(lst.out, want))


def test_more_tensors_than_a_launch_takes():
    gs = [make(11, torch.float32, "wide", i) for i in range(2000)]
    outs, norm = dit.clip_grads([g.cuda() for g in gs], 3.0)
    torch.cuda.synchronize()
    ref.check_clip(norm, outs, gs, 3.0)
