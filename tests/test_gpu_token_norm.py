"""The weighted RMSNorm, its E4M3 output and its gradient on the GPU, against
the 64-bit reference of tests/_token_ref.py (whose tolerances count the
kernels' roundings)."""
import numpy as np
import pytest
import torch

import _token_ref as ref
import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built, guarded, offset_copy
from diffusion_transformer_elementwise_gb300.synth import seed_for

pytestmark = pytest.mark.gpu
EPS = 1e-6
IDS = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
dtypes = pytest.mark.parametrize("dtype", ref.TYPES, ids=IDS.get)

# Widths: one element, around one lane's granule, around a group of 128 and a
# unit, teams of several warps, the widest in registers (16384 of 16 bits, 8192 of
# fp32) and beyond it, odd ones of each kind.
WIDTHS = [1, 7, 8, 64, 127, 128, 129, 256, 264, 1000, 2048, 3077, 4096, 8192, 8200, 16384, 16392,
          20001]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def make(shape, dtype, *seed, std=1.0, mean=0.0, spread=False):
    rng = np.random.default_rng(seed_for(*seed))
    v = rng.standard_normal(shape) * std + mean
    if spread:
        v = v * 10.0 ** rng.uniform(-2, 2, size=(shape[0], 1))
    return torch.from_numpy(v).to(dtype)


def inputs(rows, D, dtype, tag, offset=0.0):
    return (make((rows, D), dtype, tag, "h", rows, D, spread=True),
            make((rows, D), dtype, tag, "u", rows, D),
            make((D,), dtype, tag, "w", D, std=0.2, mean=1.0 - offset))


def bits(t):
    return t.cpu().flatten().clone().view(torch.uint8) if t.numel() else torch.empty(0)


@pytest.mark.parametrize("D", WIDTHS)
@dtypes
def test_norm_and_add(dtype, D):
    rows = 5
    h, u, w = inputs(rows, D, dtype, "norm", 1.0)
    hd, ud, wd = h.cuda(), u.cuda(), w.cuda()
    out, fresh = guarded((rows, D), dtype, "cuda")
    got = dit.rmsnorm(hd, wd, EPS, 1.0, out=out)
    assert got is out
    res, rfresh = guarded((rows, D), dtype, "cuda")
    r2, o2 = dit.add_rmsnorm(hd, ud, wd, EPS, 1.0, residual_out=res)
    torch.cuda.synchronize()
    ref.check_norm(out, h, w, EPS, 1.0, "norm")
    assert torch.equal(bits(r2), bits(ref.residual(h, u)))
    ref.check_norm(o2, r2, w, EPS, 1.0, "add")
    assert fresh() and rfresh()
    assert torch.equal(bits(hd), bits(h)) and torch.equal(bits(ud), bits(u))


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("D", WIDTHS)
@dtypes
def test_fp8(dtype, D, group):
    rows = 5
    h, u, w = inputs(rows, D, dtype, "fp8")
    h[3] = 0
    u[3] = 0
    buf = torch.full((rows * D + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = buf[32:32 + rows * D].view(rows, D)
    q, s = dit.rmsnorm_fp8(h.cuda(), w.cuda(), EPS, group, out=out)
    r2, q2, s2 = dit.add_rmsnorm_fp8(h.cuda(), u.cuda(), w.cuda(), EPS, group)
    torch.cuda.synchronize()
    assert q is out and q2.dtype == torch.float8_e4m3fn
    ref.check_fp8(q, s, h, w, EPS, 0.0, group, "norm")
    assert torch.equal(bits(r2), bits(ref.residual(h, u)))
    ref.check_fp8(q2, s2, r2, w, EPS, 0.0, group, "add")
    assert bool((buf[:32] == 0xA5).all()) and bool((buf[32 + rows * D:] == 0xA5).all())
    assert not s[3].any() and not q.view(torch.uint8)[3].any()


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("D", WIDTHS)
@dtypes
def test_backward(dtype, D, skip):
    rows = 7
    x, k, w = inputs(rows, D, dtype, "back", 1.0)
    g = make((rows, D), dtype, "back", "g", D, std=0.3)
    gx, fresh = guarded((rows, D), dtype, "cuda")
    gw, wfresh = guarded((D,), dtype, "cuda")
    got = dit.rmsnorm_backward(g.cuda(), x.cuda(), w.cuda(), EPS, 1.0,
                               grad_residual=k.cuda() if skip else None, grad_x=gx, grad_weight=gw)
    torch.cuda.synchronize()
    assert got[0] is gx and got[1] is gw and fresh() and wfresh()
    ref.check_norm_grad(gx, gw, g, x, w, EPS, 1.0, k if skip else None)


@pytest.mark.parametrize("rows,D", [(1, 4096), (2, 64), (126, 2048), (128, 3077), (129, 3077),
                                    (100, 8192), (3, 16384), (64, 100), (3000, 200), (1300, 1000),
                                    (700, 4096), (5000, 33), (40, 20000)])
@dtypes
def test_backward_many_rows(dtype, rows, D):
    """More rows than CTAs, and CTAs of several teams."""
    x, k, w = inputs(rows, D, dtype, "rows")
    g = make((rows, D), dtype, "rows", "g", rows, D, std=0.3)
    gx, gw = dit.rmsnorm_backward(g.cuda(), x.cuda(), w.cuda(), EPS, grad_residual=k.cuda())
    again = dit.rmsnorm_backward(g.cuda(), x.cuda(), w.cuda(), EPS, grad_residual=k.cuda())
    frozen = dit.rmsnorm_backward(g.cuda(), x.cuda(), w.cuda(), EPS, grad_residual=k.cuda(),
                                  need_weight=False)
    torch.cuda.synchronize()
    ref.check_norm_grad(gx, gw, g, x, w, EPS, 0.0, k)
    assert torch.equal(bits(gx), bits(again[0])) and torch.equal(bits(gw), bits(again[1]))
    assert torch.equal(bits(gx), bits(frozen[0])) and frozen[1] is None


@pytest.mark.parametrize("rows,D", [(1, 8192), (3001, 96), (1201, 1024), (700, 4096), (17, 40000)])
@dtypes
def test_forward_many_rows(dtype, rows, D):
    h, u, w = inputs(rows, D, dtype, "many")
    r, o = dit.add_rmsnorm(h.cuda(), u.cuda(), w.cuda(), EPS)
    for group in (0, 128):
        r8, q, s = dit.add_rmsnorm_fp8(h.cuda(), u.cuda(), w.cuda(), EPS, group)
        ref.check_fp8(q, s, r, w, EPS, 0.0, group)
        assert torch.equal(bits(r8), bits(r))
    ref.check_norm(o, r, w, EPS, 0.0)
    assert torch.equal(bits(r), bits(ref.residual(h, u)))


@pytest.mark.parametrize("D", [1, 8, 136, 1000, 4096, 3077, 20000])
@pytest.mark.parametrize("off", [1, 4])
@dtypes
def test_tensors_off_a_16_byte_boundary(dtype, off, D):
    """Every tensor at another offset from a 16-byte boundary."""
    rows = 3
    h, u, w = inputs(rows, D, dtype, "off")
    hd, ud, wd = offset_copy(h, off), offset_copy(u, 0), offset_copy(w, off + 1)
    res, out = offset_copy(torch.zeros_like(h), off + 2), offset_copy(torch.zeros_like(h), off)
    dit.add_rmsnorm(hd, ud, wd, EPS, residual_out=res, out=out)
    codes = torch.empty(rows * D + 8, dtype=torch.uint8, device="cuda")[off:off + rows * D].view(rows, D)
    _, s = dit.rmsnorm_fp8(hd, wd, EPS, 128, out=codes)
    gx, gw = dit.rmsnorm_backward(ud, hd, wd, EPS, grad_x=offset_copy(torch.zeros_like(h), off),
                                  grad_weight=offset_copy(torch.zeros_like(w), off))
    torch.cuda.synchronize()
    assert torch.equal(bits(res), bits(ref.residual(h, u)))
    ref.check_norm(out, res, w, EPS, 0.0)
    ref.check_fp8(codes, s, h, w, EPS, 0.0, 128)
    ref.check_norm_grad(gx, gw, u, h, w, EPS, 0.0)


@pytest.mark.parametrize("D", [64, 4096, 8192])
@dtypes
def test_weight_alone_off_a_16_byte_boundary(dtype, D):
    rows = 6
    h, u, w = inputs(rows, D, dtype, "woff")
    hd, ud, wd = h.cuda(), u.cuda(), offset_copy(w, 3)
    res, out = dit.add_rmsnorm(hd, ud, wd, EPS)
    gx, gw = dit.rmsnorm_backward(ud, hd, wd, EPS)
    torch.cuda.synchronize()
    ref.check_norm(out, res, w, EPS, 0.0)
    ref.check_norm_grad(gx, gw, u, h, w, EPS, 0.0)
    for group in (0, 128):
        q, s = dit.rmsnorm_fp8(hd, wd, EPS, group)
        ref.check_fp8(q, s, h, w, EPS, 0.0, group)


@pytest.mark.parametrize("rows,D", [(200, 3077), (150, 129), (1300, 1001), (90, 16389)])
@dtypes
def test_in_place_of_odd_widths(dtype, rows, D):
    """Outputs over their inputs where rows share 16-byte granules, in every
    form that allows it, equal the results in other memory."""
    h, u, w = (t.cuda() for t in inputs(rows, D, dtype, "oddplace"))
    g = make((rows, D), dtype, "oddplace", "g", rows, D).cuda()
    res, out = dit.add_rmsnorm(h, u, w, EPS)
    gx, gw = dit.rmsnorm_backward(g, h, w, EPS, grad_residual=u)
    for _ in range(3):
        x = h.clone()
        r, o = dit.add_rmsnorm(x, u, w, EPS, residual_out=x)
        assert torch.equal(bits(r), bits(res)) and torch.equal(bits(o), bits(out))
        for group in (0, 128):
            q, s = dit.rmsnorm_fp8(res, w, EPS, group)
            x = h.clone()
            _, q2, s2 = dit.add_rmsnorm_fp8(x, u, w, EPS, group, residual_out=x)
            assert torch.equal(bits(x), bits(res)) and torch.equal(bits(q), bits(q2))
            assert torch.equal(bits(s), bits(s2))
        g2, u2 = g.clone(), u.clone()
        a = dit.rmsnorm_backward(g2, h, w, EPS, grad_residual=u, grad_x=g2)
        b = dit.rmsnorm_backward(g, h, w, EPS, grad_residual=u2, grad_x=u2)
        for t in (a, b):
            assert torch.equal(bits(t[0]), bits(gx)) and torch.equal(bits(t[1]), bits(gw))


@pytest.mark.parametrize("D", [200, 3077, 4096, 20000])
@dtypes
def test_rows_of_extreme_values(dtype, D):
    """Zeros, the lowest value, infinities, NaN, squares beyond and below
    fp32's range, one element among zeros -- each a row of its own, between ordinary
    rows, which they must not touch."""
    top = torch.finfo(dtype).max
    x = make((14, D), dtype, "extreme", D)
    x[1] = 0
    x[2] = -top
    x[3, D // 2] = float("inf")
    x[4, 0] = -float("inf")
    x[4, D - 1] = float("nan")
    x[5, D - 1] = float("nan")
    x[6] = 0
    x[6, D - 1] = top
    x[7] = 0
    x[7, 3] = torch.finfo(dtype).tiny
    if dtype != torch.float16:
        x[8] *= 2.0 ** 70
        x[9] *= 2.0 ** -80
        x[10] = 2.0 ** -120
        x[11] *= 2.0 ** 55
    w = make((D,), dtype, "extreme", "w", D, std=0.2, mean=1.0)
    g = make((14, D), dtype, "extreme", "g", D)
    for eps in (EPS, 0.0):
        out = dit.rmsnorm(x.cuda(), w.cuda(), eps)
        torch.cuda.synchronize()
        # r of a tiny mean square under eps = 0 may be one subnormal step of it off
        rows = [i for i in range(14) if eps > 0 or i not in (7, 9, 10)]
        ref.check_norm(out[rows], x[rows], w, eps, 0.0, f"eps {eps}")
    for group in (0, 128):
        q, s = dit.rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group)
        torch.cuda.synchronize()
        rows = [i for i in range(14) if i not in (9, 10)]  # scales below fp32's normal range
        ref.check_fp8(q[rows], s[rows], x[rows], w, EPS, 0.0, group, f"group {group}")
    gx, gw = dit.rmsnorm_backward(g.cuda(), x.cuda(), w.cuda(), EPS)
    torch.cuda.synchronize()
    for i in range(14):
        if i in (3, 4, 5):
            assert bool(torch.isnan(gx[i].float()).any())
            continue
        ref.check_norm_grad(gx[i:i + 1], None, g[i:i + 1], x[i:i + 1], w, EPS, 0.0, what=f"row {i}")
    assert bool(torch.isnan(gw.float()).any())


@dtypes
def test_fp8_of_tiny_rows(dtype):
    """Rows whose scale is far below one: the codes keep their three bits."""
    if dtype == torch.float16:
        pytest.skip("fp16 does not reach below 2^-24")
    x = make((4, 384), dtype, "tiny8")
    x = x * torch.tensor([1.0, 2.0 ** -60, 2.0 ** -80, 2.0 ** -90], dtype=torch.float64)[:, None].to(dtype)
    w = make((384,), dtype, "tiny8", "w", std=0.2, mean=1.0)
    for group in (0, 128):
        q, s = dit.rmsnorm_fp8(x.cuda(), w.cuda(), EPS, group)
        torch.cuda.synchronize()
        ref.check_fp8(q, s, x, w, EPS, 0.0, group)


def test_in_place_and_shapes():
    h, u, w = (t.cuda() for t in inputs(24, 512, torch.bfloat16, "inplace"))
    want, o1 = dit.add_rmsnorm(h, u, w)
    h2 = h.clone().view(2, 3, 4, 512)
    r, o2 = dit.add_rmsnorm(h2, u.view(2, 3, 4, 512), w, residual_out=h2)
    assert r is h2 and o2.shape == h2.shape
    assert torch.equal(bits(h2), bits(want)) and torch.equal(bits(o1), bits(o2))
    q, s = dit.rmsnorm_fp8(h2, w, group=128)
    assert q.shape == h2.shape and s.shape == (2, 3, 4, 4)
    q, s = dit.rmsnorm_fp8(h2[0, 0, 0], w)  # one token
    assert q.shape == (512,) and s.shape == (1,)
    # the gradient over its own inputs
    g = make((24, 512), torch.bfloat16, "inplace", "g").cuda()
    a = dit.rmsnorm_backward(g, h, w, grad_residual=u)
    g2, u2 = g.clone(), u.clone()
    b = dit.rmsnorm_backward(g2, h, w, grad_residual=u, grad_x=g2)
    c = dit.rmsnorm_backward(g, h, w, grad_residual=u2, grad_x=u2)
    torch.cuda.synchronize()
    for t in (b, c):
        assert torch.equal(bits(t[0]), bits(a[0])) and torch.equal(bits(t[1]), bits(a[1]))


def test_empty():
    w = torch.ones(64, device="cuda")
    e = torch.empty((0, 64), device="cuda")
    assert dit.rmsnorm(e, w).shape == (0, 64)
    r, q, s = dit.add_rmsnorm_fp8(e, e, w, group=128, residual_out=torch.empty_like(e))
    assert q.shape == (0, 64) and s.shape == (0, 1)
    gx, gw = dit.rmsnorm_backward(e, e, w, grad_weight=torch.full((64,), 3.0, device="cuda"))
    torch.cuda.synchronize()
    assert gx.shape == (0, 64) and not gw.any()
    z = torch.empty((4, 0), device="cuda")
    assert dit.rmsnorm(z, torch.empty(0, device="cuda")).shape == (4, 0)


@dtypes
def test_rows_of_no_columns_have_scale_zero(dtype):
    z, w = torch.empty((5, 0), dtype=dtype, device="cuda"), torch.empty(0, dtype=dtype, device="cuda")
    scales, fresh = guarded((5, 1), torch.float32, "cuda")
    q, s = dit.rmsnorm_fp8(z, w, scales=scales)
    r, q2, s2 = dit.add_rmsnorm_fp8(z, z, w, residual_out=torch.empty_like(z),
                                    scales=torch.full((5, 1), 3.0, device="cuda"))
    torch.cuda.synchronize()
    assert q.shape == (5, 0) and s is scales and not s.any() and not s2.any()
    assert fresh()
    assert dit.rmsnorm_fp8(z, w, group=128)[1].shape == (5, 0)


def test_refusals():
    x = torch.zeros((4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        dit.rmsnorm(x.t(), torch.ones(4, device="cuda"))       # not contiguous
    with pytest.raises(ValueError):
        dit.rmsnorm(x, w[:32])
    with pytest.raises(TypeError):
        dit.rmsnorm(x, w.half())
    with pytest.raises(TypeError):
        dit.rmsnorm(x.double(), w.double())
    with pytest.raises(ValueError):
        dit.add_rmsnorm(x, x[:2].contiguous(), w)
    with pytest.raises(ValueError):
        dit.rmsnorm_fp8(x, w, scales=torch.empty(4, device="cuda"))
    with pytest.raises(TypeError):
        dit.rmsnorm_fp8(x, w, out=torch.empty_like(x))
    with pytest.raises(dit.DitError):
        dit.rmsnorm(x, w, eps=-1.0)
    with pytest.raises(dit.DitError):
        dit.rmsnorm(x, w, weight_offset=float("nan"))
    with pytest.raises(dit.DitError):
        dit.rmsnorm(x, w, out=x)
    with pytest.raises(dit.DitError):
        many = torch.zeros((200, 64), device="cuda")
        dit.rmsnorm_backward(many, many, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_streams_and_graphs():
    """On a stream of its own, by argument and by context; captured, with new
    values in the same tensors before a replay."""
    h, u, w = (t.cuda() for t in inputs(300, 1024, torch.float16, "graph"))
    g = make((300, 1024), torch.float16, "graph", "g").cuda()

    def step(stream=None):
        r, o = dit.add_rmsnorm(h, u, w, stream=stream)
        _, q, s = dit.add_rmsnorm_fp8(h, u, w, group=128, stream=stream)
        gx, gw = dit.rmsnorm_backward(g, r, w, grad_residual=o, stream=stream)
        return [r, o, q.view(torch.uint8), s, gx, gw]

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = step(side)
    b = step(side.cuda_stream)
    with torch.cuda.stream(side):
        c = step()
    torch.cuda.synchronize()
    for got in (a, b, c):
        for x, y in zip(got, want):
            assert torch.equal(bits(x), bits(y))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for scale in (1.0, 0.5):
        h.mul_(scale)
        want = step()
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(outs, want):
            assert torch.equal(bits(x), bits(y))


def test_long_tensor_offsets():
    """Byte offsets past 2^32: the last rows of [70000, 32768] bf16 (4.6 GB)."""
    rows, D = 70000, 32768
    x = torch.empty((rows, D), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    tail = make((3, D), torch.bfloat16, "long")
    x[-3:] = tail.cuda()
    w = make((D,), torch.bfloat16, "long", "w", std=0.2, mean=1.0)
    out = dit.rmsnorm(x, w.cuda())
    torch.cuda.synchronize()
    ref.check_norm(out[-3:], tail, w, EPS, 0.0)
    del out
    gx, _ = dit.rmsnorm_backward(x, x, w.cuda(), need_weight=False)
    torch.cuda.synchronize()
    ref.check_norm_grad(gx[-3:], None, tail, tail, w, EPS, 0.0)
