"""The weighted RMSNorm over many rows of odd and even widths, so that a team of
warps takes several rows one after another, and over rows of extreme values,
against the 64-bit reference.

An SM holds at most 64 warps, so a team of k warps is one of at most 64 / k an
SM.  A warp holds at most 4 units of 512 bytes: a row of b bytes has a team of
at least b / 2048 warps, and at most 64 * 2048 / b rows of an SM are held at once (64
where a row is less than a warp's).  The sizes below have more rows than that on
152 SMs."""
import numpy as np
import pytest
import torch

import _token_ref as ref
import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built, guarded
from diffusion_transformer_elementwise_gb300.synth import seed_for

pytestmark = pytest.mark.gpu
EPS = 1e-6
IDS = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
dtypes = pytest.mark.parametrize("dtype", ref.TYPES, ids=IDS.get)


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def normal(shape, dtype, *seed, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed_for("rows", *seed, *shape) % (1 << 62))
    v = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    return v.mul_(std).add_(mean).to(dtype)


def bits(t):
    return t.flatten().view(torch.uint8)


def codes(rows, D):
    """An E4M3 output between canaries."""
    buf = torch.full((rows * D + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    return buf[32:32 + rows * D].view(rows, D), \
        lambda: bool((buf[:32] == 0xA5).all()) and bool((buf[32 + rows * D:] == 0xA5).all())


# the last one's rows fill a CTA's registers in each type
SIZES = [(20000, 129), (25000, 256), (30000, 131), (12000, 1001), (4097, 3077), (1500, 8189)]


@pytest.mark.parametrize("rows,D", SIZES)
@dtypes
def test_forward_of_several_rows_a_team(dtype, rows, D):
    h, u = normal((rows, D), dtype, "h"), normal((rows, D), dtype, "u")
    h *= torch.exp2(torch.arange(rows, device="cuda") % 9 - 4.0).to(dtype)[:, None]
    w = normal((D,), dtype, "w", std=0.2, mean=1.0)
    hb, ub = h.clone(), u.clone()
    out, f1 = guarded((rows, D), dtype, "cuda")
    out2, f2 = guarded((rows, D), dtype, "cuda")
    res, f3 = guarded((rows, D), dtype, "cuda")
    dit.rmsnorm(h, w, EPS, out=out)
    dit.add_rmsnorm(h, u, w, EPS, residual_out=res, out=out2)
    eight, fresh = [], [f1, f2, f3]
    for group in (0, 128):
        n = -(-D // 128) if group else 1
        for add in (False, True):
            q, f = codes(rows, D)
            s, g = guarded((rows, n), torch.float32, "cuda")
            r, k = guarded((rows, D), dtype, "cuda")
            if add:
                dit.add_rmsnorm_fp8(h, u, w, EPS, group, residual_out=r, out=q, scales=s)
            else:
                dit.rmsnorm_fp8(h, w, EPS, group, out=q, scales=s)
            eight.append((group, add, q, s, r))
            fresh += [f, g, k]
    torch.cuda.synchronize()
    assert all(f() for f in fresh)
    assert torch.equal(bits(h), bits(hb)) and torch.equal(bits(u), bits(ub))
    want = (h.float() + u.float()).to(dtype)
    assert torch.equal(bits(res), bits(want))
    # the outputs of rows from everywhere, and of the last ones
    n = max(100, 400_000 // D)
    rng = np.random.default_rng(rows)
    at = torch.from_numpy(np.concatenate([rng.choice(rows, n, replace=False),
                                          np.arange(rows - 16, rows)])).cuda()
    ref.check_norm(out[at], h[at], w, EPS, 0.0, "norm")
    ref.check_norm(out2[at], res[at], w, EPS, 0.0, "add")
    for group, add, q, s, r in eight:
        x = res if add else h
        ref.check_fp8(q[at], s[at], x[at], w, EPS, 0.0, group, f"group {group} add {add}")
        if add:
            assert torch.equal(bits(r), bits(want))


@pytest.mark.parametrize("rows,D", [(20000, 129), (4097, 3077), (30000, 131)])
@dtypes
def test_backward_of_several_rows_a_team(dtype, rows, D):
    x, k = normal((rows, D), dtype, "x"), normal((rows, D), dtype, "k")
    g = normal((rows, D), dtype, "g", std=0.3)
    w = normal((D,), dtype, "w", std=0.2, mean=1.0)
    gx, f1 = guarded((rows, D), dtype, "cuda")
    gw, f2 = guarded((D,), dtype, "cuda")
    dit.rmsnorm_backward(g, x, w, EPS, grad_residual=k, grad_x=gx, grad_weight=gw)
    torch.cuda.synchronize()
    assert f1() and f2()
    ref.check_norm_grad(gx, gw, g, x, w, EPS, 0.0, k)


@pytest.mark.parametrize("D", [200, 3077, 4096, 20000])
@dtypes
def test_fp8_of_small_rows(dtype, D):
    """Rows whose mean square is far below eps: r = 1000, their scales are
    2^-80 and less but normal fp32 numbers (fp16: ordinary rows of its range)."""
    x = normal((6, D), dtype, "small")
    if dtype == torch.float16:
        x[1] *= 2.0 ** -10
    else:
        x[1] *= 2.0 ** -80
        x[3] = 2.0 ** -120
        x[4] = -2.0 ** -110
    w = normal((D,), dtype, "w", std=0.2, mean=1.0)
    for group in (0, 128):
        q, s = dit.rmsnorm_fp8(x, w, EPS, group)
        _, q2, s2 = dit.add_rmsnorm_fp8(x, torch.zeros_like(x), w, EPS, group)
        torch.cuda.synchronize()
        ref.check_fp8(q, s, x, w, EPS, 0.0, group, f"group {group}")
        ref.check_fp8(q2, s2, x, w, EPS, 0.0, group, f"group {group}, with an update")


@pytest.mark.parametrize("D", [200, 3077, 4096, 20000])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=IDS.get)
def test_mean_squares_below_fp32_without_eps(dtype, D):
    """eps = 0: the mean square of these rows is below 2^-150 and rounds to zero,
    so r is +inf as the header says: infinities with the signs of the products, NaN for
    zeros.  The rows between them are ordinary."""
    x = normal((7, D), dtype, "zero")
    x[x == 0] = 1.0
    x[1] *= 2.0 ** -80
    x[3] = 0
    x[3, 3] = 2.0 ** -126
    x[5] = 0
    w = normal((D,), dtype, "w", std=0.1, mean=1.0)
    assert float(w.float().min()) > 0
    out = dit.rmsnorm(x, w, 0.0)
    _, added = dit.add_rmsnorm(x, torch.zeros_like(x), w, 0.0)
    coded = [dit.rmsnorm_fp8(x, w, 0.0, group)[1] for group in (0, 128)]
    torch.cuda.synchronize()
    for o in (out, added):
        ref.check_norm(o[::2], x[::2], w, 0.0, 0.0)
        o = o.float()
        assert torch.equal(o[1], x[1].float() * float("inf"))
        assert float(o[3, 3]) == float("inf") and int(torch.isnan(o[3]).sum()) == D - 1
        assert bool(torch.isnan(o[5]).all())
    for s in coded:
        for i in (1, 3, 5):
            assert not bool(torch.isfinite(s[i]).any()), i
        for i in (0, 2, 4, 6):
            assert bool(torch.isfinite(s[i]).all()), i
