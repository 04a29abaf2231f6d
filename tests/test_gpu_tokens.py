"""A run of the token-transformer operators together: forward, backward and
clipping of tokens.step, against the same steps in 64 bits on the CPU, and its
gradients against differences of the 64-bit loss."""
import numpy as np
import pytest
import torch

import _token_ref as ref
import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300 import tokens
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
EPS, SCALE = 1e-6, 8.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def bits(t):
    return t.cpu().flatten().clone().view(torch.uint8)


def forward64(ids, table, weights, stand_ins):
    """(norm inputs, last y) of the definition without roundings."""
    ok = (ids >= 0) & (ids < len(table))
    x = np.where(ok[:, None], table[np.where(ok, ids, 0)] * SCALE, 0.0)
    kept, y = [x], ref.norm(x, weights[0], EPS, 0.0)
    for a, w in zip(stand_ins, weights[1:]):
        x = x + y * a
        kept.append(x)
        y = ref.norm(x, w, EPS, 0.0)
    return kept, y


def backward64(gy, ids, V, weights, stand_ins, kept):
    gx, _, gw, _ = ref.norm_grad(gy, kept[-1], weights[-1], EPS, 0.0)
    grads = [gw]
    for k in range(len(stand_ins) - 1, -1, -1):
        gx, _, gw, _ = ref.norm_grad(gx * stand_ins[k], kept[k], weights[k], EPS, 0.0, gx)
        grads.append(gw)
    gt = np.zeros((V, gx.shape[1]))
    ok = (ids >= 0) & (ids < V)
    np.add.at(gt, ids[ok], gx[ok])
    return [gt * SCALE] + grads[::-1]


def setup(n, V, D, blocks, dtype, padded):
    ids, table, weights, stand_ins = tokens.make_inputs(n, V, D, blocks, dtype, padded=padded)
    gy = draw("act", (n, D), seed_for("tokens", "gy", n, D), dtype, "cuda")
    host = (ids.cpu().numpy(), ref.f64(table), [ref.f64(w) for w in weights],
            [ref.f64(a) for a in stand_ins])
    return ids, table, weights, stand_ins, gy, host


@pytest.mark.parametrize("n,V,D,padded", [(40, 30, 96, 0), (300, 50, 264, 33), (20, 7, 129, 3)])
def test_step_in_fp32(n, V, D, padded):
    """fp32 throughout: the only differences are fp32 roundings, which a site
    (a norm, a product, an addition) multiplies little: five norms of relative error 2^-18 at most
    (ref.REL) each way, so 2^-18 * 10 of a row's size, times 8 for rows that a
    site shrinks."""
    ids, table, weights, stand_ins, gy, host = setup(n, V, D, 2, "fp32", padded)
    y, grads, norm = tokens.step(gy, ids, table, weights, stand_ins, 1.0, SCALE, EPS)
    torch.cuda.synchronize()
    kept, want = forward64(*host)
    tol = 80 * ref.REL
    real = host[0] >= 0
    assert np.abs(ref.f64(y) - want)[real].max() <= tol * np.abs(want).max()
    assert not ref.f64(y)[~real].any()
    exact = backward64(ref.f64(gy), host[0], V, host[2], host[3], kept)
    total = np.sqrt(sum((g ** 2).sum() for g in exact))
    assert abs(float(norm) - total) <= tol * total
    c = min(1.0, 1.0 / (total + 1e-6))
    assert total > 1.0
    for i, (g, e) in enumerate(zip(grads, exact)):
        assert np.abs(ref.f64(g) - e * c).max() <= tol * np.abs(e * c).max(), i
    # rows of the table that no token names
    unused = np.setdiff1d(np.arange(V), host[0])
    assert not ref.f64(grads[0])[unused].any()


def test_gradients_against_differences():
    """The step's gradients (fp32) against central differences of the 64-bit
    loss sum(y * gy) along random directions of the table and each weight: step
    h = 1e-5, so the difference itself is off by about h^2, and the kernels by
    fp32 roundings."""
    n, V, D = 24, 9, 64
    ids, table, weights, stand_ins, gy, host = setup(n, V, D, 1, "fp32", 2)
    _, grads, norm = tokens.step(gy, ids, table, weights, stand_ins, 1e6, SCALE, EPS)
    torch.cuda.synchronize()
    rng = np.random.default_rng(3)
    g64 = ref.f64(gy)

    def loss(t, ws):
        return (forward64(host[0], t, ws, host[3])[1] * g64).sum()

    h = 1e-5
    for i in range(len(grads)):
        leaf = host[1] if i == 0 else host[2][i - 1]
        d = rng.standard_normal(leaf.shape)
        ends = []
        for s in (h, -h):
            t, ws = host[1], list(host[2])
            if i == 0:
                t = t + s * d
            else:
                ws[i - 1] = leaf + s * d
            ends.append(loss(t, ws))
        want = (ends[0] - ends[1]) / (2 * h)
        got = (ref.f64(grads[i]) * d).sum()
        size = np.abs(ref.f64(grads[i]) * d).sum()
        assert abs(got - want) <= 1e-4 * size, i


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_captured_step_equals_the_eager_one(dtype):
    """16-bit storage, a padded batch: a replay gives the eager step's bits,
    with other ids and another gradient each time."""
    ids, table, weights, stand_ins, gy, _ = setup(700, 300, 512, 2, dtype, 50)
    graph, out = tokens.capture_step(gy, ids, table, weights, stand_ins, 1.0, SCALE, EPS)
    for r in range(3):
        ids.copy_(torch.roll(ids, 17 * r) if r else ids)
        gy.mul_(1.0 if r == 0 else 0.5)
        want = tokens.step(gy, ids, table, weights, stand_ins, 1.0, SCALE, EPS)
        graph.replay()
        torch.cuda.synchronize()
        # bits: in fp16 the padded rows' gradients (r = 1000 at each norm)
        # overflow, and the norm is NaN on both sides
        for a, b in zip([out[0], out[2], *out[1]], [want[0], want[2], *want[1]]):
            assert torch.equal(bits(a), bits(b))


def test_decode_follows_forward():
    """Single tokens: the same residual stream as forward, bit for bit, and
    codes of the last norm."""
    for n in (1, 5):
        ids, table, weights, stand_ins, _, _ = setup(n, 64, 1024, 2, "bf16", 0)
        x, y = tokens.forward(ids, table, weights, stand_ins, SCALE, EPS)
        x8, q, s = tokens.decode(ids, table, weights, stand_ins, SCALE, EPS)
        torch.cuda.synchronize()
        assert torch.equal(x, x8)
        ref.check_fp8(q, s, x, weights[-1], EPS, 0.0, 128)
