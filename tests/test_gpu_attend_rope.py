"""Rotary angles, the rotation of queries and keys, the norm of heads in the same
pass and its gradient, against 64 bits (tests/_attend_ref.py)."""
import math

import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import check_rope, check_rope_grad, check_table, f64
from _gpu import ensure_built, guarded, offset_copy
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("attend", tag, *shape), dtype, "cuda")


def angles(rows, R):
    """A table of cos and sin of any angles."""
    a = act(rows, max(R, 1), tag="angle", dtype="fp32").double()[:, :R] * 3
    return a.cos().float(), a.sin().float()


# --- the table ------------------------------------------------------------

@pytest.mark.parametrize("sections", [[1], [64], [3, 5], [20, 22, 22], [0, 7, 0, 2], [1] * 8, [300, 212]])
@pytest.mark.parametrize("kind", ["int32", "int64", "fp32"])
@pytest.mark.parametrize("tokens", [1, 7, 1025])
def test_table(sections, kind, tokens):
    A = len(sections)
    u = draw("gate", (A, tokens), seed_for("table", A, tokens, kind), "fp32", "cuda").double()
    p = {"int32": (u * 2.0 ** 20).to(torch.int32), "int64": (u * 2.0 ** 40).to(torch.int64),
         "fp32": (u * 1000.0).float()}[kind]
    f = dit.rotary_frequencies(sections, shared=A % 2 == 0)
    assert f.dtype is torch.float64 and f.shape == (sum(sections),)
    cos, sin = dit.rotary_table(p, f, sections)
    check_table(cos, sin, p, f, sections)


def test_table_frequencies_far_and_odd():
    f = torch.tensor([0.0, 1e-300, -0.37, 2 * math.pi, 7.5, -123456.75, math.inf, math.nan, 1e-20, -1e-20],
                     dtype=torch.float64, device="cuda")
    p = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1], dtype=torch.int64, device="cuda")
    for q in (p, p.to(torch.int32), (p.double() * 0.37).float(), p.float() * 2.0 ** -40):
        cos, sin = dit.rotary_table(q, f)
        check_table(cos, sin, q[None], f, [10])
    far = torch.tensor([math.inf, -math.inf, math.nan, 1.0], device="cuda")
    cos, sin = dit.rotary_table(far, f[2:4])
    assert torch.isnan(cos[:3]).all() and torch.isnan(sin[:3]).all() and torch.isfinite(cos[3]).all()


def test_table_of_nothing():
    f = dit.rotary_frequencies(4)
    cos, sin = dit.rotary_table(torch.empty(0, dtype=torch.int64, device="cuda"), f)
    assert cos.shape == (0, 4)
    cos, sin = dit.rotary_table(torch.zeros(3, dtype=torch.int64, device="cuda"), f[:0])
    assert cos.shape == (3, 0)


# --- rotation and norm ------------------------------------------------------

SHAPES = [  # B, L, Hq, Hk, D, R
    (1, 1, 1, 0, 2, 1), (1, 1, 1, 1, 64, 32), (1, 5, 3, 2, 128, 64), (2, 3, 4, 1, 128, 32),
    (3, 7, 2, 2, 80, 40), (1, 130, 5, 1, 80, 10), (2, 2, 1, 3, 256, 128), (1, 3, 2, 1, 257, 100),
    (1, 2, 1, 1, 1024, 512), (2, 33, 8, 2, 96, 48), (1, 9, 2, 1, 33, 16), (1, 4, 2, 1, 72, 0),
    (1, 3, 2, 2, 192, 12), (1, 700, 6, 2, 64, 32), (1, 2, 2, 1, 512, 256), (1, 3, 1, 1, 1, 0)]


def layouts(kind, B, L, Hq, Hk, D, dtype, tag=""):
    """Queries and keys as [B, L, H, D] (or [L, H, D]) views: contiguous, of one packed projection,
    heads before tokens, or off a 16-byte boundary."""
    if kind == "packed":
        qkv = act(B, L, Hq + 2 * Hk, D, tag="qkv" + tag, dtype=dtype)
        return qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    q = act(B, L, Hq, D, tag="q" + tag, dtype=dtype)
    k = act(B, L, Hk, D, tag="k" + tag, dtype=dtype)
    if kind == "heads":
        return (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k))
    if kind == "shifted":
        return offset_copy(q, 1), offset_copy(k, 3)
    if kind == "three" and B == 1:
        return q[0], k[0]
    return q, k


@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("kind", ["plain", "packed", "heads", "shifted", "three"])
@pytest.mark.parametrize("shape", SHAPES)
def test_rope(shape, kind, dtype):
    B, L, Hq, Hk, D, R = shape
    q, k = layouts(kind, B, L, Hq, Hk, D, dtype)
    wq, wk = (act(D, tag=n, dtype=dtype) for n in ("wq", "wk"))
    for rows in {L, B * L}:
        cos, sin = angles(rows, R)
        for inter in (False, True):
            for inverse in (False, True):
                gq, gk = dit.rope(q, k, cos, sin, interleaved=inter, inverse=inverse)
                for g, x in ((gq, q), (gk, k)):
                    check_rope(g, x, cos, sin, interleaved=inter, inverse=inverse, what="rope")
            gq, gk = dit.rmsnorm_rope(q, k, wq, wk, cos, sin, 1e-5, 0.5, interleaved=inter)
            for g, x, w in ((gq, q, wq), (gk, k, wk)):
                check_rope(g, x, cos, sin, w, 1e-5, 0.5, inter, what="norm")
    g1, _ = dit.rmsnorm_rope(q, None, wq, None, None, None)
    check_rope(g1, q, None, None, wq, 1e-6, 0.0, what="norm alone")
    cos, sin = angles(L, R)
    g1, none = dit.rope(q, None, cos, sin)
    check_rope(g1, q, cos, sin)
    assert none is None


@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("D,R", [(128, 64), (80, 10), (33, 16)])
def test_in_place_and_bounds(D, R, dtype):
    B, L, Hq, Hk = 2, 9, 3, 1
    wq, wk = (act(D, tag=n, dtype=dtype) for n in ("wq", "wk"))
    cos, sin = angles(L, R)
    qkv = act(B, L, Hq + 2 * Hk, D, tag="qkv", dtype=dtype)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk]
    for call in (lambda q, k, **o: dit.rmsnorm_rope(q, k, wq, wk, cos, sin, **o),
                 lambda q, k, **o: dit.rope(q, k, cos, sin, interleaved=True, **o)):
        want = call(q, k)
        mine = qkv.clone()
        mq, mk = mine[:, :, :Hq], mine[:, :, Hq:Hq + Hk]
        got = call(mq, mk, out_q=mq, out_k=mk)  # in place, within the packed projection
        assert torch.equal(got[0], want[0]) and torch.equal(mk, want[1])
        assert torch.equal(mine[:, :, Hq + Hk:], qkv[:, :, Hq + Hk:])
        oq, fine_q = guarded(tuple(q.shape), T[dtype], "cuda")
        ok, fine_k = guarded(tuple(k.shape), T[dtype], "cuda")
        got = call(q, k, out_q=oq, out_k=ok)
        assert torch.equal(oq, want[0]) and torch.equal(ok, want[1]) and fine_q() and fine_k()


def test_infinities_and_zeros():
    x = act(4, 2, 128, tag="inf", dtype="fp32")
    x[0, 0, 5] = math.inf
    x[1, 1, 77] = math.nan
    x[2] = 0
    x[3] *= 1e25  # the mean square leaves fp32
    w = act(128, tag="w", dtype="fp32")
    cos, sin = angles(4, 64)
    y, _ = dit.rmsnorm_rope(x, None, w, None, cos, sin)
    assert torch.isnan(y[0, 0, 5]) and torch.isfinite(y[0, 1]).all() and torch.isnan(y[1, 1]).all()
    assert torch.isfinite(y[1, 0]).all() and (y[2] == 0).all() and (y[3] == 0).all()
    y, _ = dit.rope(x, None, cos, sin)
    assert int(torch.isnan(y).sum()) + int(torch.isinf(y).sum()) == 4


# --- the gradient -----------------------------------------------------------

@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("kind", ["plain", "packed", "shifted"])
@pytest.mark.parametrize("shape", SHAPES + [(2, 1000, 4, 1, 64, 32)])
def test_gradient(shape, kind, dtype):
    B, L, Hq, Hk, D, R = shape
    q, k = layouts(kind, B, L, Hq, Hk, D, dtype)
    gq, gk = layouts(kind, B, L, Hq, Hk, D, dtype, tag="grad")
    wq, wk = (act(D, tag=n, dtype=dtype) for n in ("wq", "wk"))
    for rows, inter in ((L, False), (B * L, True)):
        cos, sin = angles(rows, R)
        got = dit.rmsnorm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, 1e-5, 0.5, interleaved=inter)
        again = dit.rmsnorm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, 1e-5, 0.5, interleaved=inter)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        for gx, gw, g, x, w in ((got[0], got[2], gq, q, wq), (got[1], got[3], gk, k, wk)):
            check_rope_grad(gx, gw, g, x, cos, sin, w, 1e-5, 0.5, inter)
        frozen = dit.rmsnorm_rope_backward(gq, gk, q, k, wq, wk, cos, sin, 1e-5, 0.5, interleaved=inter,
                                           need_weight=False)
        assert torch.equal(frozen[0], got[0]) and torch.equal(frozen[1], got[1])
        assert frozen[2] is None and frozen[3] is None
    alone = dit.rmsnorm_rope_backward(gq, None, q, None, wq, None, None, None)
    check_rope_grad(alone[0], alone[2], gq, q, None, None, wq)


def test_gradient_in_place_and_of_nothing():
    q, k = layouts("plain", 2, 5, 4, 2, 128, "bf16")
    gq, gk = layouts("plain", 2, 5, 4, 2, 128, "bf16", tag="grad")
    w = act(128, tag="w")
    cos, sin = angles(5, 64)
    want = dit.rmsnorm_rope_backward(gq, gk, q, k, w, w, cos, sin)
    a, b = gq.clone(), gk.clone()
    got = dit.rmsnorm_rope_backward(a, b, q, k, w, w, cos, sin, grad_q=a, grad_k=b)
    assert all(torch.equal(x, y) for x, y in zip(got, want)) and got[0] is a
    none = dit.rmsnorm_rope_backward(gq[:, :0], gk[:, :0], q[:, :0], k[:, :0], w, w, cos[:0], sin[:0],
                                     grad_weight_q=torch.full_like(w, 3.0))
    assert none[0].numel() == 0 and (none[2] == 0).all() and (none[3] == 0).all()


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_against_differences(inter):
    """d/dt of sum(g y(x + t e)) at 0, in 64 bits, for a few directions e of x and of the weight."""
    q, _ = layouts("plain", 1, 3, 2, 0, 64, "fp32")
    g, _ = layouts("plain", 1, 3, 2, 0, 64, "fp32", tag="grad")
    w = act(64, tag="w", dtype="fp32")
    cos, sin = angles(3, 24)
    gx, _, gw, _ = dit.rmsnorm_rope_backward(g, None, q, None, w, None, cos, sin, interleaved=inter)

    def loss(x, weight):
        y = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * weight
        c, s = cos.double()[:, None], sin.double()[:, None]
        a, b = (y[..., 0:48:2], y[..., 1:48:2]) if inter else (y[..., :24], y[..., 24:48])
        ta, tb = a * c - b * s, b * c + a * s
        turned = torch.stack((ta, tb), -1).flatten(-2) if inter else torch.cat((ta, tb), -1)
        return (g.double() * torch.cat((turned, y[..., 48:]), -1)).sum()

    h = 1e-5
    for seed in range(4):
        e = act(1, 3, 2, 64, tag=f"e{seed}", dtype="fp32").double()
        d = (loss(q.double() + h * e, w.double()) - loss(q.double() - h * e, w.double())) / (2 * h)
        # differences: h^2 of a third derivative, and 2^-52 / h of the losses; gx: fp32 terms
        assert abs(float((gx.double() * e).sum() - d)) <= 1e-5 * float((gx.double() * e).abs().sum())
        e = act(64, tag=f"w{seed}", dtype="fp32").double()
        d = (loss(q.double(), w.double() + h * e) - loss(q.double(), w.double() - h * e)) / (2 * h)
        assert abs(float((gw.double() * e).sum() - d)) <= 1e-5 * float((gw.double() * e).abs().sum())


@pytest.mark.parametrize("D", [128, 33, 1024])
@pytest.mark.parametrize("tokens", [1, 5, 4000])
def test_gradient_workspace(tokens, D):
    q, g, w = act(tokens, 3, D, tag="q"), act(tokens, 3, D, tag="g"), act(D, tag="w")
    cos, sin = angles(tokens, D // 4)
    want = dit.rmsnorm_rope_backward(g, None, q, None, w, None, cos, sin)
    need = dit.library().dit_rmsnorm_rope_backward_workspace_bytes(D)
    buf = torch.full((need + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[4096:4096 + need]
    for fill in (0, 0xFF):
        ws.fill_(fill)
        got = dit.rmsnorm_rope_backward(g, None, q, None, w, None, cos, sin, workspace=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        assert bool((buf[:4096] == 0xA5).all()) and bool((buf[4096 + need:] == 0xA5).all())


def test_broadcast_inputs():
    """An input that repeats itself (stride 0) is read; as an output it is refused."""
    q = act(1, 1, 128, tag="one").expand(6, 4, 128)
    w = act(128, tag="w")
    cos, sin = angles(6, 64)
    y, _ = dit.rmsnorm_rope(q, None, w, None, cos, sin)
    assert torch.equal(y, dit.rmsnorm_rope(q.contiguous(), None, w, None, cos, sin)[0])
    with pytest.raises(dit.DitError):
        dit.rmsnorm_rope(q, None, w, None, cos, sin, out_q=q)
    back = dit.rmsnorm_rope_backward(q, None, q, None, w, None, cos, sin)
    assert back[0].shape == q.shape and np.isfinite(f64(back[0])).all()
