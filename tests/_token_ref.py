"""The token-transformer operators in 64 bits, element by element from their
formulas (include/dit_elementwise.h), and the tolerances of the kernels' fp32
arithmetic.  CPU, numpy; shares no code with the library.

Tolerances count roundings, u = 2^-24 each.  The row statistic's r is within
17 u (the fast statistic's stated bound), so a product of r with two more
rounded factors is within 20 u < 2^-19 of its exact value; REL = 2^-18 leaves
a factor of two for the second order.  A result stored in a dtype is off by half a
step of the dtype more, at least half of its smallest subnormal.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
REL = 2.0 ** -18
HALF = {torch.bfloat16: 2.0 ** -9, torch.float16: 2.0 ** -12, torch.float32: 2.0 ** -25}
# half of a step relative to a value at the bottom of its binade
REL_HALF = {k: 2 * v for k, v in HALF.items()}
SUB_HALF = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def rounding(v, dtype):
    """The most that storing v in the dtype moves it."""
    return REL_HALF[dtype] * np.abs(v) + SUB_HALF[dtype]


def residual(hidden, update):
    """hidden + update in fp32, rounded to the dtype."""
    return (hidden.cpu().float() + update.cpu().float()).to(hidden.dtype)


def inverse_rms(x, eps):
    """1 / sqrt(mean(x^2) + eps) per row; a mean square past fp32's range
    counts as infinite (the statistic is held in fp32)."""
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        ms = (x * x).mean(-1, keepdims=True)
        ms = np.where(ms >= 2.0 ** 128, np.inf, ms)
        return 1.0 / np.sqrt(ms + float(np.float32(eps)))


def norm(x, weight, eps, offset):
    """y of a [rows, D] array."""
    with np.errstate(invalid="ignore", over="ignore"):
        return x * inverse_rms(x, eps) * (weight + float(np.float32(offset)))


def check_close(got, want, tol, what=""):
    """|got - want| <= tol with NaN at the same places, infinities alike."""
    got = f64(got).reshape(np.shape(want))
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN at other places"
    with np.errstate(invalid="ignore"):
        bad = ~np.isnan(want) & ~(np.abs(got - want) <= tol) & ~(got == want)
    at = np.argwhere(bad)
    assert at.size == 0, (f"{what}: {len(at)} elements off, first {at[0]}: got {got[tuple(at[0])]!r} "
                          f"want {want[tuple(at[0])]!r} tolerance {np.broadcast_to(tol, bad.shape)[tuple(at[0])]!r}")


def check_norm(got, x, weight, eps, offset, what=""):
    want = norm(f64(x), f64(weight), eps, offset)
    with np.errstate(invalid="ignore"):
        tol = REL * np.abs(want) + rounding(want, got.dtype)
    check_close(got, want, tol, what)


def check_fp8(codes, scales, x, weight, eps, offset, group, what=""):
    """Scales within 24 u of the exact ones (r 17, the maximum's two factors
    and the scale's two operations); a code at most half an E4M3 step (step
    2^(e-3), at least 2^-9) from the exact y / scale, moved by at most 2^-21
    of itself (six roundings: r does not enter)."""
    y = norm(f64(x), f64(weight), eps, offset)
    rows, D = y.shape
    g = group or D
    c = f64(codes.view(torch.float8_e4m3fn).float()).reshape(rows, D)
    s = f64(scales).reshape(rows, -1)
    assert s.shape[1] == -(-D // g)
    for k in range(s.shape[1]):
        part, code = y[:, k * g:(k + 1) * g], c[:, k * g:(k + 1) * g]
        m = np.max(np.abs(part), axis=1, keepdims=True)  # NaN if any is
        want = m / 448.0
        check_close(scales.reshape(rows, -1)[:, k:k + 1], want, 24 * U * want + 2.0 ** -149, what + " scale")
        with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
            v = np.where(m == 0, 0.0, part / want)
        nan = np.isnan(v)
        assert np.array_equal(nan, np.isnan(code)), f"{what}: NaN codes at other places"
        v, code = v[~nan], code[~nan]
        big = np.maximum(np.abs(v), np.abs(code))
        _, e = np.frexp(big)
        step = np.ldexp(1.0, np.maximum(e - 4, -9))
        bad = np.abs(v - code) > step / 2 + np.abs(v) * 2.0 ** -21
        assert not bad.any(), f"{what}: {bad.sum()} codes off, first {code[bad][0]} for {v[bad][0]}"


def norm_grad(g, x, weight, eps, offset, skip=None):
    """(gx, the size of what it is a difference of, gw, the sum of its terms'
    sizes), by the quotient rule."""
    w = weight + float(np.float32(offset))
    r = inverse_rms(x, eps)
    D = x.shape[-1]
    n = x * r
    t = g * w
    k = (t * n).mean(-1, keepdims=True)
    gx = r * (t - n * k)
    size = np.abs(r * t) + np.abs(r * n) * (np.abs(t * n).sum(-1, keepdims=True) / D)
    if skip is not None:
        gx = gx + skip
        size = size + np.abs(skip)
    return gx, size, (g * n).sum(0), np.abs(g * n).sum(0)


def check_norm_grad(gx, gw, g, x, weight, eps, offset, skip=None, what=""):
    """gx: its two terms carry r and a sum of D products in tree order, all
    within REL of the terms' sizes.  gw: the same per term, and one rounding per addition
    -- rows over at least 152 CTAs, then at most 8 teams, 19 rows of partial sums and 32
    of them."""
    rows = x.reshape(-1, x.shape[-1]).shape[0]
    ex, size, ew, wsize = norm_grad(f64(g), f64(x), f64(weight), eps, offset,
                                    None if skip is None else f64(skip))
    check_close(gx, ex, REL * size + rounding(ex, gx.dtype), what + " gx")
    if gw is not None:
        adds = -(-rows // 152) + 8 + 19 + 32
        check_close(gw, ew, (REL + adds * U) * wsize + rounding(ew, gw.dtype), what + " gw")


def check_embedding_grad(got, g, ids, V, scale, what=""):
    """A row's sum in fp32: at most 32 additions in a segment and one per
    segment of 32, and the scale's product."""
    g, ids = f64(g).reshape(ids.numel(), -1), ids.cpu().numpy().reshape(-1).astype(np.int64)
    s = float(np.float32(scale))
    want = np.zeros((V, g.shape[1]))
    size = np.zeros_like(want)
    ok = (ids >= 0) & (ids < V)
    np.add.at(want, ids[ok], g[ok])
    np.add.at(size, ids[ok], np.abs(g[ok]))
    n = np.bincount(ids[ok], minlength=V)[:, None] if V else np.zeros((0, 1))
    want, size = want * s, size * abs(s)
    tol = (np.minimum(n, 32) + n / 32 + 4) * U * size + np.where(n > 0, rounding(want, got.dtype), 0.0)
    check_close(got, want, tol, what)


def check_clip(norm, outs, grads, max_norm=None, eps=1e-6, what=""):
    """The norm: chains of at most 20 additions in fp32 (then fp64), halved by
    the root, and its own rounding: 12 u.  The factor adds two roundings, the product
    one."""
    total = sum(float((f64(g) ** 2).sum()) for g in grads)
    want = np.sqrt(total)
    check_close(norm.reshape(()), np.float64(want), 12 * U * want + 2.0 ** -149, what + " norm")
    if outs is None:
        return
    c = min(1.0, float(np.float32(max_norm)) / (want + float(np.float32(eps))))
    for i, (o, g) in enumerate(zip(outs, grads)):
        v = f64(g) * c
        check_close(o, v, 16 * U * np.abs(v) + rounding(v, o.dtype), f"{what} out {i}")
