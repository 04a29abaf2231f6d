"""The operators around attention in 64 bits, element by element from their
formulas (include/dit_elementwise.h), and the tolerances of the kernels'
arithmetic.  CPU, numpy; shares no code with the library.

Tolerances count roundings, u = 2^-24 each.  The statistic of a head's norm is a sum
of at most 1024 squares in a tree (at most 32 chained additions in a lane and 5 across
lanes; the root halves its error), a product and a reciprocal root of 2 ulp: r is within 25 u.  A normed value carries two products more and the weight's addition, a turned one a product,
a sum and the table's roundings as given (the reference reads the same table): within 31 u of
the two products' sizes.  REL = 2^-18 (64 u) leaves a factor of two for the second order.
A result stored in a dtype is off by half a step more.
"""
from __future__ import annotations

import numpy as np
import torch
from _token_ref import REL, SUB_HALF, U, check_close, f64, rounding


def angles(positions, freqs, sections):
    """[tokens, R] angles modulo a turn, from positions [axes, tokens] and fp64 frequencies.  Products in
    extended precision where the host has it: see angle_error."""
    out, column = [], 0
    for a, n in enumerate(sections):
        out.append(np.outer(positions[a].astype(np.longdouble),
                            freqs[column:column + n].astype(np.longdouble)))
        column += n
    return np.concatenate(out, 1)


def check_table(cos, sin, positions, freqs, sections, what=""):
    """cos and sin within: the frequency in turns (two fp64 roundings, 2^-52 of the angle), the
    integer positions' fraction of a turn (64 bits, rounded: a position of p units multiplies an error of
    2^-65 turns, so 2 pi 2^-65 |p| radians at most), fp32's part of a turn (half an ulp of a
    value below pi: 2^-23), and fp32 sine and cosine of at most 2 ulp and their rounding (2^-23
    of their size and less): 2^-22 in all, and an angle's own uncertainty in 64 bits."""
    p, f = f64(positions).reshape(len(sections), -1), f64(freqs)
    x = angles(p, f, sections)
    size = np.abs(x).astype(np.float64)
    if not positions.is_floating_point():
        axis = np.repeat(np.arange(len(sections)), sections)
        whole = np.abs(p[axis]).T * (2 * np.pi * 2.0 ** -65)
    else:
        whole = 0.0
    for got, want in ((cos, np.cos(x)), (sin, np.sin(x))):
        want = want.astype(np.float64)
        finite = np.isfinite(size)
        want = np.where(finite, want, np.nan)
        tol = 2.0 ** -22 + size * 2.0 ** -51 + whole
        check_close(got, want, np.where(finite, tol, 0.0), what)


def pairs(D, R, interleaved):
    j = np.arange(R)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + R)


def rotate(x, cos, sin, interleaved, inverse=False):
    """(turned, the size of its terms) of [B, L, H, D] by tables that broadcast to [B, L, 1, R]."""
    R = cos.shape[-1]
    c, d = pairs(x.shape[-1], R, interleaved)
    if inverse:
        sin = -sin
    y, size = x.copy(), np.abs(x)
    a, b = x[..., c], x[..., d]
    with np.errstate(invalid="ignore", over="ignore"):
        y[..., c], y[..., d] = a * cos - b * sin, b * cos + a * sin
        size[..., c] = np.abs(a * cos) + np.abs(b * sin)
        size[..., d] = np.abs(b * cos) + np.abs(a * sin)
    return y, size


def table(cos, B, L):
    t = f64(cos)
    return t.reshape((t.shape[0] // L, L, 1, t.shape[-1]))  # [1 or B, L, 1, R]


def four(x):
    x = f64(x)
    return x if x.ndim == 4 else x[None]


def inverse_rms(x, eps):
    with np.errstate(over="ignore", divide="ignore", invalid="ignore"):
        return 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + float(np.float32(eps)))


def check_rope(got, x, cos, sin, weight=None, eps=1e-6, offset=0.0, interleaved=False, inverse=False,
               what=""):
    x4 = four(x)
    B, L = x4.shape[:2]
    n = x4
    if weight is not None:
        n = x4 * inverse_rms(x4, eps) * (f64(weight) + float(np.float32(offset)))
    if cos is None:
        want, size = n, np.abs(n)
    else:
        want, size = rotate(n, table(cos, B, L), table(sin, B, L), interleaved, inverse)
    check_close(got, want.reshape(x.shape), (REL * size).reshape(x.shape)
                + rounding(want, got.dtype).reshape(x.shape), what)


def check_rope_grad(gx, gw, g, x, cos, sin, weight, eps=1e-6, offset=0.0, interleaved=False, what=""):
    """gx: two terms that carry r (twice) and sums of D products in tree order, within REL
    of the terms' sizes.  gw: the same per term, and one rounding per addition: each of at most
    608 CTAs and 8 warps has its part of the rows, then 8 warps' and at most 19 + 5 CTAs'."""
    g4, x4 = four(g), four(x)
    B, L, H, D = x4.shape
    w = f64(weight) + float(np.float32(offset))
    if cos is None:
        u, usize = g4, np.abs(g4)
    else:
        u, usize = rotate(g4, table(cos, B, L), table(sin, B, L), interleaved, inverse=True)
    r = inverse_rms(x4, eps)
    n, t = x4 * r, u * w
    tsize = usize * np.abs(w)
    want = r * (t - n * (t * n).mean(-1, keepdims=True))
    size = r * (tsize + np.abs(n) * (tsize * np.abs(n)).mean(-1, keepdims=True))
    check_close(gx, want.reshape(x.shape),
                (REL * size + rounding(want, gx.dtype)).reshape(x.shape), what + " gx")
    if gw is not None:
        terms = (u * n).reshape(-1, D)
        sizes = (usize * np.abs(n)).reshape(-1, D).sum(0)
        want = terms.sum(0)
        # a chain holds at most the rows a warp takes
        adds = 2 * -(-B * L * H // 152) + 64
        check_close(gw, want, (REL + adds * U) * sizes + rounding(want, gw.dtype), what + " gw")


def e4m3_step(v):
    _, e = np.frexp(np.abs(v))
    return np.ldexp(1.0, np.maximum(e - 4, -9))


def check_rows_e4m3(codes, scales, x, what=""):
    """Scales within a rounding of m / 448; a code at most half a step from x 448 / m (moved by at most
    four roundings: two parts of the quotient, the product's)."""
    x, s = f64(x), f64(scales)
    c = f64(codes.view(torch.float8_e4m3fn).float())
    m = np.abs(x).max(-1)
    want = np.where(np.isfinite(m), m / 448.0, np.nan)
    check_close(scales, want, U * np.abs(want) + SUB_HALF[torch.float32], what + " scale")
    with np.errstate(invalid="ignore", divide="ignore"):
        v = np.where(m[..., None] == 0, 0.0, x * (448.0 / m[..., None]))
    v = np.where(np.isfinite(m)[..., None], v, np.nan)
    assert np.array_equal(np.isnan(v), np.isnan(c)), what + ": NaN codes at other places"
    ok = ~np.isnan(v)
    bad = np.abs(v - c)[ok] > (e4m3_step(np.maximum(np.abs(v), np.abs(c))) / 2 + np.abs(v) * 4 * U)[ok]
    assert not bad.any(), f"{what}: {bad.sum()} codes off"
    assert s.shape == m.shape


def attend(q, k, v, scale):
    """(out, lse, sum of p |v|) of one head: q [D], k and v [tokens, D]."""
    if len(k) == 0:
        return np.zeros(v.shape[1]), -np.inf, np.zeros(v.shape[1])
    s = (k @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    p = p / total
    return p @ v, m + np.log(total), p @ np.abs(v)


def weight_error(dtype, fp8):
    """The most that a weight is moved, relative to it, where weights are rounded for the tensor cores (E4M3: to
    fp16)."""
    if dtype is torch.float32:
        return 2.0 ** -19  # two parts of a number, or none
    return 2.0 ** -11 if fp8 or dtype is torch.float16 else 2.0 ** -8


def check_attention(out, lse, q, k, v, tokens, scale, fp8=False, what=""):
    """out and lse [B, Hq, ...] against rows in 64 bits: k(b, head) and v(b, head) give the values
    of sequence b's tokens that count.  With S = |scale| sum |q k| (the size of a logit's terms)
    a logit is off by (D + 8) u S in the worst order, a weight by as much relative to itself, more by its
    exponential (2^-21) and its rounding (weight_error); the output by that share of
    sum p |v| twice (its own and the sum's), and by what fp16 cannot hold of a weight below 2^-14 of
    the largest (2^-25 of the largest value each)."""
    B, Hq, D = q.shape
    for b in range(B):
        for h in range(Hq):
            kk, vv = k(b, h), v(b, h)
            qq = f64(q[b, h])
            want, wl, size = attend(qq, kk, vv, scale)
            S = float((np.abs(kk) @ np.abs(qq)).max() * abs(scale)) if len(kk) else 0.0
            logit = (D + 8) * U * S + 2.0 ** -22 * S
            rel = 2 * (logit + 2.0 ** -20) + weight_error(q.dtype, fp8)
            tol = rel * size + rounding(want, out.dtype)
            if q.dtype is torch.float16 or fp8:
                tol = tol + len(kk) * 2.0 ** -24 * np.abs(vv).max(initial=0.0)
            check_close(out[b, h], want, tol, f"{what} out {b} {h}")
            if lse is not None:
                check_close(lse[b, h].reshape(()), np.float64(wl),
                            logit + 2.0 ** -20 * (1 + abs(wl) if np.isfinite(wl) else 1), f"{what} lse {b} {h}")
