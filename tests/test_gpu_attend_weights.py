"""Weights of attention that differ by many powers of two, and values that differ the other way: what counts is a
token's weight times its value, whatever the largest weight and the largest value are.

The logits are one product each (queries and keys have one column that is not zero), so that they are known to a few
roundings, and the outputs' error is that of the weights."""
import math

import numpy as np
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import f64
from _gpu import ensure_built
from _token_ref import U, check_close, rounding

pytestmark = pytest.mark.gpu
T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Rows:
    """A sequence of `n` tokens: logit[t] for even query heads and -logit[t] for odd ones, and value rows whose
    largest magnitude is size[t].  The logits are multiples of 1/2 up to 100 in magnitude, the product of a query of
    1 or -1 and a key (E4M3: a code of 1 and its scale).  `B` sequences share the
    pages: the more there are, the longer is the part of one that a warp has."""

    def __init__(self, logit, size, D, Hq, dtype, fp8, seed=0, B=1):
        n, page = len(logit), 16
        g = torch.Generator().manual_seed(seed + n)
        pages = -(-n // page) + 1
        v = torch.rand(n, D, generator=g, dtype=torch.float64) * 2 - 1
        v[:, 0] = 1.0
        size = torch.tensor(size, dtype=torch.float64)
        signs = [1.0 if h % 2 == 0 or dtype == "fp16" else -1.0 for h in range(Hq)]
        if dtype == "fp16":  # (one sign, and an output of less than 2^10)
            p = torch.tensor(logit, dtype=torch.float64).softmax(0)
            size = size * 2.0 ** min(0, 10 - math.frexp(float((p * size).sum()))[1])
        k = torch.zeros(n, D, dtype=torch.float64)
        k[:, D // 2] = torch.tensor(logit, dtype=torch.float64)
        order = torch.randperm(pages, generator=g)[:pages - 1]
        self.pages = order[None].int().repeat(B, 1).cuda()
        t = torch.arange(n)
        at = (order[t // page], torch.zeros(n, dtype=torch.long), t % page)
        shape = (pages, 1, page, D)
        if fp8:
            # a key's code is 1, its scale the logit; codes of values up to 1, scales their size (powers of two)
            kc, vc = (torch.full(shape, 0x7F, dtype=torch.uint8) for _ in "kv")
            ks, vs = (torch.full(shape[:3], math.nan) for _ in "kv")
            one = torch.zeros(n, D)
            one[:, D // 2] = 1.0
            kc[at], vc[at] = (x.to(torch.float8_e4m3fn).view(torch.uint8) for x in (one, v.float()))
            ks[at], vs[at] = k[:, D // 2].float(), size.float()
            self.cache = dit.KVCache(kc.cuda(), vc.cuda(), ks.cuda(), vs.cuda())
            self.v = f64(v.float().to(torch.float8_e4m3fn).float()) * f64(vs[at])[:, None]
        else:
            kc, vc = (torch.full(shape, math.nan, dtype=T[dtype]) for _ in "kv")
            kc[at], vc[at] = k.to(T[dtype]), (v * size[:, None]).to(T[dtype])
            self.cache = dit.KVCache(kc.cuda(), vc.cuda())
            self.v = f64(vc[at])
            assert torch.equal(kc[at].double(), k), "the logits are held exactly"
        q = torch.zeros(B, Hq, D)
        q[:, :, D // 2] = torch.tensor(signs)
        self.signs = signs
        self.q, self.logit = q.to(T[dtype]).cuda(), np.array(logit)
        self.lengths = torch.tensor([n] * B).cuda()
        self.size = f64(size)

    def check(self, window=0):
        """A logit of magnitude S is off by 8 u S and a weight by its exponential's 2^-21 more; the output by that
        share of sum p |v| twice (its own and the sum's), by its weights' rounding to fp16 (half a step, 2^-11 of
        each: fp16 caches, and bf16 queries over E4M3; bf16 caches 2^-8; two parts of fp16 or tf32 2^-19: fp32 queries, and
        fp16 ones over E4M3), and, where the weights are fp16, by what they cannot hold:
        they are kept in units that put the largest weight times its row's scale at 2^12 and more, so a token loses
        2^-25 / 2^12 of that, times its codes (at most 1), at most."""
        out, lse = dit.paged_attention(self.q, self.cache, self.pages, self.lengths, scale=1.0, window=window,
                                       need_lse=True)
        fp8 = self.cache.k_scales is not None
        dtype = self.q.dtype
        share = 2.0 ** -19
        if dtype is not torch.float32 and not (fp8 and dtype is torch.float16):
            share = 2.0 ** -8 if dtype is torch.bfloat16 and not fp8 else 2.0 ** -11
        lo = len(self.logit) - window if window else 0
        v, size = self.v[lo:], self.size[lo:]
        for h in range(self.q.shape[1]):
            s = self.logit[lo:] * self.signs[h]
            p = np.exp(s - s.max())
            wl = s.max() + math.log(p.sum())
            p /= p.sum()
            want, terms = p @ v, p @ np.abs(v)
            logit = 8 * U * np.abs(s).max()
            tol = (2 * (logit + 2.0 ** -20) + share) * terms + rounding(want, dtype)
            if share != 2.0 ** -8:
                tol = tol + len(s) * 2.0 ** -37 * (p * size if fp8 else p * size.max()).max()
            B = len(out)
            for b in sorted({0, 1 % B, B // 2, B - 1}):
                check_close(out[b, h], want, tol, f"sequence {b} head {h}")
                check_close(lse[b, h].reshape(()), np.float64(wl), logit + 2.0 ** -20 * (1 + abs(wl)), f"lse {b} {h}")


def spread(n, make):
    return [make(i) for i in range(n)]


def near(n):
    return spread(n, lambda i: (i % 7) * 0.5)


# name: logits and the sizes of the values' rows (powers of two)
KINDS = {
    # one row of large values that has next to no weight, first, last, and in the middle
    "large first": lambda n: ([-40.0] + near(n - 1), [2.0 ** 20] + [1.0] * (n - 1)),
    "large last": lambda n: (near(n - 1) + [-40.0], [1.0] * (n - 1) + [2.0 ** 20]),
    "large between": lambda n: (near(n // 2) + [-60.0] + near(n - n // 2 - 1),
                                [1.0] * (n // 2) + [2.0 ** 40] + [1.0] * (n - n // 2 - 1)),
    # the token with all the weight has small values
    "small first": lambda n: ([16.0] + [0.0] * (n - 1), [2.0 ** -10] + [1.0] * (n - 1)),
    "small last": lambda n: ([0.0] * (n - 1) + [80.0], [2.0 ** 26] * (n - 1) + [1.0]),
    # a maximum that rises little by little, over a first row that was large
    "rising": lambda n: (spread(n, lambda i: min(100.0, (i // 32) * 0.5)), [2.0 ** 30] + [1.0] * (n - 1)),
    "falling": lambda n: (spread(n, lambda i: max(-100.0, -(i // 32) * 0.5)), spread(n, lambda i: 2.0 ** min(40, i // 64))),
    # sizes over all of the range
    "any": lambda n: (spread(n, lambda i: (i * 37 % 160 - 80) * 0.5), spread(n, lambda i: 2.0 ** (i * 11 % 81 - 40))),
}


@pytest.mark.parametrize("n", [2, 33, 700, 6000])
@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("kind", KINDS)
def test_e4m3(kind, dtype, n):
    for D, Hq in ((64, 2), (128, 6), (256, 2), (128, 16), (48, 12), (40, 2)):
        rows = Rows(*KINDS[kind](n), D, Hq, dtype, True)
        rows.check()
        if n == 700:
            rows.check(window=650)


@pytest.mark.parametrize("n", [2, 700, 6000])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_caches_of_the_dtype(kind, dtype, n):
    for D, Hq in ((64, 2), (128, 16), (33, 2)):
        Rows(*KINDS[kind](n), D, Hq, dtype, False).check()


@pytest.mark.parametrize("dtype", T)
@pytest.mark.parametrize("kind", KINDS)
def test_long_parts(kind, dtype):
    """A warp has some three thousand tokens of a sequence, one tile after the other."""
    Rows(*KINDS[kind](9000), 64, 2, dtype, True, B=400).check()


@pytest.mark.parametrize("D,Hq", [(64, 2), (128, 6), (256, 2), (128, 16), (33, 2)])
@pytest.mark.parametrize("fp8", [False, True])
def test_fp16_weights(D, Hq, fp8):
    """Tokens of 2^-25 of the largest weight and more, whose values are a hundred times its own."""
    n = 20000
    for first in (17.5, 12.0, 9.0):
        Rows([first] + [0.0] * (n - 1), [2.0 ** -7] + [1.0] * (n - 1), D, Hq, "fp16", fp8, B=200).check()
