"""The 64-bit reference of the token-transformer operators against itself
(CPU): its gradients against differences, its E4M3 check against planted
mistakes."""
import numpy as np
import pytest
import torch

import _token_ref as ref

RNG = np.random.default_rng(11)


def test_gradient_against_differences():
    x, g, w, k = (RNG.standard_normal(s) for s in ((5, 12), (5, 12), (12,), (5, 12)))
    gx, _, gw, _ = ref.norm_grad(g, x, w, 1e-3, 1.0, k)

    def loss(x, w):
        return (ref.norm(x, w, 1e-3, 1.0) * g).sum() + (x * k).sum()

    h = 1e-6
    for i in range(5):
        for j in range(12):
            d = np.zeros_like(x)
            d[i, j] = h
            assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * h) - gx[i, j]) < 1e-7
    for j in range(12):
        d = np.zeros_like(w)
        d[j] = h
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * h) - gw[j]) < 1e-7


def test_fp8_check_sees_a_wrong_code_and_scale():
    x = torch.from_numpy(RNG.standard_normal((3, 300))).float()
    w = torch.ones(300)
    y = ref.norm(ref.f64(x), np.ones(300), 1e-6, 0.0)
    s = np.abs(y[:, :]).max(1, keepdims=True) / 448
    q = torch.from_numpy(y / s).float().to(torch.float8_e4m3fn)
    st = torch.from_numpy(s).float()
    ref.check_fp8(q, st, x, w, 1e-6, 0.0, 0)
    bad = q.view(torch.uint8).clone()
    bad[1, 7] ^= 1
    with pytest.raises(AssertionError):
        ref.check_fp8(bad, st, x, w, 1e-6, 0.0, 0)
    with pytest.raises(AssertionError):
        ref.check_fp8(q, st * (1 + 1e-5), x, w, 1e-6, 0.0, 0)


def test_close_check_sees_differences():
    t = torch.tensor([1.0, float("nan"), float("inf")])
    ref.check_close(t, np.array([1.0, np.nan, np.inf]), 0.0)
    for want in ([1.0 + 1e-7, np.nan, np.inf], [1.0, 0.0, np.inf], [1.0, np.nan, 3.0]):
        with pytest.raises(AssertionError):
            ref.check_close(t, np.array(want), 1e-9)
