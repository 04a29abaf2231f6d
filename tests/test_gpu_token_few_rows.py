"""The norm's gradient of few rows, around the bounds of its two forms: one
cluster without a workspace, and two launches that add in it."""
import pytest
import torch

import _token_ref as ref
import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built, guarded
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


# rows, columns, and whether the call adds in the workspace it is given: wide
# rows of more than 2^18 elements do, and all that registers do not hold
@pytest.mark.parametrize("dtype,rows,D,adds", [
    ("bf16", 128, 16384, True), ("fp16", 64, 8200, True), ("bf16", 17, 16384, True),
    ("bf16", 32, 8193, True), ("bf16", 16, 16384, False), ("fp16", 31, 8200, False),
    ("bf16", 1, 16384, False), ("bf16", 128, 8184, False), ("fp32", 128, 8189, False),
    ("fp32", 3, 8200, True), ("fp32", 129, 64, True)])
@pytest.mark.parametrize("skip", [False, True])
def test_the_workspace_is_used_where_the_rule_says(dtype, rows, D, adds, skip):
    x, g, k = (draw("act", (rows, D), seed_for("few", t, rows, D), dtype, "cuda") for t in "xgk")
    w = draw("act", (D,), seed_for("few", "w", D), dtype, "cuda")
    need = dit.library().dit_rmsnorm_backward_workspace_bytes(rows, D)
    ws = torch.full((max(need, 256),), 0xA5, dtype=torch.uint8, device="cuda")
    gx, f1 = guarded((rows, D), x.dtype, "cuda")
    gw, f2 = guarded((D,), x.dtype, "cuda")
    dit.rmsnorm_backward(g, x, w, EPS, grad_residual=k if skip else None, grad_x=gx, grad_weight=gw,
                         workspace=ws)
    torch.cuda.synchronize()
    assert f1() and f2()
    ref.check_norm_grad(gx, gw, g, x, w, EPS, 0.0, k if skip else None)
    assert bool((ws != 0xA5).any()) == adds
    if adds:
        assert need > 0
        with pytest.raises(dit.DitError):
            dit.rmsnorm_backward(g, x, w, EPS, workspace=ws[:need - 1])
