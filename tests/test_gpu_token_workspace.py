"""The workspaces of the token-transformer operators: nothing is written past
the size that the _workspace_bytes functions give (a canary behind it), what they
hold at the start does not matter, and a workspace may be used again by the
next call on its stream."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
PAD = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


class Guarded:
    """A workspace of exactly `nbytes` between canaries, filled with `fill`."""

    def __init__(self, nbytes, fill):
        self.buf = torch.full((nbytes + 2 * PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.ws = self.buf[PAD:PAD + nbytes]
        self.ws.fill_(fill)

    def intact(self):
        return bool((self.buf[:PAD] == 0xA5).all()) and \
            bool((self.buf[PAD + self.ws.numel():] == 0xA5).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 20001), (3, 8200), (129, 33), (130, 129), (150, 1001), (153, 64), (400, 77),
                                    (5, 4096), (2, 20001)])
def test_norm_backward(rows, D, dtype):
    x, g = (draw("act", (rows, D), seed_for("ws", k, rows, D), dtype, "cuda") for k in "xg")
    w = draw("act", (D,), seed_for("ws", "w", D), dtype, "cuda")
    want = dit.rmsnorm_backward(g, x, w)
    n = dit.library().dit_rmsnorm_backward_workspace_bytes(rows, D)
    for fill in (0, 0xFF):
        ws = Guarded(n, fill)
        for _ in range(2):
            got = dit.rmsnorm_backward(g, x, w, workspace=ws.ws)
            torch.cuda.synchronize()
            assert ws.intact()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("n,V,D", [(257, 50, 33), (300, 3, 64), (5000, 900, 24), (4097, 1, 129),
                                   (6400, 5000, 8)])
def test_embedding_backward(n, V, D):
    g = draw("act", (n, D), seed_for("ws", "e", n, D), "bf16", "cuda")
    u = draw("gate", (n,), seed_for("ws", "ids", n), "fp32", "cuda")
    ids = ((u.double() + 1) * 0.5 * (V + 1)).long() - 1
    want = dit.embedding_backward(g, ids, V)
    need = dit.library().dit_embedding_backward_workspace_bytes(n, D)
    for fill in (0, 0xFF):
        ws = Guarded(need, fill)
        for _ in range(2):
            got = dit.embedding_backward(g, ids, V, workspace=ws.ws)
            torch.cuda.synchronize()
            assert ws.intact() and torch.equal(got, want)


@pytest.mark.parametrize("count,n", [(1, 3), (64, 5000), (65, 5000), (1000, 700), (3, 40_000_000)])
def test_clip(count, n):
    flat = draw("act", (count * n,), seed_for("ws", "c", count, n), "bf16", "cuda")
    gs = [flat[i * n:(i + 1) * n] for i in range(count)]
    outs = torch.empty_like(flat)
    lst = dit.TensorList(gs, [outs[i * n:(i + 1) * n] for i in range(count)])
    norm = dit.clip_grads(lst, 1.0)[1]
    want = outs.clone()
    need = dit.library().dit_grad_norm_workspace_bytes(count)
    for fill in (0, 0xFF):
        ws = Guarded(need, fill)
        for _ in range(2):
            again = dit.clip_grads(lst, 1.0, workspace=ws.ws)[1]
            only = dit.grad_norm(lst, workspace=ws.ws)
            torch.cuda.synchronize()
            assert ws.intact() and torch.equal(outs, want)
            assert float(again) == float(norm) == float(only)
