"""The first calls of a process, made while a graph is being captured: nothing
of the token-transformer operators needs a call before."""
import os
import subprocess
import sys

import pytest

from _gpu import ensure_built

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
import diffusion_transformer_elementwise_gb300 as dit

g = torch.Generator(device="cuda").manual_seed(5)
rand = lambda *s, t=torch.bfloat16: torch.randn(s, generator=g, device="cuda").to(t)
cases = []
for t, rows, D in ((torch.bfloat16, 300, 1024), (torch.float32, 70, 513), (torch.float16, 3, 40000)):
    cases.append((rand(rows, D, t=t), rand(rows, D, t=t), rand(D, t=t)))
ids = torch.randint(-1, 900, (5000,), generator=g, device="cuda")
table, gt = rand(900, 257), rand(5000, 257)
grads = [rand(n, t=torch.float32) for n in (5, 70000, 333)]

def work():
    out = []
    for x, u, w in cases:
        out += [dit.rmsnorm(x, w), *dit.add_rmsnorm(x, u, w), *dit.rmsnorm_backward(u, x, w)]
        out += [*dit.rmsnorm_fp8(x, w), *dit.add_rmsnorm_fp8(x, u, w, group=128)]
    out += [dit.embedding(ids, table), dit.embedding_backward(gt, ids, 900),
            dit.embedding_backward(gt[:100], ids[:100], 900), dit.grad_norm(grads)]
    clipped, norm = dit.clip_grads(grads, 0.5)
    return out + [*clipped, norm]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = work()
graph.replay()
torch.cuda.synchronize()
same = lambda a, b: torch.equal(a.reshape(-1).view(torch.uint8), b.reshape(-1).view(torch.uint8))
assert all(same(a, b) for a, b in zip(captured, work(), strict=True))
print("captured", len(captured))
"""


def test_first_calls_are_captured():
    ensure_built()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("captured"), r.stdout + r.stderr
