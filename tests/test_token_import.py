"""The package imports, and refuses what it refused, in a torch that lacks the
private names the bindings take where there are any."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import diffusion_transformer_elementwise_gb300 as dit
x = torch.zeros(2, 8)
for call in (lambda: dit.rmsnorm(x, x[0]), lambda: dit.residual_gate_add(x[None], x[None], x[None])):
    try:
        call()
    except TypeError:
        continue
    raise AssertionError("a CPU tensor was accepted")
print("imported")
"""


def test_without_torch_private_names():
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout == "imported\n", r.stdout + r.stderr
