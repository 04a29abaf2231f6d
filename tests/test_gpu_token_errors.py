"""A launch that the CUDA runtime rejects is reported by its own call and by no
later one.  The launches go to a stream whose capture has been invalidated (by
waiting for it, an error that the driver returns): nothing reaches the GPU."""
import ctypes

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built

pytestmark = pytest.mark.gpu
LAUNCH = 7  # DIT_ERR_LAUNCH


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def calls():
    """Calls with their outputs and workspaces given, by what they launch."""
    new = lambda *s, t=torch.float32: torch.zeros(s, dtype=t, device="cuda")
    x, w, gx, gw = new(300, 64), new(64) + 1.0, new(300, 64), new(64)
    ids, table, ws = new(300, t=torch.int64), new(9, 64), new(1 << 20, t=torch.uint8)
    lst, norm = dit.TensorList([x], out=[gx]), new(1)
    return {
        "norm": lambda s: dit.rmsnorm(x, w, out=gx, stream=s),
        "norm_backward_rows": lambda s: dit.rmsnorm_backward(x, x, w, grad_x=gx, grad_weight=gw,
                                                             workspace=ws, stream=s),
        "norm_backward_cluster": lambda s: dit.rmsnorm_backward(
            x[:100], x[:100], w, grad_x=gx[:100], grad_weight=gw, stream=s),
        "embedding": lambda s: dit.embedding(ids, table, out=gx, stream=s),
        "embedding_backward": lambda s: dit.embedding_backward(x, ids, 9, out=table, workspace=ws,
                                                               stream=s),
        "clip": lambda s: dit.clip_grads(lst, 1.0, norm=norm, workspace=ws, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward_rows", "norm_backward_cluster",
                                  "embedding", "embedding_backward", "clip"])
def test_a_rejected_launch_is_not_reported_again(name):
    driver = ctypes.CDLL("libcuda.so.1")
    made = calls()
    for call in made.values():
        call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    handle = ctypes.c_void_p(side.cuda_stream)
    relaxed = 2
    assert driver.cuStreamBeginCapture_v2(handle, relaxed) == 0
    assert driver.cuStreamSynchronize(handle) != 0  # invalidates the capture
    with pytest.raises(dit.DitError) as refused:
        made[name](side)
    graph = ctypes.c_void_p()
    assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
    assert refused.value.status == LAUNCH
    for call in made.values():
        call(None)
        call(side)
    torch.cuda.synchronize()
