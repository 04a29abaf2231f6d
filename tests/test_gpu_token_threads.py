"""The token-transformer operators from several host threads at once, each on a
stream of its own: the bits of one thread's calls made alone."""
import threading

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built

pytestmark = pytest.mark.gpu


def test_calls_of_several_threads():
    ensure_built()
    g = torch.Generator(device="cuda").manual_seed(11)
    rand = lambda *s, t: torch.randn(s, generator=g, device="cuda").to(t)
    cases = []
    for t, rows, D in ((torch.bfloat16, 100, 1000), (torch.float16, 900, 257),
                       (torch.float32, 300, 2048), (torch.bfloat16, 7, 20001)):
        ids = torch.randint(-1, 50, (rows,), generator=g, device="cuda")
        cases.append((rand(rows, D, t=t), rand(rows, D, t=t), rand(D, t=t), ids))

    def work(case):
        x, u, w, ids = case
        r, o = dit.add_rmsnorm(x, u, w)
        _, q, s = dit.add_rmsnorm_fp8(x, u, w, group=128)
        gx, gw = dit.rmsnorm_backward(u, r, w, grad_residual=o)
        gt = dit.embedding_backward(gx, ids, 50)
        e = dit.embedding(ids, gt)
        (a, b), norm = dit.clip_grads([gt, gw], 1.0)
        return [r, o, q.view(torch.uint8), s, gx, gw, gt, e, a, b, norm]

    want = [work(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got, errors = [None] * len(cases), []
    start = threading.Barrier(len(cases))

    def run(i):
        try:
            start.wait(60)
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    got[i] = work(cases[i])
        except Exception as e:  # reported below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not errors, errors
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x.flatten().view(torch.uint8), y.flatten().view(torch.uint8))
