"""The token-transformer entry points without a GPU: sizes, types, overlaps
and workspaces are checked on the host before anything is launched.  Pointers
are plain integers that are never dereferenced."""
import ctypes

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from diffusion_transformer_elementwise_gb300 import library
from diffusion_transformer_elementwise_gb300._token import Tensor
from diffusion_transformer_elementwise_gb300.build import build

(OK, NULLP, SHAPE, DTYPE, LAYOUT, ALIAS, EPS, LAUNCH, MISALIGNED, NODEV, BADOP, WORKSPACE,
 BADSTAT, SCALAR, FORMAT, NOMEM) = range(16)
BF16, FP16, FP32 = 0, 1, 2
A = 1 << 20
X, U, W, O, R, S, G, K, WS, IDS = (A * k for k in range(1, 11))
NAN, INF = float("nan"), float("inf")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="the pointers are not real: a valid call would launch")


@pytest.fixture(scope="module")
def lib():
    build()
    return library()


def test_status_strings(lib):
    names = {lib.dit_status_string(k).decode() for k in range(16)}
    assert len(names) == 16 and all(n.startswith("DIT_") for n in names)


def norm(lib, out=O, x=X, w=W, rows=4, D=8, eps=1e-6, off=0.0, dt=BF16):
    return lib.dit_rmsnorm(out, x, w, rows, D, eps, off, dt, None)


def add(lib, r=R, out=O, x=X, u=U, w=W, rows=4, D=8, eps=1e-6, off=0.0, dt=BF16):
    return lib.dit_add_rmsnorm(r, out, x, u, w, rows, D, eps, off, dt, None)


def add8(lib, r=R, out=O, s=S, x=X, u=U, w=W, rows=4, D=8, group=0, eps=1e-6, off=0.0, dt=BF16):
    return lib.dit_add_rmsnorm_fp8(r, out, s, x, u, w, rows, D, group, eps, off, dt, None)


def test_norm(lib):
    assert norm(lib) == NODEV and add(lib) == NODEV and add8(lib) == NODEV
    assert lib.dit_rmsnorm_fp8(O, S, X, W, 4, 8, 128, 1e-6, 0.0, BF16, None) == NODEV
    assert norm(lib, dt=3) == DTYPE and add8(lib, dt=-1) == DTYPE
    for bad in (dict(rows=-1), dict(D=-1), dict(D=(1 << 24) + 1), dict(rows=1 << 31)):
        assert norm(lib, **bad) == SHAPE and add(lib, **bad) == SHAPE and add8(lib, **bad) == SHAPE
    for e in (-1e-6, NAN, INF):
        assert norm(lib, eps=e) == EPS and add8(lib, eps=e) == EPS
    for e in (NAN, INF, -INF):
        assert norm(lib, off=e) == SCALAR
    for g in (-1, 1, 64, 256):
        assert add8(lib, group=g) == FORMAT
        assert lib.dit_rmsnorm_fp8(O, S, X, W, 4, 8, g, 1e-6, 0.0, BF16, None) == FORMAT
    assert norm(lib, rows=0, out=None, x=None, w=None) == OK
    assert add8(lib, D=0, r=None, out=None, s=None, x=None, u=None, w=None) == OK
    for n in ("out", "x", "w"):
        assert norm(lib, **{n: None}) == NULLP
    for n in ("r", "out", "s", "x", "u", "w"):
        assert add8(lib, **{n: None}) == NULLP
    assert norm(lib, x=X + 1) == MISALIGNED and norm(lib, x=X + 2, dt=FP32) == MISALIGNED
    assert norm(lib, x=X + 2) == NODEV
    assert add8(lib, out=O + 1) == NODEV      # codes are bytes
    assert add8(lib, s=S + 2) == MISALIGNED


def test_norm_overlaps(lib):
    b = 4 * 8 * 2
    assert add(lib, r=X) == NODEV             # the residual in place
    assert add(lib, r=X + 2) == ALIAS
    assert add(lib, r=U) == ALIAS and add(lib, out=X) == ALIAS and add(lib, out=R) == ALIAS
    assert norm(lib, out=X) == ALIAS and norm(lib, out=W) == ALIAS
    assert norm(lib, out=X + b) == NODEV and norm(lib, out=X + b - 2) == ALIAS
    assert add8(lib, r=X) == NODEV and add8(lib, out=X + b - 1) == ALIAS
    assert add8(lib, s=O + 4 * 8) == NODEV and add8(lib, s=O + 4 * 8 - 4) == ALIAS
    assert add8(lib, s=X) == ALIAS and add8(lib, out=W) == ALIAS
    # scales per 128 columns take more room
    assert add8(lib, D=256, group=128, s=S, out=S + 4 * 2 * 4 - 8) == ALIAS
    assert add8(lib, D=256, group=0, s=S, out=S + 4 * 4) == NODEV


def back(lib, gx=O, gw=S, g=G, k=K, x=X, w=W, rows=4, D=8, eps=1e-6, off=0.0, dt=BF16, ws=WS,
         n=None):
    n = lib.dit_rmsnorm_backward_workspace_bytes(rows, D) if n is None else n
    return lib.dit_rmsnorm_backward(gx, gw, g, k, x, w, rows, D, eps, off, dt, ws, n, None)


def test_norm_backward(lib):
    wb = lib.dit_rmsnorm_backward_workspace_bytes
    assert wb(10_000, 4096) == 304 * 4096 * 4 and wb(129, 8) == 4352
    assert wb(128, 8189) == wb(0, 8) == 0 and wb(1, 8190) == 32768  # few rows need none
    assert wb(-1, 8) == -1 and wb(1, 1 << 25) == -1 and wb(1 << 31, 8) == -1
    assert back(lib) == NODEV and back(lib, k=None) == NODEV
    assert back(lib, gw=None, ws=None, n=0) == NODEV      # a frozen weight
    assert back(lib, rows=0, gw=None) == OK and back(lib, D=0) == OK
    assert back(lib, rows=0, gx=None, g=None, k=None, x=None, w=None) == NODEV  # gw is still written
    for name in ("gx", "g", "x", "w"):
        assert back(lib, **{name: None}) == NULLP
    assert back(lib, ws=None) == NODEV
    assert back(lib, rows=200, ws=None) == WORKSPACE and back(lib, rows=200, ws=WS + 16) == WORKSPACE
    assert back(lib, rows=200, n=wb(200, 8) - 1) == WORKSPACE
    assert back(lib, dt=4) == DTYPE and back(lib, rows=-1, n=0) == SHAPE
    assert back(lib, eps=-1.0) == EPS and back(lib, off=NAN) == SCALAR
    assert back(lib, g=G + 1) == MISALIGNED and back(lib, gw=S + 1) == MISALIGNED
    assert back(lib, gx=G) == NODEV and back(lib, gx=K) == NODEV
    assert back(lib, gx=G + 16) == ALIAS and back(lib, gx=X) == ALIAS and back(lib, gx=W) == ALIAS
    assert back(lib, gw=W) == ALIAS and back(lib, gw=O) == ALIAS and back(lib, gw=G) == ALIAS
    assert back(lib, rows=200, ws=X) == ALIAS and back(lib, rows=200, ws=O) == ALIAS


def test_embedding(lib):
    def f(out=O, ids=IDS, t=X, n=4, V=10, D=8, scale=1.0, dt=BF16, it=1):
        return lib.dit_embedding(out, ids, t, n, V, D, scale, dt, it, None)
    assert f() == NODEV and f(it=0, ids=IDS + 4) == NODEV
    assert f(it=2) == FORMAT and f(dt=3) == DTYPE
    assert f(n=-1) == SHAPE and f(V=-1) == SHAPE and f(V=1 << 31) == SHAPE and f(D=(1 << 24) + 1) == SHAPE
    assert f(scale=NAN) == SCALAR and f(scale=INF) == SCALAR
    assert f(n=0, out=None, ids=None, t=None) == OK
    assert f(V=0, t=None) == NODEV            # every row is zero
    assert f(out=None) == NULLP and f(ids=None) == NULLP and f(t=None) == NULLP
    assert f(ids=IDS + 4) == MISALIGNED and f(out=O + 1) == MISALIGNED
    assert f(out=X) == ALIAS and f(out=IDS) == ALIAS


def test_embedding_backward(lib):
    wb = lib.dit_embedding_backward_workspace_bytes
    # pairs twice, the list of runs (a count and 32 entries), 2 * 32 partial rows
    assert wb(1000, 64) == 2 * 8192 + 256 + 2 * 32 * 64 * 4 and wb(256, 64) == wb(0, 64) == 0
    assert wb(-1, 64) == -1 and wb(1, 1 << 25) == -1

    def f(gt=O, g=G, ids=IDS, n=4, V=10, D=8, scale=1.0, dt=BF16, it=1, ws=WS, b=None):
        return lib.dit_embedding_backward(gt, g, ids, n, V, D, scale, dt, it, ws,
                                          wb(n, D) if b is None else b, None)
    assert f() == NODEV
    assert f(n=0, g=None, ids=None, ws=None) == NODEV     # all zeros are still written
    assert f(V=0, gt=None) == OK and f(D=0) == OK
    assert f(it=-1) == FORMAT and f(dt=9) == DTYPE and f(scale=NAN) == SCALAR
    assert f(n=-1, b=0) == SHAPE and f(V=-2) == SHAPE
    assert f(gt=None) == NULLP and f(g=None) == NULLP and f(ids=None) == NULLP
    assert f(ws=None) == NODEV                # few tokens need none
    assert f(n=1000) == NODEV
    assert f(n=1000, ws=None) == WORKSPACE and f(n=1000, ws=WS + 8) == WORKSPACE
    assert f(n=1000, b=wb(1000, 8) - 1) == WORKSPACE
    assert f(ids=IDS + 4) == MISALIGNED
    assert f(gt=G) == ALIAS and f(gt=IDS) == ALIAS
    assert f(n=1000, gt=WS) == ALIAS and f(n=1000, ws=G) == ALIAS and f(n=1000, ws=IDS) == ALIAS


def descs(*d):
    return ctypes.addressof(_keep((Tensor * max(1, len(d)))(*[Tensor(*t) for t in d])))


_kept = []


def _keep(a):
    _kept.append(a)
    return a


def test_clip(lib):
    wb = lib.dit_grad_norm_workspace_bytes
    assert wb(0) == wb(1) == wb(960) == 1216 * 8 and wb(961) == 2 * 1216 * 8 and wb(-1) == -1

    def f(*d, count=None, m=1.0, eps=1e-6, norm=S, ws=WS, b=None):
        n = len(d) if count is None else count
        return lib.dit_clip_grads(norm, descs(*d), n, m, eps, ws, wb(n) if b is None else b, None)

    def g(*d, norm=S):
        return lib.dit_grad_norm(norm, descs(*d), len(d), WS, wb(len(d)), None)
    t = (G, O, 100, BF16)
    assert f(t) == NODEV and g(t) == NODEV and g((G, None, 100, FP32)) == NODEV
    assert f((G, G, 100, BF16)) == NODEV                  # in place
    assert f((None, None, 0, BF16), t) == NODEV
    assert f(t, count=-1, b=0) == SHAPE and f((G, O, -1, BF16)) == SHAPE
    assert f((G, O, 1 << 50, BF16)) == SHAPE
    assert f((G, O, 10, 3)) == DTYPE
    for m in (-1.0, NAN, INF):
        assert f(t, m=m) == SCALAR
    assert f(t, eps=-1.0) == EPS
    assert f((None, O, 10, BF16)) == NULLP and f((G, None, 10, BF16)) == NULLP
    assert f(t, norm=None) == NULLP
    assert f((G + 1, O, 10, BF16)) == MISALIGNED and f(t, norm=S + 2) == MISALIGNED
    assert f(t, ws=None) == WORKSPACE and f(t, b=100) == WORKSPACE and f(t, ws=WS + 8) == WORKSPACE
    # outputs against inputs, outputs, the norm and the workspace
    assert f((G, G + 2, 100, BF16)) == ALIAS
    assert f((G, O, 100, BF16), (K, O + 198, 100, BF16)) == ALIAS
    assert f((G, O, 100, BF16), (K, O + 200, 100, BF16)) == NODEV
    assert f((G, O, 100, BF16), (K, G + 100, 10, BF16)) == ALIAS
    assert f((G, G, 100, BF16), (G, O, 100, BF16)) == ALIAS   # read by one, written by the other
    assert f((G, O, 100, BF16), (G, K, 100, BF16)) == NODEV   # read twice
    assert f((G, S, 100, BF16)) == ALIAS and f((G, WS, 10, BF16)) == ALIAS and f((WS, O, 10, BF16)) == ALIAS
    assert g((G, None, 10, BF16), norm=G) == ALIAS


def test_python_refusals():
    x, w = torch.zeros(4, 8), torch.zeros(8)
    for call in (lambda: dit.rmsnorm(x, w), lambda: dit.add_rmsnorm(x, x, w),
                 lambda: dit.rmsnorm_fp8(x, w), lambda: dit.rmsnorm_backward(x, x, w),
                 lambda: dit.embedding(torch.zeros(3, dtype=torch.int64), x),
                 lambda: dit.embedding_backward(x, torch.zeros(4, dtype=torch.int64), 10),
                 lambda: dit.grad_norm([x]), lambda: dit.clip_grads([x], 1.0)):
        with pytest.raises(TypeError):  # CPU tensors: no CPU path
            call()
    with pytest.raises(TypeError):
        dit.embedding(torch.zeros(3), x)
    with pytest.raises(ValueError):
        dit.rmsnorm(torch.zeros(()), w)
    with pytest.raises(ValueError):
        dit.rmsnorm_fp8(x, w, group=64)
    with pytest.raises(ValueError):
        dit.embedding_backward(x, torch.zeros(3, dtype=torch.int64), 10)
    with pytest.raises(ValueError):
        dit.grad_norm([])
