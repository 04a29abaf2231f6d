"""The entry points around attention without a GPU: sizes, types, strides,
overlaps and workspaces are checked on the host before anything is launched.
Pointers are plain integers that are never dereferenced."""
import ctypes

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from diffusion_transformer_elementwise_gb300 import library
from diffusion_transformer_elementwise_gb300._attend import Cache
from diffusion_transformer_elementwise_gb300.build import build

(OK, NULLP, SHAPE, DTYPE, LAYOUT, ALIAS, EPS, LAUNCH, MISALIGNED, NODEV, BADOP, WORKSPACE,
 BADSTAT, SCALAR, FORMAT, NOMEM) = range(16)
BF16, FP16, FP32, E4M3 = range(4)
A = 1 << 24
Q, K, QO, KO, GQ, GK, WQ, WK, COS, SIN, GW, GW2, WS, CK, CV, SK, SV, IDS, LSE, PG = (
    A * k for k in range(1, 21))
NAN, INF = float("nan"), float("inf")

pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="the pointers are not real: a valid call would launch")


@pytest.fixture(scope="module")
def lib():
    build()
    return library()


_kept = []


def keep(x):
    _kept.append(x)
    return ctypes.addressof(x)


def heads(p, token=256, head=64, batch=0):
    return None if p is None else keep((ctypes.c_int64 * 4)(p, batch, token, head))


def table(lib, cos=COS, sin=SIN, p=Q, f=K, n=5, sections=(4, 4), kind=1, axes=None):
    s = None if sections is None else keep((ctypes.c_int64 * max(1, len(sections)))(*sections))
    return lib.dit_rotary_table(cos, sin, p, f, n, s, len(sections or ()) if axes is None else axes, kind,
                                None)


def test_table(lib):
    assert table(lib) == NODEV and table(lib, kind=2, p=Q + 4) == NODEV
    assert table(lib, kind=3) == FORMAT and table(lib, kind=-1) == FORMAT
    assert table(lib, n=-1) == SHAPE and table(lib, n=1 << 31) == SHAPE
    assert table(lib, sections=()) == SHAPE and table(lib, sections=(1,) * 9) == SHAPE
    assert table(lib, sections=(-1, 4)) == SHAPE and table(lib, sections=(400, 113)) == SHAPE
    assert table(lib, sections=None, axes=1) == NULLP
    assert table(lib, n=0, cos=None) == OK and table(lib, sections=(0, 0)) == OK
    for name in ("cos", "sin", "p", "f"):
        assert table(lib, **{name: None}) == NULLP
    assert table(lib, p=Q + 4) == MISALIGNED and table(lib, f=K + 4) == MISALIGNED
    assert table(lib, cos=COS + 2) == MISALIGNED
    assert table(lib, cos=SIN) == ALIAS and table(lib, cos=Q) == ALIAS and table(lib, sin=K) == ALIAS
    assert table(lib, cos=SIN + 5 * 8 * 4) == NODEV and table(lib, cos=SIN + 5 * 8 * 4 - 4) == ALIAS


def rope(lib, qo=QO, ko=KO, q=Q, k=K, cos=COS, sin=SIN, B=2, L=3, Hq=4, Hk=2, D=64, R=32, rows=3, inter=0,
         inverse=0, dt=BF16, strides=None, norm=False, wq=WQ, wk=WK, eps=1e-6, off=0.0):
    s = {n: dict(token=256, head=64, batch=768) for n in ("qo", "ko", "q", "k")}
    s.update(strides or {})
    h = [heads(p, **s[n]) for n, p in (("qo", qo), ("ko", ko), ("q", q), ("k", k))]
    if norm:
        return lib.dit_rmsnorm_rope(*h, wq, wk, cos, sin, B, L, Hq, Hk, D, R, rows, eps, off, inter, dt, None)
    return lib.dit_rope(*h, cos, sin, B, L, Hq, Hk, D, R, rows, inter, inverse, dt, None)


def test_rope(lib):
    for norm in (False, True):
        def f(**kw):
            return rope(lib, norm=norm, **kw)
        assert f() == NODEV and f(rows=6) == NODEV and f(inter=1) == NODEV
        assert f(dt=3) == DTYPE and f(inter=2) == LAYOUT
        for bad in (dict(B=-1), dict(L=-1, rows=-1), dict(Hq=-1), dict(Hk=65536), dict(D=1025), dict(R=33),
                    dict(R=-1), dict(rows=4), dict(B=1 << 20, L=1 << 20, rows=1 << 20)):
            assert f(**bad) == SHAPE, bad
        assert f(B=0, rows=0, qo=None, q=None) == OK and f(D=0, R=0) == OK
        assert f(Hk=0, k=None, ko=None) == NODEV and f(R=0, cos=None, sin=None) == NODEV
        for n in ("qo", "ko", "q", "k", "cos", "sin"):
            assert f(**{n: None}) == NULLP
        assert f(q=Q + 1) == MISALIGNED and f(cos=COS + 2) == MISALIGNED and f(q=Q + 2) == NODEV
        # strides: none negative, none beyond 2^40
        assert f(strides=dict(q=dict(token=-1, head=64, batch=0))) == SHAPE
        assert f(strides=dict(q=dict(token=(1 << 40) + 1, head=64, batch=0))) == SHAPE
        assert f(strides=dict(q=dict(token=0, head=0, batch=0))) == NODEV      # an input that repeats
        assert f(strides=dict(qo=dict(token=0, head=64, batch=768))) == ALIAS  # an output must not
        assert f(strides=dict(qo=dict(token=128, head=64, batch=768))) == ALIAS
        # overlaps
        assert f(qo=Q) == NODEV and f(ko=K) == NODEV and f(qo=Q + 2) == ALIAS
        assert f(qo=Q, strides=dict(qo=dict(token=512, head=64, batch=2048))) == ALIAS
        assert f(qo=K) == ALIAS and f(ko=Q) == ALIAS and f(ko=QO) == ALIAS
        assert f(qo=COS) == ALIAS and f(ko=SIN) == ALIAS
        # views of one packed projection [tokens, 4 + 2 + 2, 64]
        packed = dict(token=512, head=64, batch=1536)
        p = {n: packed for n in ("qo", "ko", "q", "k")}
        assert f(q=Q, qo=Q, k=Q + 512, ko=Q + 512, strides=p) == NODEV
        assert f(q=Q, qo=Q, k=Q + 510, ko=Q + 510, strides=p) == ALIAS
        assert f(q=Q, k=Q + 512, ko=Q + 768, strides=p) == NODEV and f(q=Q, k=Q + 512, ko=Q + 770, strides=p) == ALIAS
        # heads that interleave: [tokens, heads, 2, 64]
        two = dict(token=512, head=128, batch=1536)
        p = {n: two for n in ("qo", "ko", "q", "k")}
        assert f(q=Q, qo=Q + 128, strides=p) == NODEV and f(q=Q, qo=Q + 126, strides=p) == ALIAS
    assert rope(lib, inverse=2) == LAYOUT
    assert rope(lib, norm=True, wq=None) == NULLP and rope(lib, norm=True, wk=WK + 1) == MISALIGNED
    assert rope(lib, norm=True, qo=WQ) == ALIAS and rope(lib, norm=True, ko=WQ) == ALIAS
    assert rope(lib, norm=True, eps=-1.0) == EPS and rope(lib, norm=True, off=INF) == SCALAR


def back(lib, oq=QO, ok=KO, gwq=GW, gwk=GW2, gq=GQ, gk=GK, q=Q, k=K, wq=WQ, wk=WK, cos=COS, sin=SIN, B=2, L=3,
         Hq=4, Hk=2, D=64, R=32, rows=3, eps=1e-6, off=0.0, inter=0, dt=BF16, ws=WS, n=None):
    n = lib.dit_rmsnorm_rope_backward_workspace_bytes(D) if n is None else n
    h = [heads(p, batch=768) for p in (oq, ok, gq, gk, q, k)]
    return lib.dit_rmsnorm_rope_backward(h[0], h[1], gwq, gwk, *h[2:], wq, wk, cos, sin, B, L, Hq, Hk, D, R, rows,
                                         eps, off, inter, dt, ws, n, None)


def test_rope_backward(lib):
    wb = lib.dit_rmsnorm_rope_backward_workspace_bytes
    assert wb(64) == 608 * 2 * 64 * 4 and wb(0) == 0 and wb(-1) == wb(1025) == -1
    assert back(lib) == NODEV and back(lib, gwq=None) == NODEV
    assert back(lib, gwq=None, gwk=None, ws=None, n=0) == NODEV
    assert back(lib, Hk=0, ok=None, gk=None, k=None, wk=None, gwk=None) == NODEV
    assert back(lib, B=0, rows=0, oq=None, gq=None, q=None, ws=None) == NODEV  # the weights' are zero
    assert back(lib, B=0, rows=0, gwq=None, gwk=None) == OK and back(lib, D=0, R=0) == OK
    for name in ("oq", "ok", "gq", "gk", "q", "k", "wq", "wk", "cos", "sin"):
        assert back(lib, **{name: None}) == NULLP, name
    assert back(lib, ws=None) == WORKSPACE and back(lib, ws=WS + 8) == WORKSPACE and back(lib, n=wb(64) - 1) == WORKSPACE
    assert back(lib, gwq=GW + 1) == MISALIGNED and back(lib, gq=GQ + 1) == MISALIGNED
    assert back(lib, oq=GQ) == NODEV and back(lib, ok=GK) == NODEV and back(lib, oq=Q) == ALIAS
    assert back(lib, oq=GK) == ALIAS and back(lib, oq=GQ + 16) == ALIAS and back(lib, oq=WQ) == ALIAS
    assert back(lib, gwq=WQ) == ALIAS and back(lib, gwq=Q) == ALIAS and back(lib, gwk=QO) == ALIAS
    assert back(lib, gwq=GW2) == ALIAS and back(lib, gwq=COS) == ALIAS
    assert back(lib, ws=Q) == ALIAS and back(lib, ws=SIN) == ALIAS and back(lib, ws=GW) == ALIAS
    assert back(lib, eps=NAN) == EPS and back(lib, off=NAN) == SCALAR and back(lib, dt=5, n=0) == DTYPE


def cache(**kw):
    c = dict(k=CK, v=CV, k_scales=SK, v_scales=SV, pages=10, heads=2, page_size=16, D=64, page_stride=2048,
             scale_stride=32, format=BF16)
    c.update(kw)
    return keep(Cache(**c))


def rows(fn, c=None, k=Q, v=K, n=5, ids=IDS, it=1, dt=BF16, ks=None, vs=None):
    return fn(cache() if c is None else c, heads(k, **(ks or {})), heads(v, **(vs or {})), n, ids, it, dt, None)


def test_cache(lib):
    for fn in (lib.dit_cache_write, lib.dit_cache_read):
        def f(c=None, **kw):
            return rows(fn, c, **kw)
        assert f() == NODEV and f(cache(format=E4M3)) == NODEV and f(cache(format=E4M3), dt=FP32) == NODEV
        assert f(c=0) in (NULLP,) and f(dt=3) == DTYPE and f(it=2) == FORMAT
        assert f(dt=FP16) == DTYPE and f(cache(format=4)) == FORMAT and f(cache(format=-1)) == FORMAT
        for bad in (dict(pages=-1), dict(heads=-1), dict(page_size=0), dict(D=1025), dict(page_stride=2047),
                    dict(pages=1 << 30), dict(page_stride=1 << 41), dict(format=E4M3, scale_stride=31)):
            assert f(cache(**bad)) == SHAPE, bad
        assert f(n=-1) == SHAPE and f(n=0, k=None) == OK and f(cache(heads=0), k=None) == OK
        assert f(cache(k=None)) == NULLP and f(cache(format=E4M3, v_scales=None)) == NULLP
        assert f(k=None) == NULLP and f(v=None) == NULLP and f(ids=None) == NULLP
        assert f(cache(k=CK + 1)) == MISALIGNED and f(cache(k=CK + 1, format=E4M3)) == NODEV
        assert f(k=Q + 1) == MISALIGNED and f(ids=IDS + 4) == MISALIGNED and f(ids=IDS + 4, it=0) == NODEV
        assert f(cache(format=E4M3, k_scales=SK + 2)) == MISALIGNED
        assert f(k=CK) == ALIAS and f(v=CK) == ALIAS and f(cache(format=E4M3), k=SK) == ALIAS
        assert f(cache(pages=0)) == (OK if fn is lib.dit_cache_write else NODEV)
    w, r = lib.dit_cache_write, lib.dit_cache_read
    assert rows(w, cache(v=CK)) == ALIAS and rows(w, cache(v=CK + 2 * 2048)) == ALIAS
    joined = dict(v=CK + 2 * 2048, page_stride=4096)  # halves of one allocation
    assert rows(w, cache(**joined)) == NODEV and rows(r, cache(**joined)) == NODEV
    assert rows(w, cache(**dict(joined, v=CK + 2 * 2047))) == ALIAS
    assert rows(w, cache(format=E4M3, v_scales=SK)) == ALIAS
    assert rows(w, ids=CK) == ALIAS and rows(w, k=K) == NODEV        # the same rows twice are read
    assert rows(r, k=K) == ALIAS and rows(r, k=IDS) == ALIAS
    assert rows(r, ks=dict(token=64, head=64)) == ALIAS and rows(w, ks=dict(token=0, head=0)) == NODEV


def attend(lib, o=QO, lse=LSE, q=Q, c=None, pages=PG, ps=4, width=4, lengths=IDS, B=3, Hq=4, scale=0.1,
           window=0, it=0, dt=BF16, ws=WS, n=None, os=None, D=64, H=2):
    n = lib.dit_paged_attention_workspace_bytes(Hq, H, D) if n is None else n
    return lib.dit_paged_attention(heads(o, **(os or {})), lse, heads(q), cache() if c is None else c, pages, ps,
                                   width, lengths, B, Hq, scale, window, it, dt, ws, n, None)


def test_attention(lib):
    wb = lib.dit_paged_attention_workspace_bytes
    assert wb(4, 2, 64) == 9728 + 160 * 17 * 2 * 2 * 66 * 4
    assert wb(64, 1, 64) == 9728 + 160 * 17 * 2 * 16 * 66 * 4
    assert wb(4, 3, 64) == wb(0, 1, 64) == wb(4, 0, 64) == wb(4, 2, 0) == wb(4, 2, 513) == -1
    assert attend(lib) == NODEV and attend(lib, lse=None) == NODEV and attend(lib, it=1) == NODEV
    assert attend(lib, c=cache(format=E4M3)) == NODEV and attend(lib, c=cache(format=E4M3), dt=FP32) == NODEV
    assert attend(lib, dt=FP16) == DTYPE and attend(lib, dt=7) == DTYPE and attend(lib, it=2) == FORMAT
    for bad in (dict(B=-1), dict(width=-1), dict(ps=3), dict(window=-1), dict(Hq=3, n=0), dict(Hq=0, n=0),
                dict(width=1 << 28, ps=1 << 28), dict(c=cache(D=520, page_stride=1 << 20), n=0)):
        assert attend(lib, **bad) == SHAPE, bad
    for s in (NAN, INF, -INF):
        assert attend(lib, scale=s) == SCALAR
    assert attend(lib, B=0, o=None, q=None, lengths=None) == OK
    assert attend(lib, B=1, ps=0) == NODEV
    for name in ("o", "q", "lengths", "pages"):
        assert attend(lib, **{name: None}) == NULLP
    assert attend(lib, width=0, pages=None) == NODEV
    assert attend(lib, q=Q + 1) == MISALIGNED and attend(lib, lse=LSE + 2) == MISALIGNED
    assert attend(lib, pages=PG + 2) == MISALIGNED and attend(lib, lengths=IDS + 4, it=1) == MISALIGNED
    assert attend(lib, ws=None) == WORKSPACE and attend(lib, ws=WS + 64) == WORKSPACE
    assert attend(lib, n=wb(4, 2, 64) - 1) == WORKSPACE
    for name in ("o", "lse", "ws"):
        for other in (Q, PG, IDS, CK, CV):
            assert attend(lib, **{name: other}) == ALIAS, (name, other)
    assert attend(lib, o=LSE) == ALIAS and attend(lib, o=WS) == ALIAS and attend(lib, lse=WS) == ALIAS
    assert attend(lib, o=SK, c=cache(format=E4M3)) == ALIAS and attend(lib, o=SK) == NODEV
    assert attend(lib, os=dict(token=64, head=64)) == ALIAS


def test_python_refusals():
    x, w = torch.zeros(4, 2, 8), torch.zeros(8)
    ids = torch.zeros(4, dtype=torch.int64)
    for call in (lambda: dit.rope(x, x, x, x), lambda: dit.rmsnorm_rope(x, x, w, w, None, None),
                 lambda: dit.rmsnorm_rope_backward(x, x, x, x, w, w, None, None),
                 lambda: dit.rotary_table(ids, torch.zeros(4, dtype=torch.float64)),
                 lambda: dit.KVCache(x, x), lambda: dit.cache_write(None, x, x, ids),
                 lambda: dit.cache_read(None, ids), lambda: dit.paged_attention(x, None, ids, ids)):
        with pytest.raises(TypeError):  # CPU tensors: no CPU path
            call()
    f = dit.rotary_frequencies([2, 3], theta=100.0, device="cpu")
    assert f.tolist() == pytest.approx([1.0, 0.1, 1.0, 100.0 ** (-1 / 3), 100.0 ** (-2 / 3)])
    assert dit.rotary_frequencies([2, 2], 16.0, shared=True, device="cpu").tolist() == [1.0, 0.5, 0.25, 0.125]
