"""The operators around attention of libdit_elementwise.so
(include/dit_elementwise.h): rotary angles, the rotation of queries and keys with the norm
of each head in the same pass, its gradient, a paged cache of keys and
values, and the attention of one new token per sequence over it.

Argument marshalling, as in ``_token``: CUDA tensors of one dtype, the current
torch stream unless ``stream`` says otherwise, :class:`DitError` on a non-OK
status; what a call allocates comes from the stream it launches on; no function takes
part in autograd.  Tensors of heads ([..., tokens, heads, D]) may be views with any strides
whose last dimension is contiguous, such as the queries of a packed projection.
"""
from __future__ import annotations

import ctypes

import torch

from ._binding import _FP8, DTYPE_CODES, _cuda, _dtype, _stream, library
from ._token import ID_CODES, _call, _empty, _workspace

POSITION_CODES = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
E4M3 = 3


class Cache(ctypes.Structure):
    """dit_cache of include/dit_elementwise.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("page_size", ctypes.c_int64), ("D", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("scale_stride", ctypes.c_int64),
                ("format", ctypes.c_int64)]


def declare(lib) -> None:
    """The argument types of the entry points."""
    vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    for name, args in (
            ("dit_rotary_table", [vp] * 4 + [i64, vp, i64, ci, vp]),
            ("dit_rope", [vp] * 6 + [i64] * 7 + [ci, ci, ci, vp]),
            ("dit_rmsnorm_rope", [vp] * 8 + [i64] * 7 + [cf, cf, ci, ci, vp]),
            ("dit_rmsnorm_rope_backward",
             [vp] * 12 + [i64] * 7 + [cf, cf, ci, ci, vp, i64, vp]),
            ("dit_cache_write", [vp] * 3 + [i64, vp, ci, ci, vp]),
            ("dit_cache_read", [vp] * 3 + [i64, vp, ci, ci, vp]),
            ("dit_paged_attention",
             [vp] * 5 + [i64, i64, vp, i64, i64, cf, i64, ci, ci, vp, i64, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ci
    for name, n in (("dit_rmsnorm_rope_backward_workspace_bytes", 1),
                    ("dit_paged_attention_workspace_bytes", 3)):
        getattr(lib, name).argtypes = [i64] * n
        getattr(lib, name).restype = i64


# ---------------------------------------------------------------------------
# views of heads
# ---------------------------------------------------------------------------

_SIZE = 32  # bytes of a dit_heads
_WORDS = [ctypes.c_int64 * (4 * n) for n in range(7)]
_addressof = ctypes.addressof


def _heads(dims, like, *views):
    """The dit_heads of views ([..., tokens, heads, D], of `dims` dimensions, 3 or 4): (device index,
    dtype code, their array, its address), after a check that they are CUDA tensors of one dtype
    and device, with contiguous rows, and each of the shape of its entry in `like`.  The usual
    case takes one pass; what is wrong is found out in a second (_refuse)."""
    words = []
    try:
        first = views[0]
        dtype, dev = first.dtype, first.get_device()
        ok = dev >= 0
        for t, shape in zip(views, like):
            stride = t.stride()
            if (t.dtype is not dtype or t.get_device() != dev or t.shape != shape
                    or len(stride) != dims or (stride[-1] != 1 and shape[-1] > 1)):
                ok = False
                break
            words += (t.data_ptr(), stride[0] if dims == 4 else 0, stride[-3], stride[-2])
        code = DTYPE_CODES[dtype] if ok else 0
    except (AttributeError, KeyError, IndexError):
        ok = False
    if not ok:
        return None
    array = _WORDS[len(views)](*words)
    return dev, code, array, _addressof(array)


def _refuse(dims, like, names, views):
    """Raises what is wrong with the views of a _heads that returned None."""
    for name, t in zip(names, views):
        _tensor(t, name)
    dev = views[0].get_device()
    for name, t, shape in zip(names, views, like):
        if t.get_device() != dev:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, expected cuda:{dev}")
        _match(name, t, shape)
        if t.dim() != dims:
            raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError(f"the rows of {name} (its last dimension) must be contiguous")
    _dtype(views[0], *zip(names, views))
    raise ValueError("tensors that do not go together")


def _tensor(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor (there is no CPU path)")


def _match(name, t, shape):
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, got {tuple(t.shape)}")


def _angles(cos, sin, B, L, dev):
    """(R, rows, addresses) of a rotary table for B batches of L tokens."""
    if cos is None and sin is None:
        return 0, B * L, None, None
    try:
        shape = cos.shape
        ok = (cos.dtype is torch.float32 and sin.dtype is torch.float32 and sin.shape == shape
              and cos.get_device() == dev and sin.get_device() == dev and cos.is_contiguous()
              and sin.is_contiguous() and len(shape) >= 2)
    except AttributeError:
        ok = False
    if not ok:
        _cuda(("cos", cos), ("sin", sin))
        if cos.dtype is not torch.float32 or sin.dtype is not torch.float32:
            raise TypeError("cos and sin must be float32")
        if cos.shape != sin.shape or cos.dim() < 2:
            raise ValueError("cos and sin must be [rows, R], of one shape")
        raise ValueError(f"cos is on cuda:{cos.get_device()}, expected cuda:{dev}")
    R = shape[-1]
    rows = (shape[0] if len(shape) == 2 else cos.numel() // R) if R else B * L
    if rows != L and rows != B * L:
        raise ValueError(f"cos and sin have {rows} rows, for {B} x {L} tokens")
    return R, rows, cos.data_ptr(), sin.data_ptr()


def _shapes(q, k):
    """(B, L, Hq, Hk, D, dimensions, q's shape, k's shape) of queries and keys ([B, L, H, D], or
    [L, H, D])."""
    if not isinstance(q, torch.Tensor) or (k is not None and not isinstance(k, torch.Tensor)):
        _tensor(q, "q")
        _tensor(k, "k")
    sq = q.shape
    n = len(sq)
    if n == 3:
        B = 1
        L, Hq, D = sq
    elif n == 4:
        B, L, Hq, D = sq
    else:
        _tensor(q, "q")
        raise ValueError("q must be [tokens, heads, D] or [B, L, heads, D]")
    if k is None:
        return B, L, Hq, 0, D, n, sq, None
    sk = k.shape
    if len(sk) != n or sk[-1] != D or sk[:-2] != sq[:-2]:
        _tensor(k, "k")
        raise ValueError(f"k must be of q's shape but for its heads, got {tuple(sk)} for {tuple(sq)}")
    return B, L, Hq, sk[-2], D, n, sq, sk


def _weight(w, name, D, ref, dev):
    try:
        if (w.dtype is ref.dtype and w.get_device() == dev and w.shape == (D,)
                and w.is_contiguous()):
            return w.data_ptr()
    except AttributeError:
        pass
    _tensor(w, name)
    raise ValueError(f"{name} must be a contiguous [{D}] {ref.dtype} tensor on {ref.device}, got "
                     f"{tuple(w.shape)} {w.dtype} on {w.device}")


# ---------------------------------------------------------------------------
# angles and rotation
# ---------------------------------------------------------------------------

def rotary_frequencies(sections, theta=10000.0, shared=False, device="cuda"):
    """The angle per unit of position of every column, float64 [R]: theta^(-j / n) for column j
    of the n of an axis (`sections`: an int for one axis, or a count for each), or --
    shared=True -- one spectrum theta^(-j / R) that the axes share out.  Made
    once, for rotary_table."""
    sections = [sections] if isinstance(sections, int) else [int(n) for n in sections]
    R = sum(sections)
    e = [j / R for j in range(R)] if shared else [j / n for n in sections for j in range(n)]
    return torch.tensor([float(theta) ** -v for v in e], dtype=torch.float64, device=device)


def rotary_table(positions, freqs, sections=None, cos=None, sin=None, stream=None):
    """cos and sin of positions[axis(j), t] * freqs[j], float32 [tokens, R].  positions: int32, int64
    or float32, [tokens] for one axis or [axes, tokens]; freqs: float64 [R]; sections: the
    number of columns of each axis, in order (None: one axis).  The frequency is held in
    turns, to 2^-52 of it; beyond that the angle is reduced without loss, however far the
    position.  Returns (cos, sin)."""
    _tensor(positions, "positions")
    if positions.dtype not in POSITION_CODES:
        raise TypeError("positions must be int32, int64 or float32")
    if positions.dim() not in (1, 2):
        raise ValueError("positions must be [tokens] or [axes, tokens]")
    axes = positions.shape[0] if positions.dim() == 2 else 1
    T = positions.shape[-1]
    _tensor(freqs, "freqs")
    if freqs.dtype is not torch.float64 or freqs.dim() != 1:
        raise TypeError("freqs must be a float64 [R] tensor")
    R = freqs.numel()
    if sections is None:
        sections = [R]
    elif isinstance(sections, int):
        sections = [sections]
    if len(sections) != axes or sum(sections) != R:
        raise ValueError(f"sections must be {axes} counts whose sum is {R}, got {list(sections)}")
    if axes == 0:
        raise ValueError("positions must have an axis")
    if cos is None:
        cos = _empty((T, R), torch.float32, positions.device, stream)
    if sin is None:
        sin = _empty((T, R), torch.float32, positions.device, stream)
    dev = _cuda(("positions", positions), ("freqs", freqs), ("cos", cos), ("sin", sin))
    for name, t in (("cos", cos), ("sin", sin)):
        if t.dtype is not torch.float32:
            raise TypeError(f"{name} must be float32")
        _match(name, t, (T, R))
    counts = (ctypes.c_int64 * axes)(*sections)
    _call(dev, library().dit_rotary_table, "dit_rotary_table", cos.data_ptr(), sin.data_ptr(),
          positions.data_ptr(), freqs.data_ptr(), T, ctypes.addressof(counts), axes,
          POSITION_CODES[positions.dtype], _stream(dev, stream))
    return cos, sin


def rope(q, k, cos, sin, interleaved=False, inverse=False, out_q=None, out_k=None, stream=None):
    """Queries and keys ([B, L, heads, D] or [tokens, heads, D] each; k may be None) turned by their
    tokens' angles: the pairs of columns (j, j + R), or (2j, 2j + 1) where
    interleaved, by row t of cos and sin ([B * L, R], or [L, R] for all batches);
    columns from 2R on are copied.  inverse=True turns back, which is the gradient.
    out_q may be q, out_k may be k.  Returns (out_q, out_k)."""
    B, L, Hq, Hk, D, n, sq, sk = _shapes(q, k)
    if out_q is None:
        out_q = _empty(sq, q.dtype, q.device, stream)
    if k is None:
        if out_k is not None:
            raise ValueError("out_k without k")
        like, views = (sq, sq), (q, out_q)
    else:
        if out_k is None:
            out_k = _empty(sk, k.dtype, k.device, stream)
        like, views = (sq, sq, sk, sk), (q, out_q, k, out_k)
    found = _heads(n, like, *views)
    if found is None:
        _refuse(n, like, ("q", "out_q", "k", "out_k"), views)
    dev, dt, _keep, at = found
    R, rows, pc, ps = _angles(cos, sin, B, L, dev)
    kp, ko = (at + 2 * _SIZE, at + 3 * _SIZE) if k is not None else (None, None)
    _call(dev, library().dit_rope, "dit_rope", at + _SIZE, ko, at, kp, pc, ps, B, L, Hq, Hk, D, R,
          rows, int(interleaved), int(inverse), dt, _stream(dev, stream))
    return out_q, out_k


def rmsnorm_rope(q, k, weight_q, weight_k, cos, sin, eps=1e-6, weight_offset=0.0,
                 interleaved=False, out_q=None, out_k=None, stream=None):
    """rope of the weighted RMSNorm of each head (over its D columns) in one pass: weight_q
    and weight_k are [D], weight_offset 1 for weights stored as their difference from one.
    cos=sin=None: the norm alone.  out_q may be q, out_k may be k.  Returns (out_q, out_k)."""
    B, L, Hq, Hk, D, n, sq, sk = _shapes(q, k)
    if out_q is None:
        out_q = _empty(sq, q.dtype, q.device, stream)
    if k is None:
        if out_k is not None or weight_k is not None:
            raise ValueError("out_k or weight_k without k")
        like, views = (sq, sq), (q, out_q)
    else:
        if out_k is None:
            out_k = _empty(sk, k.dtype, k.device, stream)
        like, views = (sq, sq, sk, sk), (q, out_q, k, out_k)
    found = _heads(n, like, *views)
    if found is None:
        _refuse(n, like, ("q", "out_q", "k", "out_k"), views)
    dev, dt, _keep, at = found
    wq = _weight(weight_q, "weight_q", D, q, dev)
    wk, kp, ko = None, None, None
    if k is not None:
        wk, kp, ko = _weight(weight_k, "weight_k", D, q, dev), at + 2 * _SIZE, at + 3 * _SIZE
    R, rows, pc, ps = _angles(cos, sin, B, L, dev)
    _call(dev, library().dit_rmsnorm_rope, "dit_rmsnorm_rope", at + _SIZE, ko, at, kp, wq, wk, pc,
          ps, B, L, Hq, Hk, D, R, rows, eps, weight_offset, int(interleaved), dt,
          _stream(dev, stream))
    return out_q, out_k


def rmsnorm_rope_backward(grad_out_q, grad_out_k, q, k, weight_q, weight_k, cos, sin, eps=1e-6,
                          weight_offset=0.0, interleaved=False, grad_q=None, grad_k=None,
                          grad_weight_q=None, grad_weight_k=None, need_weight=True,
                          workspace=None, stream=None):
    """Gradients of rmsnorm_rope(q, k, ...): returns (grad_q, grad_k, grad_weight_q,
    grad_weight_k).  need_weight=False (frozen weights): the last two are None.
    grad_q may be grad_out_q, grad_k may be grad_out_k.  workspace: a uint8
    CUDA tensor of at least dit_rmsnorm_rope_backward_workspace_bytes(D) bytes
    (allocated if None)."""
    B, L, Hq, Hk, D, n, sq, sk = _shapes(q, k)
    if grad_q is None:
        grad_q = _empty(sq, q.dtype, q.device, stream)
    like, views = (sq, sq, sq), (q, grad_out_q, grad_q)
    if k is None:
        if (grad_out_k is not None or grad_k is not None or weight_k is not None
                or grad_weight_k is not None):
            raise ValueError("a key's tensor without k")
    else:
        if grad_k is None:
            grad_k = _empty(sk, k.dtype, k.device, stream)
        like, views = like + (sk, sk, sk), views + (k, grad_out_k, grad_k)
    found = _heads(n, like, *views)
    if found is None:
        _refuse(n, like, ("q", "grad_out_q", "grad_q", "k", "grad_out_k", "grad_k"), views)
    dev, dt, _keep, at = found
    lib = library()
    wq = _weight(weight_q, "weight_q", D, q, dev)
    wk, k_at = None, (None,) * 3
    if k is not None:
        wk, k_at = _weight(weight_k, "weight_k", D, q, dev), (at + 3 * _SIZE, at + 4 * _SIZE, at + 5 * _SIZE)
    ws, wp, wn, gq, gk = None, None, 0, None, None
    if not need_weight:
        grad_weight_q = grad_weight_k = None
    else:
        if grad_weight_q is None:
            grad_weight_q = _empty((D,), q.dtype, q.device, stream)
        gq = _weight(grad_weight_q, "grad_weight_q", D, q, dev)
        if k is not None:
            if grad_weight_k is None:
                grad_weight_k = _empty((D,), q.dtype, q.device, stream)
            gk = _weight(grad_weight_k, "grad_weight_k", D, q, dev)
        ws, wp, wn = _workspace(workspace, lib.dit_rmsnorm_rope_backward_workspace_bytes(D), q, stream)
    R, rows, pc, ps = _angles(cos, sin, B, L, dev)
    _call(dev, lib.dit_rmsnorm_rope_backward, "dit_rmsnorm_rope_backward", at + 2 * _SIZE, k_at[2],
          gq, gk, at + _SIZE, k_at[1], at, k_at[0], wq, wk, pc, ps, B, L, Hq, Hk, D, R, rows, eps,
          weight_offset, int(interleaved), dt, wp, wn, _stream(dev, stream))
    return grad_q, grad_k, grad_weight_q, grad_weight_k


# ---------------------------------------------------------------------------
# the paged cache
# ---------------------------------------------------------------------------

class KVCache:
    """A paged cache: k and v are [pages, heads, page_size, D], contiguous but for the
    pages' stride (both may be halves of one allocation).  Of bf16, fp16 or
    fp32, or of float8_e4m3fn (or uint8) with a float32 scale per row, k_scales and v_scales [pages,
    heads, page_size].  It holds the tensors; replacing a tensor's storage
    (set_, resize_) after this makes it stale."""

    def __init__(self, k, v, k_scales=None, v_scales=None):
        named = (("k", k), ("v", v))
        fp8 = k_scales is not None or v_scales is not None
        if fp8:
            named += (("k_scales", k_scales), ("v_scales", v_scales))
        for name, t in named:
            _tensor(t, name)
            if t.get_device() != k.get_device():
                raise ValueError(f"{name} is on {t.device}, expected {k.device}")
            step = 1  # (sizes of one have any stride)
            for size, stride in zip(t.shape[:0:-1], t.stride()[:0:-1]):
                if size > 1 and stride != step and t.numel() > 0:
                    raise ValueError(f"the pages of {name} must be contiguous")
                step *= size
        if k.dim() != 4 or v.shape != k.shape or v.dtype is not k.dtype:
            raise ValueError("k and v must be [pages, heads, page_size, D], of one shape and dtype")
        if fp8:
            if k.dtype is not _FP8 and k.dtype is not torch.uint8:
                raise TypeError(f"a cache with scales is float8_e4m3fn or uint8, got {k.dtype}")
            for name, t in named[2:]:
                if t.dtype is not torch.float32 or t.shape != k.shape[:3]:
                    raise ValueError(f"{name} must be float32 {tuple(k.shape[:3])}, got {t.dtype} "
                                     f"{tuple(t.shape)}")
            self.format = E4M3
        elif k.dtype in DTYPE_CODES:
            self.format = DTYPE_CODES[k.dtype]
        else:
            raise TypeError(f"unsupported cache dtype {k.dtype}: bf16, fp16, fp32, or E4M3 with scales")
        if k.shape[0] > 1:
            for a, b in zip((t for _, t in named[::2]), (t for _, t in named[1::2])):
                if a.stride(0) != b.stride(0):
                    raise ValueError("the pages of k and v must have one stride")
        self.k, self.v, self.k_scales, self.v_scales = k, v, k_scales, v_scales
        self.pages, self.heads, self.page_size, self.D = k.shape
        self.dtype, self.device = k.dtype, k.device
        n, rows = self.heads * self.page_size * self.D, self.heads * self.page_size
        self.array = Cache(k.data_ptr(), v.data_ptr(), k_scales.data_ptr() if fp8 else None,
                           v_scales.data_ptr() if fp8 else None, *k.shape,
                           k.stride(0) if self.pages > 1 else n,
                           (k_scales.stride(0) if self.pages > 1 else rows) if fp8 else 0,
                           self.format)
        self.address = ctypes.addressof(self.array)
        self.needs = {}  # the attention's workspace by the number of query heads
        self.device_index = k.get_device()

    @classmethod
    def empty(cls, pages, heads, page_size, D, dtype=torch.bfloat16, device="cuda"):
        """A cache in new memory, its pages not initialised; dtype float8_e4m3fn: E4M3 with scales."""
        k, v = (torch.empty((pages, heads, page_size, D), dtype=dtype, device=device) for _ in "kv")
        if dtype is not _FP8:
            return cls(k, v)
        return cls(k, v, *(torch.empty((pages, heads, page_size), dtype=torch.float32, device=device)
                           for _ in "kv"))


def _slots(cache, k, v, slots):
    """Checks the rows [tokens, heads, D] and their slots; (device, dtype code, id code, array, address)."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if not isinstance(slots, torch.Tensor) or slots.dtype not in ID_CODES:
        raise TypeError("slots must be an int32 or int64 CUDA tensor")
    if slots.dim() != 1:
        raise ValueError("slots must be [tokens]")
    like = ((slots.shape[0], cache.heads, cache.D),) * 2
    found = _heads(3, like, k, v)
    if found is None:
        _refuse(3, like, ("k", "v"), (k, v))
    dev, dt, keep, at = found
    if dev != cache.device_index:
        raise ValueError(f"k is on cuda:{dev}, expected {cache.device}")
    if slots.get_device() != dev or not slots.is_contiguous():
        _tensor(slots, "slots")
        raise ValueError(f"slots must be contiguous, on cuda:{dev}")
    if cache.format != E4M3 and cache.format != dt:
        raise TypeError(f"k is {k.dtype}, the cache {cache.dtype}")
    return dev, dt, ID_CODES[slots.dtype], keep, at


def cache_write(cache, k, v, slots, stream=None):
    """Write keys and values [tokens, heads, D] (bf16, fp16 or fp32; the cache's dtype unless it is
    E4M3) to places slots[t] = page * page_size + place: int32 or int64, a token whose slot is outside the
    cache (e.g. -1) is not written.  Within the cache the slots of a call must
    differ.  E4M3: one scale per row, its largest magnitude / 448."""
    dev, dt, it, _keep, at = _slots(cache, k, v, slots)
    _call(dev, library().dit_cache_write, "dit_cache_write", cache.address, at, at + _SIZE,
          slots.shape[0], slots.data_ptr(), it, dt, _stream(dev, stream))


def cache_read(cache, slots, dtype=None, k=None, v=None, stream=None):
    """The keys and values of the places slots[t] (cache_write), [tokens, heads, D] each, rows of
    zeros where a slot is outside the cache.  dtype: of the result, for an E4M3 cache (bf16 if None
    and no k is given).  Returns (k, v)."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if not isinstance(slots, torch.Tensor) or slots.dtype not in ID_CODES:
        raise TypeError("slots must be an int32 or int64 CUDA tensor")
    shape = (slots.numel(), cache.heads, cache.D)
    if dtype is None:
        dtype = (k.dtype if k is not None else v.dtype if v is not None
                 else torch.bfloat16 if cache.format == E4M3 else cache.dtype)
    if k is None:
        k = _empty(shape, dtype, cache.device, stream)
    if v is None:
        v = _empty(shape, dtype, cache.device, stream)
    dev, dt, it, _keep, at = _slots(cache, k, v, slots)
    if k.dtype is not dtype:
        raise TypeError(f"k is {k.dtype}, expected {dtype}")
    _call(dev, library().dit_cache_read, "dit_cache_read", cache.address, at, at + _SIZE,
          slots.shape[0], slots.data_ptr(), it, dt, _stream(dev, stream))
    return k, v


def paged_attention(q, cache, pages, lengths, scale=None, window=0, out=None, lse=None,
                    need_lse=False, workspace=None, stream=None):
    """Attention of one new token per sequence: q [B, Hq, D] over the first lengths[b] tokens of sequence
    b (the last `window` of them, if that is not 0), token t at place t % page_size of
    page pages[b, t // page_size] of the cache (KVCache).  Hq is a multiple
    of the cache's heads; query head h reads key head h // (Hq / heads).
    pages: int32 [B, width], rows contiguous (one row for all sequences may be expanded); a page outside the cache leaves its tokens out.
    lengths: int32 or int64 [B].  scale: of the logits (D^-0.5 if None).  A sequence without a token has
    out 0 and lse -inf.  lse (float32 [B, Hq], where given or needed): the
    logarithm of the sum of the exponentials.  workspace: a uint8 CUDA tensor of
    at least dit_paged_attention_workspace_bytes(Hq, heads, D) bytes (allocated if
    None).  Returns (out, lse)."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if not isinstance(q, torch.Tensor):
        _tensor(q, "q")
    shape = q.shape
    if len(shape) != 3 or shape[2] != cache.D:
        _tensor(q, "q")
        raise ValueError(f"q must be [B, heads, {cache.D}], got {tuple(shape)}")
    B, Hq, D = shape
    if cache.heads == 0 or Hq == 0 or Hq % cache.heads:
        raise ValueError(f"q has {Hq} heads, the cache {cache.heads}")
    if out is None:
        out = _empty(shape, q.dtype, q.device, stream)
    found = _heads(3, (shape, shape), q, out)
    if found is None:
        _refuse(3, (shape, shape), ("q", "out"), (q, out))
    dev, dt, _keep, at = found
    if dev != cache.device_index:
        raise ValueError(f"q is on cuda:{dev}, expected {cache.device}")
    if cache.format != E4M3 and cache.format != dt:
        raise TypeError(f"q is {q.dtype}, the cache {cache.dtype}")
    if (not isinstance(pages, torch.Tensor) or pages.dtype is not torch.int32 or pages.dim() != 2
            or pages.shape[0] != B or pages.get_device() != dev
            or (pages.stride(1) != 1 and pages.shape[1] > 1)):
        _tensor(pages, "pages")
        raise ValueError(f"pages must be int32 [{B}, width] on cuda:{dev} with contiguous rows, got "
                         f"{pages.dtype} {tuple(pages.shape)} on {pages.device}")
    if (not isinstance(lengths, torch.Tensor) or lengths.dtype not in ID_CODES
            or lengths.shape != (B,) or lengths.get_device() != dev or not lengths.is_contiguous()):
        _tensor(lengths, "lengths")
        raise ValueError(f"lengths must be a contiguous int32 or int64 [{B}] tensor on cuda:{dev}, "
                         f"got {lengths.dtype} {tuple(lengths.shape)} on {lengths.device}")
    if lse is None:
        if need_lse:
            lse = _empty((B, Hq), torch.float32, q.device, stream)
    elif (not isinstance(lse, torch.Tensor) or lse.dtype is not torch.float32
          or lse.shape != (B, Hq) or lse.get_device() != dev or not lse.is_contiguous()):
        _tensor(lse, "lse")
        raise ValueError(f"lse must be a contiguous float32 [{B}, {Hq}] tensor on cuda:{dev}")
    lib = library()
    need = cache.needs.get(Hq)
    if need is None:
        need = cache.needs[Hq] = lib.dit_paged_attention_workspace_bytes(Hq, cache.heads, D)
    ws, wp, wn = _workspace(workspace, need, q, stream)
    width = pages.shape[1]
    _call(dev, lib.dit_paged_attention, "dit_paged_attention", at + _SIZE,
          None if lse is None else lse.data_ptr(), at, cache.address, pages.data_ptr(),
          pages.stride(0) if B > 1 else width, width, lengths.data_ptr(), B, Hq,
          D ** -0.5 if scale is None else scale,
          # (of 64 bits there; no sequence is as long)
          max(-1, min(int(window), 1 << 62)), ID_CODES[lengths.dtype], dt, wp, wn,
          _stream(dev, stream))
    return out, lse
