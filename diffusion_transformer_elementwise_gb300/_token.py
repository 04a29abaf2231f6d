"""The token-transformer operators of libdit_elementwise.so
(include/dit_elementwise.h): weighted RMSNorm with the residual's addition and
an E4M3 output, its gradient, the embedding lookup and its gradient, the
global gradient norm and clipping.

Argument marshalling, as in ``_binding``: contiguous CUDA tensors of one dtype,
the current torch stream unless ``stream`` says otherwise, :class:`DitError`
on a non-OK status.  A tensor has any number of dimensions; its last one is
the row.  What a call allocates (outputs not given, workspaces) comes from the
stream it launches on.  No function takes part in autograd: the gradients are
functions of their own.
"""
from __future__ import annotations

import ctypes
import math

import torch

from ._binding import _FP8, DTYPE_CODES, _cuda, _dtype, _stream, check, library

ID_CODES = {torch.int32: 0, torch.int64: 1}


class Tensor(ctypes.Structure):
    """dit_tensor of include/dit_elementwise.h."""
    _fields_ = [("g", ctypes.c_void_p), ("out", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("dtype", ctypes.c_int64)]


def declare(lib) -> None:
    """The argument types of the entry points."""
    vp, i64, ci, cf = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    for name, args in (
            ("dit_rmsnorm", [vp] * 3 + [i64, i64, cf, cf, ci, vp]),
            ("dit_add_rmsnorm", [vp] * 5 + [i64, i64, cf, cf, ci, vp]),
            ("dit_rmsnorm_fp8", [vp] * 4 + [i64, i64, i64, cf, cf, ci, vp]),
            ("dit_add_rmsnorm_fp8", [vp] * 6 + [i64, i64, i64, cf, cf, ci, vp]),
            ("dit_rmsnorm_backward", [vp] * 6 + [i64, i64, cf, cf, ci, vp, i64, vp]),
            ("dit_embedding", [vp] * 3 + [i64, i64, i64, cf, ci, ci, vp]),
            ("dit_embedding_backward", [vp] * 3 + [i64, i64, i64, cf, ci, ci, vp, i64, vp]),
            ("dit_grad_norm", [vp, vp, i64, vp, i64, vp]),
            ("dit_clip_grads", [vp, vp, i64, cf, cf, vp, i64, vp])):
        getattr(lib, name).argtypes = args
        getattr(lib, name).restype = ci
    for name, n in (("dit_rmsnorm_backward_workspace_bytes", 2),
                    ("dit_embedding_backward_workspace_bytes", 2),
                    ("dit_grad_norm_workspace_bytes", 1)):
        getattr(lib, name).argtypes = [i64] * n
        getattr(lib, name).restype = i64


def _empty(shape, dtype, device, stream):
    """A tensor from the memory of the stream that the call launches on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle
                  else torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(given, nbytes, ref, stream):
    """(tensor, address, size) of the caller's workspace, or of a new one."""
    if nbytes < 0:
        raise ValueError("sizes out of range")
    if nbytes == 0:
        return None, None, 0
    if given is None:
        given = _empty((nbytes,), torch.uint8, ref.device, stream)
    else:
        _cuda(("workspace", given), ("", ref))
    return given, given.data_ptr(), given.numel() * given.element_size()


# (a torch without the private name still imports the package)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(dev, fn, what, *args):
    """The C entry point with `dev` as the current device; raises on a status."""
    if _get_device() == dev:
        st = fn(*args)
    else:
        with torch.cuda.device(dev):
            st = fn(*args)
    if st:
        check(st, what)


def _rows(x, name):
    """(rows, D) of a tensor whose last dimension is the row."""
    if not isinstance(x, torch.Tensor) or x.dim() < 1:
        raise ValueError(f"{name} must be a tensor of at least one dimension")
    D = x.shape[-1]
    return (x.numel() // D if D else math.prod(x.shape[:-1])), D


def _same(x, named, weight=None, D=0):
    """Checks that the tensors of `named` (name, tensor, ...; x among them) are
    contiguous, of x's shape and dtype, on its CUDA device, and the weight [D].
    Returns (device index, dtype code).  The usual case takes one pass; what
    is wrong is found out in a second."""
    try:
        shape, dtype, dev = x.shape, x.dtype, x.get_device()
        ok = dev >= 0 and dtype in DTYPE_CODES
        for t in named[1::2]:
            ok = (ok and t.dtype is dtype and t.is_contiguous() and t.get_device() == dev
                  and t.shape == shape)
        if weight is not None:
            ok = (ok and weight.dtype is dtype and weight.is_contiguous()
                  and weight.get_device() == dev and weight.dim() == 1 and weight.numel() == D)
    except AttributeError:
        ok = False
    if ok:
        return dev, DTYPE_CODES[dtype]
    pairs = list(zip(named[::2], named[1::2]))
    if weight is not None:
        pairs.append(("weight", weight))
    dev = _cuda(*pairs)
    dt = _dtype(x, *pairs)
    for name, t in zip(named[::2], named[1::2]):
        if t.shape != x.shape:
            raise ValueError(f"{name} must have the shape {tuple(x.shape)}, got {tuple(t.shape)}")
    if weight is not None and weight.shape != (D,):
        raise ValueError(f"weight must be [{D}], got {tuple(weight.shape)}")
    return dev, dt


def rmsnorm(x, weight, eps=1e-6, weight_offset=0.0, out=None, stream=None):
    """out = rms_norm(x, eps) * (weight_offset + weight) over the last
    dimension; weight [D], weight_offset 1 for a weight stored as its
    difference from one.  Returns out."""
    rows, D = _rows(x, "x")
    if out is None:
        out = _empty(x.shape, x.dtype, x.device, stream)
    dev, dt = _same(x, ("x", x, "out", out), weight, D)
    _call(dev, library().dit_rmsnorm, "dit_rmsnorm", out.data_ptr(), x.data_ptr(),
          weight.data_ptr(), rows, D, eps, weight_offset, dt, _stream(dev, stream))
    return out


def add_rmsnorm(hidden, update, weight, eps=1e-6, weight_offset=0.0, residual_out=None, out=None,
                stream=None):
    """residual_out = hidden + update; out = rms_norm(residual_out, eps) *
    (weight_offset + weight), in one pass.  Pass residual_out=hidden to update
    the residual in place.  Returns (residual_out, out)."""
    rows, D = _rows(hidden, "hidden")
    if residual_out is None:
        residual_out = _empty(hidden.shape, hidden.dtype, hidden.device, stream)
    if out is None:
        out = _empty(hidden.shape, hidden.dtype, hidden.device, stream)
    dev, dt = _same(hidden, ("hidden", hidden, "update", update, "residual_out", residual_out,
                             "out", out), weight, D)
    _call(dev, library().dit_add_rmsnorm, "dit_add_rmsnorm", residual_out.data_ptr(),
          out.data_ptr(), hidden.data_ptr(), update.data_ptr(), weight.data_ptr(), rows, D, eps,
          weight_offset, dt, _stream(dev, stream))
    return residual_out, out


def _codes(x, D, group, out, scales, stream):
    """The E4M3 output (float8_e4m3fn or uint8) and its scales."""
    if group not in (0, 128):
        raise ValueError("group must be 0 (one scale per row) or 128 (one per 128 columns)")
    if out is None:
        out = _empty(x.shape, _FP8 or torch.uint8, x.device, stream)
    elif out.dtype is not _FP8 and out.dtype is not torch.uint8:
        raise TypeError(f"out must be float8_e4m3fn or uint8, got {out.dtype}")
    shape = tuple(x.shape[:-1]) + ((D + 127) // 128 if group else 1,)
    if scales is None:
        scales = _empty(shape, torch.float32, x.device, stream)
    elif scales.dtype is not torch.float32 or scales.shape != shape:
        raise ValueError(f"scales must be float32 {shape}, got {scales.dtype} {tuple(scales.shape)}")
    if out.shape != x.shape:
        raise ValueError(f"out must have the shape {tuple(x.shape)}, got {tuple(out.shape)}")
    dev = x.get_device()
    if (out.get_device() != dev or scales.get_device() != dev or not out.is_contiguous()
            or not scales.is_contiguous()):
        _cuda(("x", x), ("out", out), ("scales", scales))
    return out, scales


def rmsnorm_fp8(x, weight, eps=1e-6, group=0, weight_offset=0.0, out=None, scales=None,
                stream=None):
    """rms_norm(x, eps) * (weight_offset + weight) as E4M3 codes and scales:
    the value is code * scale.  group=0: one scale per row ([..., 1]);
    group=128: one per 128 columns ([..., ceil(D / 128)]).  Returns
    (out, scales); out is float8_e4m3fn, or the uint8 tensor given."""
    rows, D = _rows(x, "x")
    out, scales = _codes(x, D, group, out, scales, stream)
    dev, dt = _same(x, ("x", x), weight, D)
    _call(dev, library().dit_rmsnorm_fp8, "dit_rmsnorm_fp8", out.data_ptr(), scales.data_ptr(),
          x.data_ptr(), weight.data_ptr(), rows, D, group, eps, weight_offset, dt,
          _stream(dev, stream))
    return out, scales


def add_rmsnorm_fp8(hidden, update, weight, eps=1e-6, group=0, weight_offset=0.0,
                    residual_out=None, out=None, scales=None, stream=None):
    """residual_out = hidden + update (the dtype of hidden), and its weighted
    norm as E4M3 codes and scales (rmsnorm_fp8), in one pass.  Returns
    (residual_out, out, scales)."""
    rows, D = _rows(hidden, "hidden")
    if residual_out is None:
        residual_out = _empty(hidden.shape, hidden.dtype, hidden.device, stream)
    out, scales = _codes(hidden, D, group, out, scales, stream)
    dev, dt = _same(hidden, ("hidden", hidden, "update", update, "residual_out", residual_out),
                    weight, D)
    _call(dev, library().dit_add_rmsnorm_fp8, "dit_add_rmsnorm_fp8", residual_out.data_ptr(),
          out.data_ptr(), scales.data_ptr(), hidden.data_ptr(), update.data_ptr(),
          weight.data_ptr(), rows, D, group, eps, weight_offset, dt, _stream(dev, stream))
    return residual_out, out, scales


def rmsnorm_backward(grad_out, x, weight, eps=1e-6, weight_offset=0.0, grad_residual=None,
                     grad_x=None, grad_weight=None, need_weight=True, workspace=None, stream=None):
    """Gradients of rmsnorm(x, weight): returns (grad_x, grad_weight).  For
    add_rmsnorm, x is its residual_out, grad_residual the gradient that
    arrives at residual_out on the skip path, and grad_x the gradient of
    hidden and of update alike.  need_weight=False (a frozen weight): grad_weight is
    not computed and None is returned for it.  grad_x may be grad_out or
    grad_residual.  workspace: a uint8 CUDA tensor of at least
    dit_rmsnorm_backward_workspace_bytes(rows, D) bytes (allocated if None)."""
    rows, D = _rows(x, "x")
    if grad_x is None:
        grad_x = _empty(x.shape, x.dtype, x.device, stream)
    if not need_weight:
        grad_weight = None
    elif grad_weight is None:
        grad_weight = _empty((D,), x.dtype, x.device, stream)
    named = ("x", x, "grad_out", grad_out, "grad_x", grad_x)
    if grad_residual is not None:
        named += ("grad_residual", grad_residual)
    dev, dt = _same(x, named, weight, D)
    lib = library()
    ws, wp, wn, gw, gr = None, None, 0, None, None
    if grad_weight is not None:
        if (grad_weight.dtype is not x.dtype or grad_weight.get_device() != dev
                or grad_weight.shape != (D,) or not grad_weight.is_contiguous()):
            raise ValueError(f"grad_weight must be a contiguous [{D}] {x.dtype} tensor on cuda:{dev}")
        gw = grad_weight.data_ptr()
        ws, wp, wn = _workspace(workspace, lib.dit_rmsnorm_backward_workspace_bytes(rows, D), x, stream)
    if grad_residual is not None:
        gr = grad_residual.data_ptr()
    _call(dev, lib.dit_rmsnorm_backward, "dit_rmsnorm_backward", grad_x.data_ptr(), gw,
          grad_out.data_ptr(), gr, x.data_ptr(), weight.data_ptr(), rows, D, eps, weight_offset, dt,
          wp, wn, _stream(dev, stream))
    return grad_x, grad_weight


def _with_ids(ids, t, named):
    """Checks ids and the tensors of `named` (name, tensor, ...) against t, one
    of them; returns (device index, dtype code)."""
    dev = t.get_device()
    ok = dev >= 0 and t.dtype in DTYPE_CODES and ids.get_device() == dev and ids.is_contiguous()
    for o in named[1::2]:
        ok = ok and o.dtype is t.dtype and o.get_device() == dev and o.is_contiguous()
    if ok:
        return dev, DTYPE_CODES[t.dtype]
    pairs = list(zip(named[::2], named[1::2]))
    dev = _cuda(*pairs, ("ids", ids))
    return dev, _dtype(t, *pairs)


def _id_type(ids):
    if not isinstance(ids, torch.Tensor) or ids.dtype not in ID_CODES:
        raise TypeError("ids must be an int32 or int64 CUDA tensor")
    return ID_CODES[ids.dtype]


def embedding(ids, table, scale=1.0, out=None, stream=None):
    """out[..., :] = table[ids[...]] * scale; a row of zeros where an id is
    outside [0, V) (e.g. -1 for a padded place).  ids: int32 or int64, any
    shape; table [V, D].  Returns out (ids.shape + (D,))."""
    it = _id_type(ids)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be [V, D]")
    V, D = table.shape
    shape = tuple(ids.shape) + (D,)
    if out is None:
        out = _empty(shape, table.dtype, table.device, stream)
    elif out.shape != shape:
        raise ValueError(f"out must be {shape}, got {tuple(out.shape)}")
    dev, dt = _with_ids(ids, table, ("table", table, "out", out))
    _call(dev, library().dit_embedding, "dit_embedding", out.data_ptr(), ids.data_ptr(),
          table.data_ptr(), ids.numel(), V, D, scale, dt, it, _stream(dev, stream))
    return out


def embedding_backward(grad_out, ids, num_rows, scale=1.0, out=None, workspace=None, stream=None):
    """Gradient of embedding(ids, table, scale) for a table of num_rows rows:
    out[v] = scale * the sum of grad_out's rows whose id is v, zeros where no
    token names v; ids outside [0, num_rows) take no part.  Tokens are sorted
    by id, so the same call gives the same bits.  workspace: a uint8 CUDA
    tensor of at least dit_embedding_backward_workspace_bytes(tokens, D) bytes
    (allocated if None).  Returns out ([num_rows, D])."""
    it = _id_type(ids)
    tokens, D = _rows(grad_out, "grad_out")
    if grad_out.shape[:-1] != ids.shape:
        raise ValueError(f"grad_out must be ids.shape + (D,), got {tuple(grad_out.shape)} for ids "
                         f"{tuple(ids.shape)}")
    V = int(num_rows)
    if V < 0:
        raise ValueError("num_rows must not be negative")
    if out is None:
        out = _empty((V, D), grad_out.dtype, grad_out.device, stream)
    elif out.shape != (V, D):
        raise ValueError(f"out must be [{V}, {D}], got {tuple(out.shape)}")
    dev, dt = _with_ids(ids, grad_out, ("grad_out", grad_out, "out", out))
    lib = library()
    ws, wp, wn = _workspace(workspace, lib.dit_embedding_backward_workspace_bytes(tokens, D), grad_out,
                            stream)
    _call(dev, lib.dit_embedding_backward, "dit_embedding_backward", out.data_ptr(),
          grad_out.data_ptr(), ids.data_ptr(), tokens, V, D, scale, dt, it, wp, wn,
          _stream(dev, stream))
    return out


class TensorList:
    """The description of many tensors (and of one output for each, or
    out=None) that grad_norm and clip_grads take: made once for gradients that
    keep their memory from step to step.  It holds the tensors; replacing a
    tensor's storage (set_, resize_) after this makes the list stale.

    Tensors: contiguous, on one CUDA device, bf16, fp16 or fp32 each.  An output
    has its tensor's dtype and size, and may be the tensor itself."""

    def __init__(self, tensors, out=None):
        self.tensors = list(tensors)
        self.out = None if out is None else list(out)
        if self.out is not None and len(self.out) != len(self.tensors):
            raise ValueError(f"{len(self.tensors)} tensors, but {len(self.out)} outputs")
        self.array = (Tensor * max(1, len(self.tensors)))()
        self.address = ctypes.addressof(self.array)
        self.device = None
        for i, t in enumerate(self.tensors):
            o = None if self.out is None else self.out[i]
            named = (("tensor %d" % i, t),) + ((("output %d" % i, o),) if o is not None else ())
            _cuda(*named)
            if self.device is None:
                self.device = t.device
            elif t.device != self.device:
                raise ValueError(f"tensor {i} is on {t.device}, expected {self.device}")
            dt = _dtype(t, *named[1:])
            if o is not None and o.shape != t.shape:
                raise ValueError(f"output {i} must have the shape {tuple(t.shape)}")
            self.array[i] = Tensor(t.data_ptr(), None if o is None else o.data_ptr(), t.numel(), dt)

    def __len__(self):
        return len(self.tensors)


def _norm_call(lst, norm, workspace, stream):
    """(norm, workspace tensor, address, size) of a call over a list."""
    if not len(lst):
        raise ValueError("no tensors")
    ref = lst.tensors[0]
    if norm is None:
        norm = _empty((), torch.float32, ref.device, stream)
    else:
        _cuda(("norm", norm), ("tensor 0", ref))
        if norm.dtype is not torch.float32 or norm.numel() != 1:
            raise TypeError("norm must be a one-element float32 CUDA tensor")
    ws, wp, wn = _workspace(workspace, library().dit_grad_norm_workspace_bytes(len(lst)), ref, stream)
    return norm, ws, wp, wn


def grad_norm(tensors, norm=None, workspace=None, stream=None):
    """The 2-norm over all elements of all tensors (a list, or a TensorList),
    as a float32 CUDA scalar.  workspace: a uint8 CUDA tensor of at least
    dit_grad_norm_workspace_bytes(len(tensors)) bytes (allocated if None)."""
    lst = tensors if isinstance(tensors, TensorList) else TensorList(tensors)
    norm, ws, wp, wn = _norm_call(lst, norm, workspace, stream)
    dev = norm.get_device()
    _call(dev, library().dit_grad_norm, "dit_grad_norm", norm.data_ptr(), lst.address, len(lst), wp,
          wn, _stream(dev, stream))
    return norm


def clip_grads(grads, max_norm, eps=1e-6, out=None, norm=None, workspace=None, stream=None):
    """out[i] = grads[i] * min(1, max_norm / (norm + eps)) with the 2-norm
    over all of them.  Pass out=grads for the in-place form; out=None
    allocates.  grads may be a TensorList with its outputs (out is then not
    given).  Returns (outputs, norm): norm is a float32 CUDA scalar, the norm
    before clipping.  workspace as for grad_norm."""
    if isinstance(grads, TensorList):
        if out is not None or grads.out is None:
            raise ValueError("a TensorList brings its own outputs: make it with out=")
        lst = grads
    else:
        grads = list(grads)
        if out is None:
            out = [_empty(g.shape, g.dtype, g.device, stream) for g in grads]
        lst = TensorList(grads, out)
    norm, ws, wp, wn = _norm_call(lst, norm, workspace, stream)
    dev = norm.get_device()
    _call(dev, library().dit_clip_grads, "dit_clip_grads", norm.data_ptr(), lst.address, len(lst),
          max_norm, eps, wp, wn, _stream(dev, stream))
    return lst.out, norm
