"""A synthetic token transformer: the memory-bound row path of a pre-norm
language model's step, with attention and MLP replaced by stand-in updates (as
``chain`` does for the diffusion transformer's blocks).

With x the residual stream, w_k the weight of site k (two per block) and f_k
the stand-in of site k, an elementwise product f_k(y) = y * a_k with a fixed
[tokens, D] tensor a_k:

    x = embedding(ids, table, scale)
    y = rmsnorm(x, w_0)
    for each site k:
        u = f_k(y)
        x, y = add_rmsnorm(x, u, w_{k+1})      (w of the last: the final norm's)

and back, from the gradient gy of the last y:

    gx, gw_last = rmsnorm_backward(gy, x_last, w_last)
    for each site k from the last:
        gy = gx * a_k                           (the stand-in's gradient)
        gx, gw_k = rmsnorm_backward(gy, x_k, w_k, grad_residual=gx)
    gtable = embedding_backward(gx, ids, V, scale)
    clip_grads([gtable, gw_0, ..., gw_last], max_norm)

``forward`` and ``backward`` run it, on the current stream; ``decode`` is the forward pass of single
tokens with the last norm's output in E4M3.  ``capture_step`` records a whole
step in one CUDA graph.
"""
from __future__ import annotations

from ._token import (
    TensorList,
    add_rmsnorm,
    add_rmsnorm_fp8,
    clip_grads,
    embedding,
    embedding_backward,
    rmsnorm,
    rmsnorm_backward,
)
from .synth import TORCH_DTYPES, draw, seed_for

SITES_PER_BLOCK = 2


def make_inputs(tokens, V, D, blocks=2, dtype="bf16", device="cuda", seed_tag="tokens", padded=0):
    """(ids, table, weights, stand_ins): ids int64 [tokens] uniform over the
    table with the last `padded` places -1, table [V, D], 2 * blocks + 1
    weights [D], 2 * blocks stand-ins [tokens, D]; seeded."""
    import torch
    u = draw("gate", (tokens,), seed_for(seed_tag, "ids", tokens, V), "fp32", device)
    ids = ((u.double() + 1.0) * 0.5 * V).long().clamp_(0, V - 1)
    if padded:
        ids[tokens - padded:] = -1
    table = draw("mod", (V, D), seed_for(seed_tag, "table", V, D), dtype, device)
    sites = SITES_PER_BLOCK * blocks
    one = torch.ones((), dtype=torch.float32, device=device)
    weights = [(draw("mod", (D,), seed_for(seed_tag, "w", k, D), "fp32", device) + one)
               .to(TORCH_DTYPES[dtype]) for k in range(sites + 1)]
    stand_ins = [draw("gate", (tokens, D), seed_for(seed_tag, "a", k, tokens, D), dtype, device)
                 for k in range(sites)]
    return ids, table, weights, stand_ins


def forward(ids, table, weights, stand_ins, scale=1.0, eps=1e-6, keep=None):
    """The forward pass; returns (x, y) after the last site.  keep: a list that
    receives every norm's input (what backward needs), in order."""
    x = embedding(ids, table, scale)
    y = rmsnorm(x, weights[0], eps)
    for a, w in zip(stand_ins, weights[1:]):
        if keep is not None:
            keep.append(x)
        # the residual in place, unless backward needs the old one
        x, y = add_rmsnorm(x, y * a, w, eps, residual_out=None if keep is not None else x)
    if keep is not None:
        keep.append(x)
    return x, y


def backward(grad_y, ids, num_rows, weights, stand_ins, kept, scale=1.0, eps=1e-6):
    """Gradients of the table and of every weight from the gradient of the
    last y; kept: what forward kept.  Returns (grad_table, grad_weights)."""
    grads = [None] * len(weights)
    gx, grads[-1] = rmsnorm_backward(grad_y, kept[-1], weights[-1], eps)
    for k in range(len(stand_ins) - 1, -1, -1):
        gx, grads[k] = rmsnorm_backward(gx * stand_ins[k], kept[k], weights[k], eps,
                                        grad_residual=gx)
    return embedding_backward(gx, ids, num_rows, scale), grads


def decode(ids, table, weights, stand_ins, scale=1.0, eps=1e-6, group=128):
    """The forward pass of single tokens, the last norm in E4M3: returns
    (x, codes, scales)."""
    x = embedding(ids, table, scale)
    y = rmsnorm(x, weights[0], eps)
    last = len(stand_ins) - 1
    for k, (a, w) in enumerate(zip(stand_ins, weights[1:])):
        if k == last:
            return add_rmsnorm_fp8(x, y * a, w, eps, group=group, residual_out=x)
        x, y = add_rmsnorm(x, y * a, w, eps, residual_out=x)
    raise ValueError("no sites")


def step(grad_y, ids, table, weights, stand_ins, max_norm=1.0, scale=1.0, eps=1e-6):
    """Forward, backward and clipping: returns (y, clipped gradients, norm),
    the gradients as [table's, weights' ...]."""
    kept = []
    _, y = forward(ids, table, weights, stand_ins, scale, eps, keep=kept)
    gt, gw = backward(grad_y, ids, table.shape[0], weights, stand_ins, kept, scale, eps)
    grads = [gt, *gw]
    clipped, norm = clip_grads(TensorList(grads, out=grads), max_norm)
    return y, clipped, norm


def capture_step(*args, **kwargs):
    """step recorded in a CUDA graph (capturing runs nothing): returns
    (graph, the step's results, which every replay writes anew)."""
    import torch
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*args, **kwargs)
    return graph, out
