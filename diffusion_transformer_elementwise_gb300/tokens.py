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

``decode_attending`` is the decoding step with attention at every first site
of a block: queries, keys and values come from the stand-in of the packed
projection, y's columns (over again, as often as it takes) times a fixed tensor, as
[B, Hq + 2 Hk, head_dim]; then

    q, k = rmsnorm_rope(q, k, w_q, w_k, cos, sin)       (in place, within the packed tensor)
    cache_write(cache, k, v, slots)
    u = paged_attention(q, cache, pages, lengths)

with cos and sin of the tokens' positions, which all sites share.
``prompt`` writes the keys and values of tokens that came before, and
``heads_forward`` and ``heads_backward`` are the same site in training, up to the rotated
queries and keys and back.
"""
from __future__ import annotations

from ._attend import (
    cache_write,
    paged_attention,
    rmsnorm_rope,
    rmsnorm_rope_backward,
    rotary_table,
)
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


def make_attention(width, heads, sites, dtype="bf16", device="cuda", seed_tag="attention"):
    """Parameters of attention sites for rows of `width` columns, heads = (Hq, Hk, head_dim): a list of (w_q,
    w_k, a), weights [head_dim] and the projection's stand-in [Hq + 2 Hk, head_dim]; seeded."""
    import torch
    Hq, Hk, d = heads
    one = torch.ones((), dtype=torch.float32, device=device)
    made = []
    for k in range(sites):
        w = [(draw("mod", (d,), seed_for(seed_tag, n, k, d), "fp32", device) + one)
             .to(TORCH_DTYPES[dtype]) for n in ("q", "k")]
        made.append((*w, draw("gate", (Hq + 2 * Hk, d), seed_for(seed_tag, "a", k, width, Hq, Hk, d), dtype,
                              device)))
    return made


def project(y, site, heads):
    """The stand-in of the packed projection: [tokens, Hq + 2 Hk, head_dim]."""
    Hq, Hk, d = heads
    n = (Hq + 2 * Hk) * d
    return y.repeat(1, -(-n // y.shape[1]))[:, :n].view(-1, Hq + 2 * Hk, d) * site[2]


def places(pages, positions, page_size):
    """The cache's places of each sequence's token at positions[b], -1 where it has none: before the start (an empty
    sequence's last token), behind the page table, or where there is no page."""
    import torch
    at, width = positions.long(), pages.shape[1]
    if width == 0:
        return torch.full_like(at, -1)
    page = pages.gather(1, (at // page_size).clamp_(0, width - 1)[:, None])[:, 0].long()
    there = (at >= 0) & (at < width * page_size) & (page >= 0)
    return torch.where(there, page * page_size + at % page_size, -1)


def prompt(y, site, heads, cache, cos, sin, slots, eps=1e-6):
    """Write the keys and values of tokens y [tokens, D] to their places; returns their rotated
    queries."""
    Hq, Hk, _ = heads
    qkv = project(y, site, heads)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    rmsnorm_rope(q, k, site[0], site[1], cos, sin, eps, out_q=q, out_k=k)
    cache_write(cache, k, v, slots)
    return q


def attend(y, site, heads, cache, cos, sin, slots, pages, lengths, eps=1e-6):
    """The update of one new token per sequence: y [B, D] to [B, Hq * head_dim]."""
    q = prompt(y, site, heads, cache, cos, sin, slots, eps)
    out, _ = paged_attention(q, cache, pages, lengths)
    return out.view(y.shape[0], -1)


def decode_attending(ids, table, weights, stand_ins, sites, heads, caches, pages, lengths, freqs,
                     scale=1.0, eps=1e-6, group=128):
    """One decoding step of B sequences: ids [B] are their new tokens, lengths [B] count them in (0: an idle row of a padded
    batch; a token without a place is not written, and attention takes the tokens that the page table holds).  sites
    and caches: one for each block (make_attention, KVCache); the second site of a
    block has its stand-in, stand_ins[1::2].  Hq * head_dim is the width D.
    Returns (x, codes, scales), the last norm in E4M3."""
    cos, sin = rotary_table(lengths - 1, freqs)
    x = embedding(ids, table, scale)
    y = rmsnorm(x, weights[0], eps)
    last = len(stand_ins) - 1
    for k, w in enumerate(weights[1:]):
        if k % SITES_PER_BLOCK == 0:
            cache = caches[k // SITES_PER_BLOCK]
            u = attend(y, sites[k // SITES_PER_BLOCK], heads, cache, cos, sin,
                       places(pages, lengths - 1, cache.page_size), pages, lengths, eps)
        else:
            u = y * stand_ins[k]
        if k == last:
            return add_rmsnorm_fp8(x, u, w, eps, group=group, residual_out=x)
        x, y = add_rmsnorm(x, u, w, eps, residual_out=x)
    raise ValueError("no sites")


def heads_forward(x, weight, site, heads, cos, sin, eps=1e-6):
    """Training's way to rotated queries and keys: norm, projection, norm and rotation of the heads.
    Returns (q, k, qkv); backward needs qkv and x."""
    Hq, Hk, _ = heads
    qkv = project(rmsnorm(x, weight, eps), site, heads)
    q, k = rmsnorm_rope(qkv[:, :Hq], qkv[:, Hq:Hq + Hk], site[0], site[1], cos, sin, eps)
    return q, k, qkv


def heads_backward(grad_q, grad_k, grad_v, x, qkv, weight, site, heads, cos, sin, eps=1e-6):
    """Gradients (of x, the norm's weight, w_q, w_k) from those of the rotated queries and keys and of the
    values."""
    import torch
    Hq, Hk, d = heads
    grad = torch.empty_like(qkv)
    _, _, gwq, gwk = rmsnorm_rope_backward(
        grad_q, grad_k, qkv[:, :Hq], qkv[:, Hq:Hq + Hk], site[0], site[1], cos, sin, eps,
        grad_q=grad[:, :Hq], grad_k=grad[:, Hq:Hq + Hk])
    grad[:, Hq + Hk:] = grad_v
    # the projection's stand-in repeats y's columns: their gradients add up
    n, D = (Hq + 2 * Hk) * d, x.shape[1]
    g = torch.nn.functional.pad((grad.float() * site[2].float()).view(-1, n), (0, -n % D))
    gy = g.view(x.shape[0], -1, D).sum(1).to(x.dtype)
    gx, gw = rmsnorm_backward(gy, x, weight, eps)
    return gx, gw, gwq, gwk


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
