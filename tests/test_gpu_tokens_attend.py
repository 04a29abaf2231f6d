"""The operators around attention as a model uses them (tokens.py): decoding steps
over a paged cache, also replayed from one CUDA graph, and the way to rotated heads and
back in training, against the same formulas in 64 bits."""
import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300 import tokens as tk
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
HEADS = (4, 2, 32)
V, D, BLOCKS, SIZE, B = 50, 128, 2, 4, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def rms(v, w):
    return v * (v.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w


def turned(x, cos, sin):
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def setup(dtype, fp8):
    _, table, weights, stand_ins = tk.make_inputs(B, V, D, blocks=BLOCKS, dtype=dtype)
    sites = tk.make_attention(D, HEADS, BLOCKS, dtype)
    t = torch.float8_e4m3fn if fp8 else table.dtype
    caches = [dit.KVCache.empty(20, HEADS[1], SIZE, HEADS[2], t) for _ in range(BLOCKS)]
    order = torch.randperm(20, generator=torch.Generator().manual_seed(1))
    pages = order[:18].view(B, 6).int().cuda()
    freqs = dit.rotary_frequencies(HEADS[2] // 2)
    return table, weights, stand_ins, sites, caches, pages, freqs


def reference(history, table, weights, stand_ins, sites, freqs, dtype):
    """x and the last norm of the newest token of one sequence, from all its tokens so far; the
    tensors between the operators rounded as they are stored."""
    rnd = lambda v: v.to(dtype).double()
    x = rnd(table[history].double())
    angles = torch.arange(len(history), device="cuda").double()[:, None] * freqs
    cos, sin = angles.cos().float().double()[:, None], angles.sin().float().double()[:, None]
    y = rnd(rms(x, weights[0].double()))
    Hq, Hk, d = HEADS
    for k, w in enumerate(weights[1:]):
        if k % 2 == 0:
            wq, wk, a = sites[k // 2]
            qkv = rnd(y.repeat(1, 2)[:, :(Hq + 2 * Hk) * d].view(-1, Hq + 2 * Hk, d) * a.double())
            q = rnd(turned(rms(qkv[:, :Hq], wq.double()), cos, sin))
            kk = rnd(turned(rms(qkv[:, Hq:Hq + Hk], wk.double()), cos, sin)).repeat_interleave(Hq // Hk, 1)
            v = qkv[:, Hq + Hk:].repeat_interleave(Hq // Hk, 1)
            s = torch.einsum("qhd,khd->hqk", q, kk) * d ** -0.5
            s = s.masked_fill(torch.ones_like(s[0]).triu(1).bool(), float("-inf"))
            u = rnd(torch.einsum("hqk,khd->qhd", s.softmax(-1), v)).reshape(len(history), -1)
        else:
            u = rnd(y * stand_ins[k][0].double())
        x = rnd(x + u)
        y = rms(x, w.double())
        if k + 1 < len(weights) - 1:
            y = rnd(y)
    return x[-1], y[-1]


def check(x, y, want, tol):
    for got, exact in zip((x, y), want):
        assert (got.double() - exact).abs().max() <= tol * exact.abs().max()


# How far the kernels' x and y may be from the reference's: it rounds at the same places, so a difference starts where a
# value near a tie rounds otherwise, one step (bf16 2^-8, fp16 2^-11, fp32 2^-23 of it), and passes through at
# most eight stored tensors a block with gains of a few; E4M3 keys, values and last norm have half steps of 2^-4.
TOL = {("bf16", False): 0.15, ("fp16", False): 0.1, ("fp32", False): 2.0 ** -4 + 2.0 ** -10, ("fp32", True): 0.35,
       ("bf16", True): 0.35}


@pytest.mark.parametrize("dtype,fp8", list(TOL))
@pytest.mark.parametrize("captured", [False, True])
def test_decoding(dtype, fp8, captured):
    table, weights, stand_ins, sites, caches, pages, freqs = setup(dtype, fp8)
    stand_ins = [a[:1].expand(B, D).contiguous() for a in stand_ins]  # (the same for every sequence)
    steps = 9
    tokens = ((draw("gate", (B, steps), seed_for("ids", B), "fp32", "cuda") + 1) * 0.5 * V).long().clamp_(0, V - 1)
    ids, lengths = tokens[:, 0].clone(), torch.ones(B, dtype=torch.int32, device="cuda")
    run = lambda: tk.decode_attending(ids, table, weights, stand_ins, sites, HEADS, caches, pages, lengths, freqs)
    graph = None
    if captured:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
    for n in range(steps):
        ids.copy_(tokens[:, n])
        lengths.fill_(n + 1)
        if graph:
            graph.replay()
        else:
            out = run()
        x, codes, scales = out
        y = codes.float() * scales
        for b in range(B):
            check(x[b], y[b], reference(tokens[b, :n + 1], table, weights, stand_ins, sites, freqs, table.dtype),
                  TOL[dtype, fp8])


def test_a_prompt_then_a_token():
    """Keys and values written all at once serve the next token as those written one by one."""
    table, weights, stand_ins, sites, caches, pages, freqs = setup("bf16", False)
    y = draw("act", (11, D), seed_for("prompt"), "bf16", "cuda")
    t = torch.arange(11, device="cuda")
    cos, sin = dit.rotary_table(t, freqs)
    slots = pages[1].long()[t // SIZE] * SIZE + t % SIZE
    q = tk.prompt(y, sites[0], HEADS, caches[0], cos, sin, slots)
    for i in range(11):
        tk.prompt(y[i:i + 1], sites[0], HEADS, caches[1], cos[i:i + 1], sin[i:i + 1], slots[i:i + 1])
    lengths = torch.tensor([11], dtype=torch.int32, device="cuda")
    a, _ = dit.paged_attention(q[10:], caches[0], pages[1:2], lengths)
    b, _ = dit.paged_attention(q[10:], caches[1], pages[1:2], lengths)
    assert torch.equal(a, b)
    k, v = dit.cache_read(caches[0], slots)
    assert torch.equal(k, dit.cache_read(caches[1], slots)[0]) and v.shape == (11, HEADS[1], HEADS[2])


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_heads_in_training(dtype):
    """Forward and back through norm, projection and rotation against autograd of the formulas in 64 bits."""
    _, _, weights, _ = tk.make_inputs(B, V, D, blocks=1, dtype=dtype)
    site = tk.make_attention(D, HEADS, 1, dtype)[0]
    x = draw("act", (70, D), seed_for("train"), dtype, "cuda")
    cos, sin = dit.rotary_table(torch.arange(70, device="cuda"), dit.rotary_frequencies(HEADS[2] // 2))
    q, k, qkv = tk.heads_forward(x, weights[0], site, HEADS, cos, sin)
    grads = [draw("act", tuple(t.shape), seed_for("grad", n), dtype, "cuda") for n, t in
             (("q", q), ("k", k), ("v", k))]
    got = tk.heads_backward(*grads, x, qkv, weights[0], site, HEADS, cos, sin)
    leaves = [t.double().requires_grad_() for t in (x, weights[0], site[0], site[1])]
    Hq, Hk, d = HEADS
    packed = rms(leaves[0], leaves[1]).repeat(1, 2)[:, :(Hq + 2 * Hk) * d].view(-1, Hq + 2 * Hk, d) * site[2].double()
    c, s = cos.double()[:, None], sin.double()[:, None]
    outs = [turned(rms(packed[:, :Hq], leaves[2]), c, s), turned(rms(packed[:, Hq:Hq + Hk], leaves[3]), c, s),
            packed[:, Hq + Hk:]]
    torch.autograd.backward(outs, [g.double() for g in grads])
    # a few stored tensors on the way, each half a step off, relative to the largest value; sums over 70 tokens
    tol = {"fp32": 2.0 ** -16, "bf16": 2.0 ** -4}[dtype]
    for a, b in list(zip((q, k), outs)) + [(g, t.grad) for g, t in zip(got, leaves)]:
        assert (a.double() - b).abs().max() <= tol * b.abs().max()


def test_streams():
    """Each call on a stream of its own, ordered by events, gives what the current stream gives."""
    table, weights, stand_ins, sites, caches, pages, freqs = setup("bf16", True)
    y = draw("act", (B, D), seed_for("streams"), "bf16", "cuda")
    lengths = torch.full((B,), 7, dtype=torch.int32, device="cuda")
    for c in caches:
        for t in (c.k, c.v):
            t.view(torch.uint8).zero_()
        c.k_scales.zero_()
        c.v_scales.zero_()
    cos, sin = dit.rotary_table(lengths - 1, freqs)
    slots = tk.places(pages, lengths - 1, SIZE)
    want = tk.attend(y, sites[0], HEADS, caches[0], cos, sin, slots, pages, lengths)
    torch.cuda.synchronize()
    Hq, Hk, _ = HEADS
    qkv = tk.project(y, sites[0], HEADS)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hk], qkv[:, Hq + Hk:]
    streams = [torch.cuda.Stream() for _ in range(4)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    cos, sin = dit.rotary_table(lengths - 1, freqs, stream=streams[0])
    streams[1].wait_stream(streams[0])
    dit.rmsnorm_rope(q, k, sites[0][0], sites[0][1], cos, sin, out_q=q, out_k=k, stream=streams[1])
    streams[2].wait_stream(streams[1])
    dit.cache_write(caches[1], k, v, slots, stream=streams[2])
    streams[3].wait_stream(streams[2])
    out, lse = dit.paged_attention(q, caches[1], pages, lengths, need_lse=True, stream=streams[3])
    torch.cuda.current_stream().wait_stream(streams[3])
    assert torch.equal(out.view(B, -1), want) and torch.isfinite(lse).all()
