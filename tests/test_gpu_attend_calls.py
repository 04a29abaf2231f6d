"""How the operators around attention may be called: first of all while a graph is
captured, from several host threads, after a launch that the runtime rejected, on
more tokens or heads than a grid has CTAs, in graphs that are replayed with other inputs."""
import ctypes
import os
import subprocess
import sys
import threading

import pytest
import torch

import diffusion_transformer_elementwise_gb300 as dit
from _attend_ref import check_attention, check_rope, check_rope_grad, f64
from _gpu import ensure_built
from diffusion_transformer_elementwise_gb300.synth import draw, seed_for

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LAUNCH = 7  # DIT_ERR_LAUNCH


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def act(*shape, tag="", dtype="bf16"):
    return draw("act", shape, seed_for("calls", tag, *shape), dtype, "cuda")


WORK = """
def inputs(dit, torch, t, D, L, fp8):
    g = torch.Generator(device="cuda").manual_seed(D + L)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(t)
    s = dict(qkv=rand(L, 12, D), gq=rand(L, 8, D), gk=rand(L, 2, D), wq=rand(D), wk=rand(D))
    s["positions"] = torch.arange(L, device="cuda")
    s["freqs"] = dit.rotary_frequencies(D // 2)
    s["cache"] = dit.KVCache.empty(2 * L // 8 + 3, 2, 8, D, torch.float8_e4m3fn if fp8 else t)
    s["pages"] = torch.arange(2 * ((L + 7) // 8), device="cuda").int().view(2, -1).flip(1).contiguous()
    at = torch.arange(L, device="cuda")
    s["slots"] = s["pages"][1].long()[at // 8] * 8 + at % 8
    for x in (s["cache"].k, s["cache"].v):
        x.view(torch.uint8).zero_()
    if fp8:
        s["cache"].k_scales.zero_()
        s["cache"].v_scales.zero_()
    s["lengths"] = torch.tensor([3, L], device="cuda")
    return s

def work(dit, s):
    cos, sin = dit.rotary_table(s["positions"], s["freqs"])
    q, k = dit.rmsnorm_rope(s["qkv"][:, :8], s["qkv"][:, 8:10], s["wq"], s["wk"], cos, sin)
    r, _ = dit.rope(q, None, cos, sin, interleaved=True, inverse=True)
    back = dit.rmsnorm_rope_backward(s["gq"], s["gk"], s["qkv"][:, :8], s["qkv"][:, 8:10], s["wq"], s["wk"], cos, sin)
    dit.cache_write(s["cache"], k, s["qkv"][:, 10:], s["slots"])
    kk, vv = dit.cache_read(s["cache"], s["slots"], dtype=k.dtype)
    out, lse = dit.paged_attention(q[-2:], s["cache"], s["pages"], s["lengths"], need_lse=True)
    return [cos, sin, q, k, r, *back, kk, vv, out, lse]
"""
exec(WORK)
KINDS = [(torch.bfloat16, 128, 300, True), (torch.float16, 64, 77, False), (torch.float32, 128, 130, False),
         (torch.bfloat16, 34, 40, False), (torch.float32, 256, 50, True), (torch.bfloat16, 80, 2000, True)]


def same(a, b):
    return torch.equal(a.reshape(-1).contiguous().view(torch.uint8), b.reshape(-1).contiguous().view(torch.uint8))


def test_first_calls_are_captured():
    script = "import torch\nimport diffusion_transformer_elementwise_gb300 as dit\n" + WORK + f"""
kinds = {[(str(t), D, L, f) for t, D, L, f in KINDS]}
sets = [inputs(dit, torch, getattr(torch, t.split(".")[1]), D, L, f) for t, D, L, f in kinds]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = [x for s in sets for x in work(dit, s)]
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in captured]
want = [x for s in sets for x in work(dit, s)]
same = lambda a, b: torch.equal(a.reshape(-1).contiguous().view(torch.uint8), b.reshape(-1).contiguous().view(torch.uint8))
assert all(same(a, b) for a, b in zip(got, want, strict=True))
print("captured", len(captured))
"""
    r = subprocess.run([sys.executable, "-c", script], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.startswith("captured"), r.stdout + r.stderr


def test_calls_of_several_threads():
    sets = [inputs(dit, torch, *kind) for kind in KINDS]
    want = [work(dit, s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got, errors = [None] * len(sets), []
    start = threading.Barrier(len(sets))

    def run(i):
        try:
            start.wait(60)
            with torch.cuda.stream(streams[i]):
                for _ in range(20):
                    got[i] = work(dit, sets[i])
        except Exception as e:  # reported below
            errors.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(sets))]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not errors, errors
    for a, b in zip(want, got):
        assert all(same(x, y) for x, y in zip(a, b))


def test_a_rejected_launch_is_not_reported_again():
    """The launches go to a stream whose capture has been invalidated: nothing reaches the GPU."""
    driver = ctypes.CDLL("libcuda.so.1")
    s = inputs(dit, torch, torch.bfloat16, 64, 40, False)
    odd = inputs(dit, torch, torch.float32, 34, 40, False)
    cos, sin = dit.rotary_table(s["positions"], s["freqs"])
    ocos, osin = dit.rotary_table(odd["positions"], odd["freqs"])
    ws = torch.zeros(1 << 23, dtype=torch.uint8, device="cuda")
    out, q = torch.empty(2, 8, 64, dtype=torch.bfloat16, device="cuda"), s["gq"][:2]
    gq, ogq = torch.empty_like(s["gq"]), torch.empty_like(odd["gq"])
    gw, ogw = torch.empty_like(s["wq"]), torch.empty_like(odd["wq"])
    oo = torch.empty(2, 8, 34, device="cuda")
    made = {
        "table": lambda st: dit.rotary_table(s["positions"], s["freqs"], cos=cos, sin=sin, stream=st),
        "rope": lambda st: dit.rope(s["gq"], None, cos, sin, out_q=gq, stream=st),
        "rope, any view": lambda st: dit.rope(odd["gq"], None, ocos, osin, out_q=ogq, stream=st),
        "gradient": lambda st: dit.rmsnorm_rope_backward(s["gq"], None, s["gq"], None, s["wq"], None, cos, sin,
                                                         grad_q=gq, grad_weight_q=gw, workspace=ws, stream=st),
        "gradient, any view": lambda st: dit.rmsnorm_rope_backward(
            odd["gq"], None, odd["gq"], None, odd["wq"], None, ocos, osin, grad_q=ogq, grad_weight_q=ogw,
            workspace=ws, stream=st),
        "write": lambda st: dit.cache_write(s["cache"], s["gk"], s["gk"], s["slots"], stream=st),
        "read": lambda st: dit.cache_read(s["cache"], s["slots"], k=torch.empty_like(s["gk"]), v=torch.empty_like(s["gk"]),
                                          stream=st),
        "attention": lambda st: dit.paged_attention(q, s["cache"], s["pages"], s["lengths"], out=out, workspace=ws,
                                                    stream=st),
        "attention, any rows": lambda st: dit.paged_attention(odd["gq"][:2], odd["cache"], odd["pages"], odd["lengths"],
                                                              out=oo, workspace=ws, stream=st)}
    for call in made.values():
        call(None)
    torch.cuda.synchronize()
    for name, call in made.items():
        side = torch.cuda.Stream()
        handle = ctypes.c_void_p(side.cuda_stream)
        relaxed = 2
        assert driver.cuStreamBeginCapture_v2(handle, relaxed) == 0
        assert driver.cuStreamSynchronize(handle) != 0  # invalidates the capture
        with pytest.raises(dit.DitError) as refused:
            call(side)
        graph = ctypes.c_void_p()
        assert driver.cuStreamEndCapture(handle, ctypes.byref(graph)) != 0
        assert refused.value.status == LAUNCH, name
        for other in made.values():
            other(None)
            other(side)
        torch.cuda.synchronize()


@pytest.mark.parametrize("tokens,Hq,Hk,D", [(300_000, 1, 1, 8), (3, 3000, 700, 16), (70_000, 2, 0, 10), (1, 9000, 1, 64)])
def test_many_tokens_and_heads(tokens, Hq, Hk, D):
    q, k = act(tokens, Hq, D, tag="q"), act(tokens, Hk, D, tag="k")
    gq, gk = act(tokens, Hq, D, tag="gq"), act(tokens, Hk, D, tag="gk")
    w = act(D, tag="w")
    a = act(tokens, D // 2, tag="a", dtype="fp32").double()
    cos, sin = a.cos().float(), a.sin().float()
    keys = (k, w, gk) if Hk else (None, None, None)
    got = dit.rmsnorm_rope(q, keys[0], w, keys[1], cos, sin)
    back = dit.rmsnorm_rope_backward(gq, keys[2], q, keys[0], w, keys[1], cos, sin)
    for i, (x, g) in enumerate(((q, gq), (k, gk))[:2 if Hk else 1]):
        check_rope(got[i], x, cos, sin, w)
        check_rope_grad(back[i], back[2 + i], g, x, cos, sin, w)


def test_many_slots():
    x = act(200_000, 1, 16, tag="slots")
    cache = dit.KVCache.empty(200_001, 1, 1, 16)
    slots = torch.randperm(200_001, generator=torch.Generator().manual_seed(2))[:200_000].cuda()
    dit.cache_write(cache, x, -x, slots)
    k, v = dit.cache_read(cache, slots)
    assert torch.equal(k, x) and torch.equal(v, -x)


def test_a_graph_with_other_lengths_and_pages():
    """The sizes of a captured call are the tables'; lengths, pages and rows may change from replay to
    replay."""
    s = inputs(dit, torch, torch.bfloat16, 128, 4000, False)
    cache, pages = s["cache"], s["pages"]
    lengths = torch.tensor([1, 1], device="cuda")
    k = act(4000, 2, 128, tag="gk")
    both = torch.cat([pages[b].long()[torch.arange(4000, device="cuda") // 8] * 8 + torch.arange(4000, device="cuda") % 8
                      for b in (0, 1)])
    dit.cache_write(cache, torch.cat((k, k.flip(0))), torch.cat((k * 0.5, k)), both)
    q = act(2, 8, 128, tag="gq")
    dit.paged_attention(q, cache, pages, lengths, need_lse=True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = dit.paged_attention(q, cache, pages, lengths, need_lse=True)
    kd, vd = f64(torch.stack((k, k.flip(0)))), f64(torch.stack((k * 0.5, k)))
    for n in ([4000, 0], [33, 3999], [0, 0], [1, 64], [2000, 2000]):
        lengths.copy_(torch.tensor(n))
        q.mul_(-1.0)
        graph.replay()
        check_attention(out, lse, q, lambda b, h: kd[b, :n[b], h // 4], lambda b, h: vd[b, :n[b], h // 4], n, 128 ** -0.5)
    swapped = pages.flip(0).contiguous()
    pages.copy_(swapped)
    lengths.copy_(torch.tensor([700, 31]))
    graph.replay()
    n = [700, 31]
    check_attention(out, lse, q, lambda b, h: kd[1 - b, :n[b], h // 4], lambda b, h: vd[1 - b, :n[b], h // 4], n, 128 ** -0.5)


def test_no_pages():
    """A page table without columns, and a cache without pages: no token anywhere."""
    for t in (torch.bfloat16, torch.float32):
        q = torch.ones(3, 4, 64, dtype=t, device="cuda")
        lengths = torch.tensor([5, 0, 9], device="cuda")
        for cache, width in ((dit.KVCache.empty(4, 2, 16, 64, t), 0), (dit.KVCache.empty(0, 2, 16, 64, t), 3)):
            out, lse = dit.paged_attention(q, cache, torch.zeros(3, width, dtype=torch.int32, device="cuda"), lengths,
                                           need_lse=True)
            assert (out == 0).all() and (lse == -float("inf")).all()
    dit.cache_write(cache, q[:, :2], q[:, :2], torch.tensor([0, 1, 2], device="cuda"))
    k, v = dit.cache_read(cache, torch.tensor([0, 1, 2], device="cuda"))
    assert (k == 0).all() and (v == 0).all()


def test_graphs_of_other_nodes():
    """Captured behind a fill, a copy and the ends of two forked streams, which are no kernels of this library."""
    s = inputs(dit, torch, torch.bfloat16, 64, 200, True)
    want = work(dit, s)
    torch.cuda.synchronize()
    source = {n: s[n].clone() for n in ("qkv", "positions", "slots", "lengths", "pages")}
    side = [torch.cuda.Stream() for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        for n, st in (("qkv", side[0]), ("positions", side[1])):
            st.wait_stream(main)
            with torch.cuda.stream(st):
                s[n].zero_()
                s[n].copy_(source[n])
        s["cache"].k.view(torch.uint8).zero_()
        s["cache"].v.view(torch.uint8).zero_()
        s["cache"].k_scales.zero_()
        s["cache"].v_scales.zero_()
        for st in side:
            main.wait_stream(st)
        cos, sin = dit.rotary_table(s["positions"], s["freqs"])
        s["slots"].zero_()
        s["slots"].copy_(source["slots"])
        got = work(dit, s)
    for _ in range(3):
        for n in ("qkv", "positions", "slots"):
            s[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want, strict=True))
        assert same(cos, want[0])


def test_rows_written_in_place_by_the_call_before():
    """A chain of calls that read what the one before has just written in place, in views of any kind."""
    for t, D in ((torch.bfloat16, 34), (torch.float32, 35), (torch.bfloat16, 128)):
        L = 700
        qkv = act(L, 4, D, tag="chain").to(t)
        w = act(D, tag="w").to(t)
        cos, sin = dit.rotary_table(torch.arange(L, device="cuda"), dit.rotary_frequencies(D // 2))
        cache = dit.KVCache.empty(L // 4, 1, 4, D, t)
        slots = torch.arange(L, device="cuda")
        pages = torch.arange(L // 4, device="cuda").int()[None].expand(L, -1).contiguous()
        lengths = slots + 1
        outs = []
        for _ in range(6):
            x = qkv.clone()
            q, k, v = x[:, :2], x[:, 2:3], x[:, 3:]
            dit.rmsnorm_rope(q, k, w, w, cos, sin, out_q=q, out_k=k)
            dit.rope(q, k, cos, sin, inverse=True, out_q=q, out_k=k)
            dit.rope(q, k, cos, sin, out_q=q, out_k=k)
            dit.cache_write(cache, k, v, slots)
            out, _ = dit.paged_attention(q, cache, pages, lengths)
            outs.append((x, out))
        torch.cuda.synchronize()
        x = qkv.clone()
        steps = [lambda: dit.rmsnorm_rope(x[:, :2], x[:, 2:3], w, w, cos, sin, out_q=x[:, :2], out_k=x[:, 2:3]),
                 lambda: dit.rope(x[:, :2], x[:, 2:3], cos, sin, inverse=True, out_q=x[:, :2], out_k=x[:, 2:3]),
                 lambda: dit.rope(x[:, :2], x[:, 2:3], cos, sin, out_q=x[:, :2], out_k=x[:, 2:3]),
                 lambda: dit.cache_write(cache, x[:, 2:3], x[:, 3:], slots)]
        for step in steps:
            step()
            torch.cuda.synchronize()
        out, _ = dit.paged_attention(x[:, :2], cache, pages, lengths)
        for a, b in outs:
            assert torch.equal(a, x) and torch.equal(b, out)
