"""Performance cases of the operators around attention.

One case is one call of one operator at one size: the table of rotary angles,
the norm of queries and keys per head with the rotation in the same pass, its
gradient, rows written into and read back from a paged key-value cache (in
the tensors' dtype, or in E4M3 with a scale per token and head), and the
attention of one new token per sequence over such a cache.  ``run`` computes
a case in elementary torch operations, or -- where ``own`` is true -- by the
package's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}
IDS = {"int32": torch.int32, "int64": torch.int64, "fp32": torch.float32}

# The largest listed cases: no drawn case moves more bytes, rows of a cache, or numbers of one
# where every sequence is as long as the longest.
MOST_BYTES = 4 * 32640 * 4096 * 2
MOST_ROWS = 32640 * 8 * 128
MOST_CACHE = 128 * 8192 * 8 * 128


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the angles of one decoding step: a token of each request, far into its text
        dict(name="table_step", op="table", tokens=64, sections="64", positions="int64",
             theta=500000.0, shared=False),
        # the angles of a long video: time, height and width in fractions of a unit
        dict(name="table_video", op="table", tokens=32640, sections="20,22,22", positions="fp32",
             theta=10000.0, shared=False),
        # one decoding step: the heads of 16 tokens, views of the packed projection
        dict(name="rope_step", op="rope", B=1, L=16, Hq=32, Hk=8, D=128, R=64, dtype="bf16",
             norm=True, pairs=False, packed=True, table="rows", offset=0.0),
        # self-attention of a whole long video: every query and key head, adjacent pairs rotated
        dict(name="rope_video", op="rope", B=1, L=32640, Hq=32, Hk=32, D=128, R=64, dtype="bf16",
             norm=True, pairs=True, packed=False, table="rows", offset=0.0),
        # training of a language model: four sequences that share their positions
        dict(name="rope_grad_long", op="rope_grad", B=4, L=2040, Hq=32, Hk=8, D=128, R=64,
             dtype="bf16", norm=True, pairs=False, packed=True, table="shared", offset=0.0),
        # the same of a small module in fp32, a quarter of each head rotated, an odd length
        dict(name="rope_grad_small", op="rope_grad", B=2, L=63, Hq=6, Hk=2, D=80, R=10,
             dtype="fp32", norm=True, pairs=False, packed=False, table="shared", offset=1.0),
        # one decoding step's keys and values into an 8-bit cache
        dict(name="write_step", op="write", T=64, Hk=8, D=128, page=16, dtype="bf16", fp8=True,
             pad=0.0, ids="int64"),
        # a long prompt's
        dict(name="write_prompt", op="write", T=32640, Hk=8, D=128, page=64, dtype="bf16",
             fp8=True, pad=0.05, ids="int64"),
        # an odd number of tokens back from small pages of 8 bits, narrow heads
        dict(name="read_odd", op="read", T=4097, Hk=4, D=80, page=16, dtype="fp16", fp8=True,
             pad=0.0, ids="int32"),
        # a long prompt back, for the attention of what follows it
        dict(name="read_prompt", op="read", T=32640, Hk=8, D=128, page=64, dtype="bf16", fp8=True,
             pad=0.05, ids="int64"),
        # one request with a very long text: its length is all there is to split
        dict(name="attend_long", op="attend", B=1, longest=131072, Hq=32, Hk=8, D=128, page=16,
             dtype="bf16", fp8=False, window=0, ragged=False),
        # many requests of all lengths over an 8-bit cache
        dict(name="attend_batch", op="attend", B=128, longest=8192, Hq=32, Hk=8, D=128, page=64,
             dtype="bf16", fp8=True, window=0, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["table", "rope", "rope", "rope_grad", "write", "read", "attend", "attend",
                     "attend"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "table":
        axes = rng.choice([1, 1, 2, 3])
        # (no more angles than the largest listed case has)
        sections = [rng.randint(4, 64 // axes) for _ in range(axes)]
        return dict(op=op, tokens=_log(rng, 1, 32639), sections=",".join(map(str, sections)),
                    positions=rng.choice(["int32", "int64", "fp32"]),
                    theta=rng.choice([10000.0, 500000.0]), shared=rng.random() < 0.5)
    D = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
    if op in ("rope", "rope_grad"):
        D = rng.choice([D, D, rng.randint(16, 256)])
        Hk = rng.choice([1, 2, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4, 5, 8])
        R = rng.choice([D // 2, D // 2, D // 4, max(1, D // 8)])
        B = rng.choice([1, 1, 2, 3, 8])
        moved = (3 if op == "rope_grad" else 2) * SIZE[dtype] * (Hq + Hk) * D + 8 * R
        most = MOST_BYTES // (B * moved) - 1
        return dict(op=op, B=B, L=min(_log(rng, 1, 32768), most), Hq=Hq, Hk=Hk, D=D, R=R,
                    dtype=dtype, norm=rng.random() < 0.75, pairs=rng.random() < 0.4,
                    packed=rng.random() < 0.5, table=rng.choice(["rows", "shared"]),
                    offset=rng.choice([0.0, 1.0]))
    page = rng.choice([1, 8, 13, 16, 16, 32, 64, 64, 128, 256])
    fp8 = rng.random() < 0.5
    Hk = rng.choice([1, 2, 4, 8, 8])
    if op in ("write", "read"):
        D = rng.choice([D, D, rng.randint(16, 256)])
        most = MOST_ROWS * 2 // (Hk * D * (SIZE[dtype] if dtype == "fp32" else 2)) - 1
        return dict(op=op, T=min(_log(rng, 1, 65536), most), Hk=Hk, D=D, page=page, dtype=dtype,
                    fp8=fp8, pad=rng.choice([0.0, 0.05]), ids=rng.choice(["int32", "int64"]))
    Hq = Hk * rng.choice([1, 2, 4, 4, 5, 8, 16])
    B = _log(rng, 1, 256)
    ragged = rng.random() < 0.6
    # (queries' heads beyond four a key's are more work on the same bytes)
    most = MOST_CACHE // (B * Hk * D * (1 if fp8 else SIZE[dtype]) * max(1, Hq // (4 * Hk))) - 1
    if not ragged:
        kept = D + 4 if fp8 else D * SIZE[dtype]
        most = min(most, (MOST_BYTES - 2 * B * Hq * D * 4) // (B * (2 * Hk * kept + 4)))
    return dict(op=op, B=B, longest=min(_log(rng, 1, 131072), most), Hq=Hq, Hk=Hk,
                D=D, page=page, dtype=dtype, fp8=fp8, window=rng.choice([0, 0, 0, 1000]),
                ragged=ragged)


def _lengths(case):
    """The sequences' lengths, from the case alone: all the longest, or spread over a factor of a
    thousand, one of them the longest and now and then one empty."""
    B, n = case["B"], case["longest"]
    if not case["ragged"]:
        return [n] * B
    r = random.Random(B * 1_000_003 + n)
    lengths = [_log(r, max(1, n // 1000), n) if r.random() < 0.97 else 0 for _ in range(B)]
    lengths[r.randrange(B)] = n
    return lengths


def _sections(case):
    return [int(s) for s in case["sections"].split(",")]


def _freqs(sections, theta, shared):
    """The angle per unit of position of every pair: a spectrum for each axis, or one spectrum that
    the axes share out."""
    R = sum(sections)
    if shared:
        e = [j / R for j in range(R)]
    else:
        e = [j / n for n in sections for j in range(n)]
    return torch.tensor([theta ** -v for v in e], dtype=torch.float64, device="cuda")


def _pages(lengths, page, g):
    """A page table in random order, -1 behind each sequence, and how many pages there are."""
    counts = [-(-n // page) for n in lengths]
    width, total = max(1, max(counts)), max(1, sum(counts))
    order = torch.randperm(total, generator=g, device="cuda").int()
    count = torch.tensor(counts, device="cuda")
    used = torch.arange(width, device="cuda")[None, :] < count[:, None]
    table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
    table[used] = order[:sum(counts)]
    return table, total


def _slots(T, page, pad, g, t):
    """A place in the cache for every token, consecutive ones within a page and the pages in random
    order, and -1 in the padded places at the end; and how many pages there are."""
    pages = -(-T // page) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    i = torch.arange(T, device="cuda")
    slots = order[i // page] * page + i % page
    pads = int(T * pad)
    if pads:
        slots[T - pads:] = -1
    return slots.to(t), pages


def _quantise(x):
    """E4M3 codes and a scale per row."""
    scale = x.abs().amax(-1, keepdim=True) / E4M3_MAX
    codes = torch.where(scale > 0, x / scale, 0.0).to(torch.float8_e4m3fn)
    return codes, scale[..., 0]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)

    def normal(*shape, std=1.0, mean=0.0, t=None):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(t or TYPES[case["dtype"]])

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda", dtype=torch.float64)

    def cache(pages, heads, page, D, filled):
        """Keys and values of a paged cache [pages, heads, page, D] and, in 8 bits, their scales."""
        t = torch.float8_e4m3fn if case["fp8"] else TYPES[case["dtype"]]
        for name, std in (("k", 1.0), ("v", 0.7)):
            c = torch.zeros((pages, heads, page, D), dtype=t, device="cuda")
            sc = torch.zeros((pages, heads, page), device="cuda") if case["fp8"] else None
            step = max(1, (1 << 26) // (heads * page * D))
            for a in range(0, pages if filled else 0, step):
                x = torch.randn((min(step, pages - a), heads, page, D), generator=g, device="cuda")
                # the rows of a head differ in size
                x *= std * torch.exp(0.5 * torch.randn(x.shape[:-1], generator=g,
                                                       device="cuda"))[..., None]
                if case["fp8"]:
                    c[a:a + step], sc[a:a + step] = _quantise(x)
                else:
                    c[a:a + step] = x
            s[name + "_cache"], s[name + "_scales"] = c, sc
        if own:  # the description of its cache that a serving program keeps
            import diffusion_transformer_elementwise_gb300 as dit
            s["cache"] = dit.KVCache(s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"])

    if case["op"] == "table":
        sections = _sections(case)
        A, T = len(sections), case["tokens"]
        if case["positions"] == "fp32":
            # places on a grid, in a unit of which a step is a fraction
            s["positions"] = (uniform(A, T) * 4096).floor().mul(0.04).float()
        else:
            s["positions"] = (uniform(A, T) * 131072).to(IDS[case["positions"]])
        s["freqs"] = _freqs(sections, case["theta"], case["shared"])
        s["sections"] = sections
        s["cos"] = torch.empty((T, sum(sections)), device="cuda")
        s["sin"] = torch.empty_like(s["cos"])
    elif case["op"] in ("rope", "rope_grad"):
        B, L, Hq, Hk, D, R = (case[k] for k in ("B", "L", "Hq", "Hk", "D", "R"))
        lead = (L,) if B == 1 else (B, L)

        def heads():
            if not case["packed"]:
                return normal(*lead, Hq, D), normal(*lead, Hk, D)
            qkv = normal(*lead, Hq + 2 * Hk, D)
            return qkv[..., :Hq, :], qkv[..., Hq:Hq + Hk, :]

        s["q"], s["k"] = heads()
        n = L if case["table"] == "shared" else B * L
        angles = (uniform(n, 1) * 32768).floor() * _freqs([R], 10000.0, False)
        s["cos"], s["sin"] = torch.cos(angles).float(), torch.sin(angles).float()
        if case["norm"]:
            s["wq"] = normal(D, std=0.1, mean=1.0 - case["offset"])
            s["wk"] = normal(D, std=0.1, mean=1.0 - case["offset"])
        s["out_q"], s["out_k"] = (torch.empty(s[n].shape, dtype=s[n].dtype, device="cuda")
                                  for n in "qk")
        if case["op"] == "rope_grad":
            s["gq"], s["gk"] = (normal(*s[n].shape, std=0.1) for n in "qk")
            if case["norm"]:
                s["gwq"], s["gwk"] = torch.empty_like(s["wq"]), torch.empty_like(s["wk"])
    elif case["op"] in ("write", "read"):
        T, Hk, D = case["T"], case["Hk"], case["D"]
        s["slots"], pages = _slots(T, case["page"], case["pad"], g, IDS[case["ids"]])
        cache(pages, Hk, case["page"], D, case["op"] == "read")
        if case["op"] == "write":
            # keys as the rotation left them, values as a view of the packed projection
            size = torch.exp(0.5 * torch.randn((T, Hk, 1), generator=g, device="cuda"))
            s["k"] = (normal(T, Hk, D).float() * size).to(TYPES[case["dtype"]])
            s["v"] = normal(T, 3 * Hk, D, std=0.7)[:, 2 * Hk:]
        else:
            s["k"], s["v"] = (torch.empty((T, Hk, D), dtype=TYPES[case["dtype"]], device="cuda")
                              for _ in "kv")
    else:
        lengths = _lengths(case)
        s["pages"], total = _pages(lengths, case["page"], g)
        cache(total, case["Hk"], case["page"], case["D"], True)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        s["q"] = normal(case["B"], case["Hq"], case["D"], std=1.5)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty((case["B"], case["Hq"]), device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import diffusion_transformer_elementwise_gb300 as dit
    c = s["case"]
    if c["op"] == "table":
        return dit.rotary_table(s["positions"], s["freqs"], s["sections"], cos=s["cos"],
                                sin=s["sin"])
    if c["op"] == "rope":
        kw = dict(interleaved=c["pairs"], out_q=s["out_q"], out_k=s["out_k"])
        if not c["norm"]:
            return dit.rope(s["q"], s["k"], s["cos"], s["sin"], **kw)
        return dit.rmsnorm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], EPS,
                                weight_offset=c["offset"], **kw)
    if c["op"] == "rope_grad":
        if not c["norm"]:
            return dit.rope(s["gq"], s["gk"], s["cos"], s["sin"], interleaved=c["pairs"],
                            inverse=True, out_q=s["out_q"], out_k=s["out_k"])
        return dit.rmsnorm_rope_backward(
            s["gq"], s["gk"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"], EPS,
            weight_offset=c["offset"], interleaved=c["pairs"], grad_q=s["out_q"],
            grad_k=s["out_k"], grad_weight_q=s["gwq"], grad_weight_k=s["gwk"])
    if c["op"] == "write":
        dit.cache_write(s["cache"], s["k"], s["v"], s["slots"])
        return [s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]
    if c["op"] == "read":
        return dit.cache_read(s["cache"], s["slots"], k=s["k"], v=s["v"])
    return dit.paged_attention(s["q"], s["cache"], s["pages"], s["lengths"], window=c["window"],
                               out=s["out"], lse=s["lse"])


def _rotate(x, cos, sin, c, inverse=False):
    """x [..., H, D] in 32 bits, cos and sin [..., 1, R]."""
    R = c["R"]
    if inverse:
        sin = -sin
    if c["pairs"]:
        a, b = x[..., 0:2 * R:2], x[..., 1:2 * R:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :R], x[..., R:2 * R]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * R:]), -1)


def _plain(s):
    c = s["case"]
    if c["op"] == "table":
        at = torch.cat([s["positions"][a].double()[:, None].expand(-1, n)
                        for a, n in enumerate(s["sections"])], 1)
        angles = at * s["freqs"]
        return angles.cos().float(), angles.sin().float()
    if c["op"] in ("rope", "rope_grad"):
        shape = s["q"].shape[:-2] if c["table"] == "rows" else (c["L"],)
        cos, sin = (s[n].view(*shape, 1, c["R"]) for n in ("cos", "sin"))
        if c["op"] == "rope":
            return [_plain_rope(s[n], s.get("w" + n), cos, sin, c) for n in "qk"]
        got = [_plain_rope_grad(s["g" + n], s[n], s.get("w" + n), cos, sin, c) for n in "qk"]
        return [p for p, _ in got] + [w for _, w in got if w is not None]
    if c["op"] == "write":
        at = torch.nonzero(s["slots"] >= 0)[:, 0]
        page, place = s["slots"][at] // c["page"], s["slots"][at] % c["page"]
        for n in "kv":
            x = s[n][at]
            if c["fp8"]:
                codes, scales = _quantise(x.float())
                s[n + "_scales"][page, :, place] = scales
                s[n + "_cache"].view(torch.uint8)[page, :, place] = codes.view(torch.uint8)
            else:
                s[n + "_cache"][page, :, place] = x
        return [s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]]
    if c["op"] == "read":
        seen = s["slots"] >= 0
        at = s["slots"].long().clamp(min=0)
        return [torch.where(seen[:, None, None], _rows(s, n, at), 0.0).to(TYPES[c["dtype"]])
                for n in "kv"]
    return _plain_attend(s, c)


def _plain_rope(x, w, cos, sin, c):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * (w.float() + c["offset"])
    return _rotate(y, cos, sin, c).to(x.dtype)


def _plain_rope_grad(g, x, w, cos, sin, c):
    u = _rotate(g.float(), cos, sin, c, inverse=True)
    if w is None:
        return u.to(g.dtype), None
    y = x.float()
    r = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    n = y * r
    t = u * (w.float() + c["offset"])
    gx = r * (t - n * (t * n).mean(-1, keepdim=True))
    return gx.to(x.dtype), (u * n).flatten(0, -2).sum(0).to(w.dtype)


def _rows(s, n, at):
    """The cache's rows of the places `at` in 32 bits: at.shape + [Hk, D]."""
    page = s["case"]["page"]
    x = s[n + "_cache"][at // page, :, at % page].float()
    if s[n + "_scales"] is not None:
        x = x * s[n + "_scales"][at // page, :, at % page][..., None]
    return x


def _plain_attend(s, c):
    B, Hq, Hk, D, page = (c[k] for k in ("B", "Hq", "Hk", "D", "page"))
    t = torch.arange(s["pages"].shape[1] * page, device="cuda")[:max(1, c["longest"])]
    at = s["pages"].long()[:, t // page].clamp(min=0) * page + t % page
    k, v = (_rows(s, n, at).transpose(1, 2) for n in "kv")  # [B, Hk, tokens, D]
    q = s["q"].float().view(B, Hk, Hq // Hk, D) * D ** -0.5
    logits = q @ k.transpose(2, 3)
    length = s["lengths"][:, None]
    seen = t[None, :] < length
    if c["window"]:
        seen &= t[None, :] >= length - c["window"]
    logits = logits.masked_fill(~seen[:, None, None, :], -math.inf)
    m = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(m > -math.inf, m, 0.0))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + m).view(B, Hq)
    return out.view(B, Hq, D).to(s["q"].dtype), lse


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "table":
        sections, T = _sections(case), case["tokens"]
        p = 8 if case["positions"] == "int64" else 4
        return dict(bytes=T * (len(sections) * p + 8 * sum(sections)) + 8 * sum(sections),
                    flops=20 * T * sum(sections))
    e = SIZE[case["dtype"]]
    if op in ("rope", "rope_grad"):
        n = case["B"] * case["L"] * (case["Hq"] + case["Hk"]) * case["D"]
        rows = case["L"] * (case["B"] if case["table"] == "rows" else 1)
        weights = 2 * case["D"] * e if case["norm"] else 0
        table = rows * case["R"] * 8
        if op == "rope":
            return dict(bytes=2 * n * e + table + weights, flops=8 * n)
        return dict(bytes=(3 if case["norm"] else 2) * n * e + table + 2 * weights, flops=16 * n)
    kept = (case["D"] + 4) if case["fp8"] else case["D"] * e
    if op in ("write", "read"):
        T = case["T"] - int(case["T"] * case["pad"])  # padded places: ids, and zeros where read
        rows = 2 * T * case["Hk"]
        ids = case["T"] * (8 if case["ids"] == "int64" else 4)
        zeros = 2 * (case["T"] - T) * case["Hk"] * case["D"] * e if op == "read" else 0
        return dict(bytes=rows * (kept + case["D"] * e) + ids + zeros, flops=4 * rows * case["D"])
    lengths = _lengths(case)
    if case["window"]:
        lengths = [min(n, case["window"]) for n in lengths]
    tokens = sum(lengths)
    table = 4 * sum(-(-n // case["page"]) for n in lengths)
    return dict(bytes=2 * tokens * case["Hk"] * kept + table
                + case["B"] * case["Hq"] * (2 * case["D"] * e + 4),
                flops=4 * tokens * case["Hq"] * case["D"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def e4m3(x):
        """E4M3 values (3 fraction bits, smallest step 2^-9, at most 448; ties to even) of the rows
        over their scales, and the scales."""
        scale = x.abs().max(dim=-1, keepdim=True).values / 448.0
        v = torch.where(scale > 0, x / scale, torch.zeros_like(x))
        _, e = torch.frexp(v)
        step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
        return torch.clamp(torch.round(v / step) * step, -448.0, 448.0), scale.squeeze(-1)

    if op == "table":
        # in turns: the whole ones do not count
        column = 0
        cos, sin = [], []
        for a, n in enumerate(s["sections"]):
            turns = torch.outer(s["positions"][a].double(), s["freqs"][column:column + n] / (2 * math.pi))
            rest = 2 * math.pi * (turns - torch.round(turns))
            cos.append(torch.cos(rest))
            sin.append(torch.sin(rest))
            column += n
        return [torch.cat(cos, dim=1), torch.cat(sin, dim=1)]
    if op in ("rope", "rope_grad"):
        R, D = case["R"], case["D"]
        if case["pairs"]:
            first = torch.arange(0, 2 * R, 2, device="cuda")
            second = first + 1
        else:
            first = torch.arange(R, device="cuda")
            second = first + R
        turn = torch.complex(s["cos"].double(), s["sin"].double())
        turn = turn.reshape((case["L"], 1, R) if case["table"] == "shared" or case["B"] == 1
                            else (case["B"], case["L"], 1, R))

        def turned(x, by):
            z = torch.complex(x[..., first], x[..., second]) * by
            y = x.clone()
            y[..., first], y[..., second] = z.real, z.imag
            return y

        outs, weights = [], []
        for n in "qk":
            x = s[n].double()
            if not case["norm"]:
                outs.append(turned(x, turn) if op == "rope" else turned(s["g" + n].double(), turn.conj()))
                continue
            w = s["w" + n].double() + case["offset"]
            inv = (torch.mean(x ** 2, dim=-1, keepdim=True) + EPS) ** -0.5
            if op == "rope":
                outs.append(turned(x * inv * w, turn))
                continue
            u = turned(s["g" + n].double(), turn.conj())
            # d/dx of sum(u w x / rms(x)), by the quotient rule
            dot = torch.sum(u * w * x, dim=-1, keepdim=True)
            outs.append(u * w * inv - x * (dot * inv ** 3 / D))
            weights.append(torch.sum((u * x * inv).reshape(-1, D), dim=0))
        return outs + weights
    page = case["page"]
    if op == "write":
        got = {n: s[n].double() for n in ("k_cache", "v_cache")}
        sc = {n: (s[n].double() if case["fp8"] else None) for n in ("k_scales", "v_scales")}
        at = torch.nonzero(s["slots"] >= 0).flatten()
        where = s["slots"][at].long()
        for n in "kv":
            x = s[n][at].double()
            flat = got[n + "_cache"].transpose(1, 2).reshape(-1, case["Hk"], case["D"])
            if case["fp8"]:
                x, scale = e4m3(x)
                fs = sc[n + "_scales"].transpose(1, 2).reshape(-1, case["Hk"])
                fs[where] = scale
                sc[n + "_scales"] = fs.reshape(-1, page, case["Hk"]).transpose(1, 2).contiguous()
            flat[where] = x
            got[n + "_cache"] = flat.reshape(-1, page, case["Hk"], case["D"]).transpose(1, 2).contiguous()
        return [got["k_cache"], got["v_cache"], sc["k_scales"], sc["v_scales"]]

    def place(n, where):
        """The rows of the places `where` (flat numbers of page and place), in 64 bits."""
        x = s[n + "_cache"][torch.div(where, page, rounding_mode="floor"), :, where % page].double()
        if case["fp8"]:
            x *= s[n + "_scales"][torch.div(where, page, rounding_mode="floor"), :, where % page].double()[..., None]
        return x

    if op == "read":
        outs = []
        for n in "kv":
            x = torch.zeros((case["T"], case["Hk"], case["D"]), dtype=torch.float64, device="cuda")
            at = torch.nonzero(s["slots"] >= 0).flatten()
            x[at] = place(n, s["slots"][at].long())
            outs.append(x)
        return outs
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full((case["B"], case["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    group = case["Hq"] // case["Hk"]
    for b, n in enumerate(_lengths(case)):
        start = max(0, n - case["window"]) if case["window"] else 0
        if n == start:
            continue
        t = torch.arange(start, n, device="cuda")
        where = s["pages"][b].long()[torch.div(t, page, rounding_mode="floor")] * page + t % page
        k, v = place("k", where), place("v", where)
        q = s["q"][b].double().reshape(case["Hk"], group, case["D"])
        logits = torch.einsum("hgd,thd->hgt", q, k) / math.sqrt(case["D"])
        lse[b] = torch.logsumexp(logits, dim=-1).reshape(-1)
        out[b] = torch.einsum("hgt,thd->hgd", torch.softmax(logits, dim=-1), v).reshape(case["Hq"], -1)
    return [out, lse]
