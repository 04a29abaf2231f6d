"""Performance cases of the token-transformer operators.

One case is one call of one operator at one size: the weighted RMSNorm with the
residual's addition (output in the tensors' dtype, or in E4M3 with dynamic
scales), its gradient, the embedding lookup and its gradient, and the clipping
of gradients by their global norm.  ``run`` computes a case in elementary torch
operations, or -- where ``own`` is true -- by the package's calls.
"""
import math
import random

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4}

# The largest listed case's bytes: no drawn case moves more.
MOST_BYTES = 4 * 32640 * 4096 * 2


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one token of one request: the call's latency
        dict(name="norm_token", op="norm", rows=1, D=4096, dtype="bf16", add=True, fp8=False,
             group=0, offset=0.0),
        # a whole long sequence at the widest model size: bandwidth
        dict(name="norm_long", op="norm", rows=32640, D=4096, dtype="bf16", add=True, fp8=False,
             group=0, offset=0.0),
        # a batch of single tokens whose normed rows feed an 8-bit product
        dict(name="norm_fp8_batch", op="norm", rows=126, D=2048, dtype="bf16", add=True, fp8=True,
             group=0, offset=1.0),
        # a prompt of odd length and width, one scale per 128 columns (the last group is ragged)
        dict(name="norm_fp8_groups_odd", op="norm", rows=4097, D=3077, dtype="fp16", add=False,
             fp8=True, group=128, offset=0.0),
        # training: the gradient through a norm whose input also feeds the skip path
        dict(name="norm_grad_long", op="norm_grad", rows=8160, D=4096, dtype="bf16", skip=True,
             offset=0.0),
        # the same of a small micro-batch in fp32, a norm without skip path
        dict(name="norm_grad_small", op="norm_grad", rows=126, D=2048, dtype="fp32", skip=False,
             offset=1.0),
        # the first operation of one decoding step for a few requests
        dict(name="embed_batch", op="embed", tokens=16, V=32000, D=2048, dtype="bf16", pad=0.0,
             scale=1.0),
        # the first operation of a long padded batch, scaled by sqrt(D)
        dict(name="embed_long", op="embed", tokens=32640, V=128000, D=4096, dtype="bf16", pad=0.05,
             scale=64.0),
        # its gradient: few tokens, so nearly all of the table's gradient is zero
        dict(name="embed_grad_small", op="embed_grad", tokens=126, V=32000, D=2048, dtype="fp32",
             pad=0.0, scale=1.0),
        # and for a long batch with the token frequencies of text
        dict(name="embed_grad_long", op="embed_grad", tokens=32640, V=128000, D=2048, dtype="bf16",
             pad=0.05, scale=math.sqrt(2048.0)),
        # the gradients of one small module, many of them vectors
        dict(name="clip_small", op="clip", tensors=60, elements=2_000_003, dtype="fp32"),
        # the gradients of a model's shard
        dict(name="clip_large", op="clip", tensors=291, elements=400_000_000, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """64 to 8192: multiples of 128, of 8, or any."""
    d = _log(rng, 64, 8192)
    step = rng.choice([128, 128, 8, 1])
    return min(8192, max(64, (d + step // 2) // step * step))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "embed", "embed_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    e = SIZE[dtype]
    if op == "clip":
        n = _log(rng, 1, 600)
        most = MOST_BYTES // (2 * e) - 64 * n
        return dict(op=op, tensors=n, elements=max(n, _log(rng, 1000, most)), dtype=dtype)
    D = _width(rng)
    if op in ("norm", "norm_grad"):
        rows = min(_log(rng, 1, 32768), MOST_BYTES // (4 * D * e) - 1)
        offset = rng.choice([0.0, 1.0])
        if op == "norm_grad":
            return dict(op=op, rows=rows, D=D, dtype=dtype, skip=rng.random() < 0.5, offset=offset)
        fp8 = rng.random() < 0.5
        return dict(op=op, rows=rows, D=D, dtype=dtype, add=rng.random() < 0.5, fp8=fp8,
                    group=rng.choice([0, 128]) if fp8 else 0, offset=offset)
    tokens = min(_log(rng, 1, 65536), MOST_BYTES // (4 * D * e) - 1)
    V = min(_log(rng, 1000, 256000), MOST_BYTES // (2 * D * e))
    return dict(op=op, tokens=tokens, V=V, D=D, dtype=dtype, pad=rng.choice([0.0, 0.05]),
                scale=rng.choice([1.0, math.sqrt(D)]))


def _sizes(case):
    """The tensors' sizes: a third of them vectors, the rest sharing what is left."""
    n, left = case["tensors"], case["elements"]
    r = random.Random(n * 1_000_003 + left)
    small = [r.randint(1, max(1, min(8192, left // (2 * n)))) for _ in range(n // 3)]
    left -= sum(small)
    share = [r.uniform(0.2, 1.0) for _ in range(n - len(small))]
    big = [max(1, int(left * s / sum(share))) for s in share]
    sizes = small + big
    r.shuffle(sizes)
    return sizes


def _ids(case, g):
    """Token ids with the frequencies of text (about 1 / rank), ranks spread over the table, and
    -1 in the padded places at the end."""
    T, V = case["tokens"], case["V"]
    u = torch.rand(T, generator=g, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(V)) - 1.0).long().clamp_(0, V - 1)
    ids = (rank * 7919) % V
    pads = int(T * case["pad"])
    if pads:
        ids[T - pads:] = -1
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, mean=0.0):
        x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
        return x.mul_(std).add_(mean).to(t)

    s = dict(case=case)
    if case["op"] in ("norm", "norm_grad"):
        rows, D = case["rows"], case["D"]
        s["weight"] = normal(D, std=0.1, mean=1.0 - case["offset"])
        # rows of a residual stream differ in size
        size = torch.exp(torch.randn((rows, 1), generator=g, device="cuda"))
        s["x"] = (normal(rows, D).float() * size).to(t)
        if case["op"] == "norm":
            if case["add"]:
                s["update"] = normal(rows, D, std=0.5)
                s["residual"] = torch.empty_like(s["x"])
            if case["fp8"]:
                s["out"] = torch.empty((rows, D), dtype=torch.float8_e4m3fn, device="cuda")
                n = -(-D // case["group"]) if case["group"] else 1
                s["scales"] = torch.empty((rows, n), dtype=torch.float32, device="cuda")
                pads = rows // 16  # a padded batch's empty rows
                if pads:
                    s["x"][rows - pads:] = 0
                    if case["add"]:
                        s["update"][rows - pads:] = 0
            else:
                s["out"] = torch.empty_like(s["x"])
        else:
            s["grad"] = normal(rows, D, std=0.1)
            s["skip"] = normal(rows, D, std=0.1) if case["skip"] else None
            s["grad_x"] = torch.empty_like(s["x"])
            s["grad_weight"] = torch.empty_like(s["weight"])
    elif case["op"] in ("embed", "embed_grad"):
        s["ids"] = _ids(case, g)
        if case["op"] == "embed":
            s["table"] = normal(case["V"], case["D"], std=0.02)
            s["out"] = torch.empty((case["tokens"], case["D"]), dtype=t, device="cuda")
        else:
            s["grad"] = normal(case["tokens"], case["D"], std=0.1)
            s["grad_table"] = torch.empty((case["V"], case["D"]), dtype=t, device="cuda")
    else:
        # each tensor at a multiple of 64 elements of one allocation, zeros between them
        sizes = _sizes(case)
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += -(-n // 64) * 64
        flat = torch.zeros(at, dtype=t, device="cuda")
        out = torch.zeros_like(flat)
        for k, (a, n) in enumerate(zip(starts, sizes)):
            # gradients of different tensors differ in size; in pieces, to hold little at once
            std = 1e-3 * 10.0 ** ((k * 7 % 10) / 5.0 - 1.0)
            for b in range(a, a + n, 1 << 26):
                m = min(1 << 26, a + n - b)
                flat[b:b + m] = torch.randn(m, generator=g, device="cuda").mul_(std)
        s["flat"], s["flat_out"] = flat, out
        s["grads"] = [flat[a:a + n] for a, n in zip(starts, sizes)]
        s["outs"] = [out[a:a + n] for a, n in zip(starts, sizes)]
        s["max_norm"] = 1.0
        if own:  # the description of its gradients that a training program keeps beside them
            import diffusion_transformer_elementwise_gb300 as dit
            s["list"] = dit.TensorList(s["grads"], out=s["outs"])
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import diffusion_transformer_elementwise_gb300 as dit
    c = s["case"]
    if c["op"] == "norm":
        kw = dict(weight_offset=c["offset"], out=s["out"])
        if c["fp8"]:
            kw.update(group=c["group"], scales=s["scales"])
            if c["add"]:
                return dit.add_rmsnorm_fp8(s["x"], s["update"], s["weight"], EPS,
                                           residual_out=s["residual"], **kw)
            return dit.rmsnorm_fp8(s["x"], s["weight"], EPS, **kw)
        if c["add"]:
            return dit.add_rmsnorm(s["x"], s["update"], s["weight"], EPS,
                                   residual_out=s["residual"], **kw)
        return [dit.rmsnorm(s["x"], s["weight"], EPS, **kw)]
    if c["op"] == "norm_grad":
        return dit.rmsnorm_backward(s["grad"], s["x"], s["weight"], EPS,
                                    weight_offset=c["offset"], grad_residual=s["skip"],
                                    grad_x=s["grad_x"], grad_weight=s["grad_weight"])
    if c["op"] == "embed":
        return [dit.embedding(s["ids"], s["table"], c["scale"], out=s["out"])]
    if c["op"] == "embed_grad":
        return [dit.embedding_backward(s["grad"], s["ids"], c["V"], c["scale"],
                                       out=s["grad_table"])]
    _, norm = dit.clip_grads(s["list"], s["max_norm"])
    return [s["flat_out"], norm]


def _plain(s):
    c = s["case"]
    if c["op"] == "norm":
        return _plain_norm(s, c)
    if c["op"] == "norm_grad":
        x, g = s["x"].float(), s["grad"].float()
        r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        n = x * r
        t = g * (s["weight"].float() + c["offset"])
        gx = r * (t - n * (t * n).mean(1, keepdim=True))
        if s["skip"] is not None:
            gx = gx + s["skip"].float()
        return gx.to(s["x"].dtype), (g * n).sum(0).to(s["x"].dtype)
    if c["op"] == "embed":
        ids = s["ids"]
        rows = s["table"][ids.clamp(0, c["V"] - 1)].float() * c["scale"]
        seen = ((ids >= 0) & (ids < c["V"]))[:, None]
        return [torch.where(seen, rows, 0.0).to(s["table"].dtype)]
    if c["op"] == "embed_grad":
        ids = s["ids"]
        seen = ((ids >= 0) & (ids < c["V"]))[:, None]
        g = torch.where(seen, s["grad"].float() * c["scale"], 0.0)
        t = torch.zeros((c["V"], c["D"]), dtype=torch.float32, device="cuda")
        t.index_put_((ids.clamp(0, c["V"] - 1),), g, accumulate=True)
        return [t.to(s["grad"].dtype)]
    x = s["flat"].float()
    norm = (x * x).sum(dtype=torch.float64).sqrt()
    scale = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    return [(x * scale).to(s["flat"].dtype), norm.float()]


def _plain_norm(s, c):
    x = s["x"].float()
    outs = []
    if c["add"]:
        res = (x + s["update"].float()).to(s["x"].dtype)
        outs.append(res)
        x = res.float()
    r = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
    y = x * r * (s["weight"].float() + c["offset"])
    if not c["fp8"]:
        return outs + [y.to(s["x"].dtype)]
    g = c["group"] or c["D"]
    n = -(-c["D"] // g)
    y = torch.nn.functional.pad(y, (0, n * g - c["D"])).view(c["rows"], n, g)
    scales = y.abs().amax(2, keepdim=True) / E4M3_MAX
    q = torch.where(scales > 0, y / scales, 0.0).to(torch.float8_e4m3fn)
    q = q.view(c["rows"], n * g)[:, :c["D"]].contiguous()
    return outs + [q, scales.view(c["rows"], n)]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and its values in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "norm":
        n, D = case["rows"] * case["D"], case["D"]
        b = n * e * (3 if case["add"] else 1) + D * e
        if case["fp8"]:
            b += n + 4 * case["rows"] * (-(-D // case["group"]) if case["group"] else 1)
        else:
            b += n * e
        return dict(bytes=b, flops=5 * n)
    if op == "norm_grad":
        n = case["rows"] * case["D"]
        return dict(bytes=n * e * (4 if case["skip"] else 3) + 2 * case["D"] * e, flops=12 * n)
    if op == "embed":
        # the table's rows that a batch names, at most one a token, and ids of 8 bytes
        read = min(case["tokens"], case["V"]) * case["D"] * e
        return dict(bytes=read + case["tokens"] * (case["D"] * e + 8), flops=case["tokens"] * case["D"])
    if op == "embed_grad":
        n = case["tokens"] * case["D"]
        return dict(bytes=n * e + case["V"] * case["D"] * e + case["tokens"] * 8, flops=2 * n)
    n = sum(_sizes(case))
    return dict(bytes=2 * n * e, flops=3 * n)


def exact(case, seed):
    def codes_of(y, group):
        """E4M3 values (3 fraction bits, smallest step 2^-9, at most 448; ties to even) of y over its
        group's scale, and the scales."""
        rows, D = y.shape
        values = torch.zeros_like(y)
        scales = []
        for a in range(0, D, group):
            part = y[:, a:a + group]
            scale = part.abs().max(dim=1, keepdim=True).values / 448.0
            v = torch.where(scale > 0, part / scale, torch.zeros_like(part))
            _, e = torch.frexp(v)
            step = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
            values[:, a:a + group] = torch.clamp(torch.round(v / step) * step, -448.0, 448.0)
            scales.append(scale)
        return [values, torch.cat(scales, dim=1)]

    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        w = s["weight"].double() + case["offset"]
        x = s["x"].double()
        first = []
        if op == "norm" and case["add"]:
            # the sum is rounded to the tensors' type before the norm reads it: a sum of two of
            # its values is exact in 64 bits up to a double rounding that fp32 does not show
            kept = (x + s["update"].double()).to(s["x"].dtype)
            first, x = [x + s["update"].double()], kept.double()
        inv = 1.0 / torch.sqrt(torch.mean(x ** 2, dim=-1, keepdim=True) + EPS)
        if op == "norm":
            y = x * inv * w
            if not case["fp8"]:
                return first + [y]
            return first + codes_of(y, case["group"] or case["D"])
        g = s["grad"].double()
        # d/dx of sum(g w x / rms(x)), by the quotient rule
        gw = g * w
        dot = torch.sum(gw * x, dim=-1, keepdim=True)
        gx = gw * inv - x * (dot * inv ** 3 / case["D"])
        if s["skip"] is not None:
            gx = gx + s["skip"].double()
        return [gx, torch.sum(g * x * inv, dim=0)]
    if op == "embed":
        out = torch.zeros((case["tokens"], case["D"]), dtype=torch.float64, device="cuda")
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["V"]))[:, 0]
        out[at] = s["table"][s["ids"][at]].double() * case["scale"]
        return [out]
    if op == "embed_grad":
        out = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device="cuda")
        at = torch.nonzero((s["ids"] >= 0) & (s["ids"] < case["V"]))[:, 0]
        out.index_add_(0, s["ids"][at], s["grad"][at].double())
        return [out * case["scale"]]
    total = 0.0
    for g in s["grads"]:
        for b in range(0, g.numel(), 1 << 26):
            total += float(torch.sum(g[b:b + (1 << 26)].double() ** 2))
    norm = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    return [s["flat"].double() * c, torch.tensor(norm, dtype=torch.float64)]
