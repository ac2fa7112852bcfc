"""The operators around the products of a decode step, as cases that can be timed: from a token's id to its row, to
attention's queries and keys, through a layer of experts, and from the logits to the next id.

    embed    rows of a block-quantized token table, scaled, as float32 or bfloat16
    rope     norms of queries and keys for each head, and the position rotation
    moe      a layer of experts with block-quantized weights, from the router's logits
    sample   the next ids under temperature, top-k, top-p and min-p, from given exponential random numbers

`own` false: the plain form, elementary torch operations in float32 (float64 for the angles and for what decides
an id), rounded once at the end.  `own` true: the calls of this repository's package.  Head counts, head sizes,
hidden sizes and vocabularies are those of the repository's benchmark layers (32 heads of 128 with 8 key/value heads
over 4096 columns, 1024 and 11008 columns, a vocabulary of 151936); 32 experts with 4 used over 1024 columns is the
layer of the prefill figure that the repository quotes; the rest is generic.
"""
import math

import torch

own = False


def listed():
    return [
        # the row of one sampled token, from a table that is also the classifier (Q8_0): the smallest call there is
        {"name": "embed_1x1024_q8", "op": "embed", "rows": 1, "vocab": 151936, "cols": 1024, "wt": 1, "f16": 0, "out": "f32"},
        # a prompt chunk's rows from a Q4_0 table
        {"name": "embed_4096x4096_q4", "op": "embed", "rows": 4096, "vocab": 32000, "cols": 4096, "wt": 2, "f16": 1, "out": "bf16"},
        # one sequence's next token: float32, as the products leave q and k; bfloat16 for attention
        {"name": "rope_1x32x128", "op": "rope", "rows": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "x": "f32", "out": "bf16",
         "norm": False, "pairs": "neighbours", "far": 30000},
        # a serving batch's tokens at far positions, with norms of queries and keys
        {"name": "rope_256x32x128", "op": "rope", "rows": 256, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128, "x": "f32", "out": "f32",
         "norm": True, "pairs": "halves", "far": 1000000},
        # a prompt's rows, norms and a rotation of half of each head
        {"name": "rope_8192x32x128", "op": "rope", "rows": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 64, "x": "bf16",
         "out": "bf16", "norm": True, "pairs": "halves", "far": 200000},
        # one token through many small experts: latency
        {"name": "moe_1_of_32x512x1024", "op": "moe", "tokens": 1, "experts": 32, "used": 4, "dim": 1024, "hidden": 512, "wt": 2, "f16": 1,
         "x": "bf16", "out": "f32", "act": "silu", "renorm": True},
        # one token through two of eight large experts: the weights' bytes
        {"name": "moe_1_of_8x11008x4096", "op": "moe", "tokens": 1, "experts": 8, "used": 2, "dim": 4096, "hidden": 11008, "wt": 2, "f16": 1,
         "x": "bf16", "out": "bf16", "act": "silu", "renorm": True},
        # a serving batch: every expert is used, by a few tokens each
        {"name": "moe_32_of_128x768x2048", "op": "moe", "tokens": 32, "experts": 128, "used": 8, "dim": 2048, "hidden": 768, "wt": 2, "f16": 1,
         "x": "bf16", "out": "bf16", "act": "silu", "renorm": True},
        # Q8_0 experts, float32 activations
        {"name": "moe_7_of_16x1408x2048_q8", "op": "moe", "tokens": 7, "experts": 16, "used": 3, "dim": 2048, "hidden": 1408, "wt": 1, "f16": 0,
         "x": "f32", "out": "f32", "act": "gelu", "renorm": False},
        # one conversation's next token
        {"name": "sample_1x151936", "op": "sample", "rows": 1, "vocab": 151936, "kind": "all", "peaks": 60},
        # a serving batch, each row with settings of its own
        {"name": "sample_64x151936_mixed", "op": "sample", "rows": 64, "vocab": 151936, "kind": "mixed", "peaks": 60},
        # many rollouts of one prompt at temperature 1, nothing cut off: every random number is read
        {"name": "sample_512x151936_free", "op": "sample", "rows": 512, "vocab": 151936, "kind": "free", "peaks": 60},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed", "rope", "moe", "moe", "sample", "sample"])
    kind = rng.choice([(1, 0), (1, 1), (2, 0), (2, 1), (2, 1)])
    if op == "embed":
        return {"op": op, "rows": log(1, 4096), "vocab": log(1000, 151936), "cols": 32 * log(8, 128), "wt": kind[0], "f16": kind[1],
                "out": rng.choice(["f32", "bf16"])}
    if op == "rope":
        heads = rng.choice([(32, 8), (32, 8), (16, 16), (14, 2), (8, 1), (5, 5)])
        dim = rng.choice([64, 128, 128, 256])
        return {"op": op, "rows": log(1, 4000), "heads": heads[0], "kv_heads": heads[1], "dim": dim, "rot": rng.choice([dim, dim, dim // 2]),
                "x": rng.choice(["f32", "bf16"]), "out": rng.choice(["f32", "bf16"]), "norm": rng.random() < 0.6,
                "pairs": rng.choice(["halves", "neighbours"]), "far": log(100, 1000000)}
    if op == "moe":
        experts = log(4, 128)
        case = {"op": op, "tokens": log(1, 48), "experts": experts, "used": rng.randint(1, min(8, experts)), "dim": 64 * log(4, 48),
                "hidden": 64 * log(3, 32), "wt": kind[0], "f16": kind[1], "x": rng.choice(["bf16", "bf16", "f32"]),
                "out": rng.choice(["f32", "bf16"]), "act": rng.choice(["silu", "silu", "gelu"]), "renorm": rng.random() < 0.6}
        return case
    return {"op": op, "rows": log(1, 400), "vocab": log(1000, 151936), "kind": rng.choice(["all", "mixed", "mixed", "free", "top_k", "top_p", "min_p", "greedy"]),
            "peaks": rng.choice([0, 8, 60, 60])}


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _image(g, wt, f16, rows, cols):
    """A matrix image: the quants of normal weights (as the writer's rule spreads them), padding to 64 bytes, the scales."""
    n = rows * cols
    size = n if wt == 1 else n // 2
    off = -(-size // 64) * 64
    W = torch.zeros(off + n // 32 * (2 if f16 else 4), dtype=torch.uint8, device="cuda")
    step = 1 << 26
    for lo in range(0, size, step):
        hi = min(size, lo + step)
        if wt == 1:
            q = torch.randn(hi - lo, device="cuda", generator=g).mul_(45).round_().clamp_(-127, 127).to(torch.int8).view(torch.uint8)
        else:
            nib = torch.randn((2, hi - lo), device="cuda", generator=g).mul_(2.8).add_(8.5).clamp_(0, 15.5).to(torch.uint8)
            q = nib[0] | (nib[1] << 4)
        W[lo:hi] = q
    d = (0.8 + 0.4 * torch.rand(n // 32, device="cuda", generator=g)) / (cols ** 0.5 * (45 if wt == 1 else 2.8))
    W[off:] = d.to(torch.float16 if f16 else torch.float32).view(torch.uint8)
    return W


def _settings(case, g):
    """Temperature, top-k, top-p and min-p of each row."""
    n, kind = case["rows"], case["kind"]

    def pick(values, dtype):
        at = torch.randint(0, len(values), (n,), device="cuda", generator=g)
        return torch.tensor(values, dtype=dtype, device="cuda")[at]

    warm = 0.6 + 0.7 * torch.rand(n, device="cuda", generator=g)
    top_k = pick([1, 20, 40, 50, 200, 1000], torch.int32)
    top_p = pick([0.5, 0.8, 0.9, 0.95, 0.99], torch.float32)
    min_p = pick([0.01, 0.02, 0.05, 0.1], torch.float32)
    if kind == "all":
        return {"temperature": warm, "top_k": torch.full_like(top_k, 40), "top_p": torch.full_like(top_p, 0.95), "min_p": torch.full_like(min_p, 0.02)}
    if kind == "mixed":
        off = torch.rand((4, n), device="cuda", generator=g)
        return {"temperature": torch.where(off[0] < 0.1, 0.0, warm), "top_k": torch.where(off[1] < 0.4, 0, top_k).to(torch.int32),
                "top_p": torch.where(off[2] < 0.4, 1.0, top_p), "min_p": torch.where(off[3] < 0.6, 0.0, min_p)}
    if kind == "greedy":
        return {"temperature": torch.zeros_like(warm), "top_k": None, "top_p": None, "min_p": None}
    return {"temperature": torch.ones_like(warm) if kind == "free" else warm, "top_k": top_k if kind == "top_k" else None,
            "top_p": top_p if kind == "top_p" else None, "min_p": min_p if kind == "min_p" else None}


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case), "op": op}
    if op == "embed":
        s["W"] = _image(g, case["wt"], case["f16"], case["vocab"], case["cols"])
        s["ids"] = torch.randint(0, case["vocab"], (case["rows"],), device="cuda", generator=g)
        return s
    if op == "rope":
        n, h, kvh, d = case["rows"], case["heads"], case["kv_heads"], case["dim"]
        # queries and keys are slices of a wider row, as a fused projection leaves them
        wide = torch.randn((n, (h + 2 * kvh) * d), device="cuda", generator=g)
        wide *= 1.0 + 4.0 * (torch.rand((1, wide.shape[1]), device="cuda", generator=g) > 0.98)
        s["wide"] = wide.to(_dtype(case["x"]))
        s["q"] = s["wide"][:, : h * d].unflatten(1, (h, d))
        s["k"] = s["wide"][:, h * d: (h + kvh) * d].unflatten(1, (kvh, d))
        s["qw"] = 1.0 + 0.2 * torch.randn(d, device="cuda", generator=g) if case["norm"] else None
        s["kw"] = 1.0 + 0.2 * torch.randn(d, device="cuda", generator=g) if case["norm"] else None
        first = torch.randint(0, case["far"], (1,), device="cuda", generator=g)
        s["pos"] = ((first + torch.arange(n, device="cuda") * 7919) % case["far"]).to(torch.int32)
        rot = case["rot"]
        s["freq"] = (500000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)).float()
        return s
    if op == "moe":
        e, d, h = case["experts"], case["dim"], case["hidden"]
        s["w1"] = _image(g, case["wt"], case["f16"], e * h, d)
        s["w3"] = _image(g, case["wt"], case["f16"], e * h, d)
        s["w2"] = _image(g, case["wt"], case["f16"], e * d, h)
        s["x"] = torch.randn((case["tokens"], d), device="cuda", generator=g).to(_dtype(case["x"]))
        s["logits"] = 1.5 * torch.randn((case["tokens"], e), device="cuda", generator=g)
        if own:
            import block_quantized_weight_q4_gb300 as qmv

            s["layer"] = qmv.Moe(case["wt"], case["wt"], qmv.SCALE_F16 if case["f16"] else qmv.SCALE_F32, e, d, h, s["w1"], s["w3"], s["w2"])
        return s
    n, v = case["rows"], case["vocab"]
    x = 2.2 * torch.randn((n, v), device="cuda", generator=g)
    if case["peaks"]:
        # the tokens that a context makes likely stand out of the rest
        at = torch.randint(0, v, (n, case["peaks"]), device="cuda", generator=g)
        sharp = 4.0 + 10.0 * torch.rand((n, 1), device="cuda", generator=g)
        x.scatter_add_(1, at, sharp * torch.rand(at.shape, device="cuda", generator=g) ** 0.5)
    x[:, v - v // 50:] = -math.inf  # the ids that a vocabulary pads itself with
    s["logits"] = x
    s["noise"] = torch.empty((n, v), device="cuda").exponential_(generator=g)
    s.update(_settings(case, g))
    return s


# ---------------------------------------------------------------------------- one pass
def _values(W, wt, f16, shape, at=None):
    """float32 weights of an image of (experts, rows, cols) matrices, of all of them or of those that `at` names."""
    e, rows, cols = shape
    n = e * rows * cols
    size = n if wt == 1 else n // 2
    q = W[:size].view(e, rows, cols // 32, 32 if wt == 1 else 16)
    d = W[-(-size // 64) * 64:].view(torch.float16 if f16 else torch.float32).view(e, rows, cols // 32, 1)
    if at is not None:
        q, d = q[at], d[at]
    if wt == 1:
        x = q.view(torch.int8).float()
    else:
        x = torch.cat((q & 15, q >> 4), dim=3).float() - 8.0
    return (x * d.float()).flatten(2)


def _plain_embed(s):
    c = s["case"]
    y = _values(s["W"], c["wt"], c["f16"], (c["vocab"], 1, c["cols"]), s["ids"])[:, 0]
    return (y * math.sqrt(c["cols"])).to(_dtype(c["out"]))


def _plain_rope_one(s, x, w):
    c = s["case"]
    x, rot = x.float(), c["rot"]
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * w
    t = s["pos"].double()[:, None, None] * s["freq"].double()
    cos, sin = t.cos().float(), t.sin().float()
    if c["pairs"] == "halves":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=2)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=3).flatten(2)
    return torch.cat((turned, x[..., rot:]), dim=2).to(_dtype(c["out"]))


def _act(name, g):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_moe(s):
    c = s["case"]
    t, e, k, d, h = c["tokens"], c["experts"], c["used"], c["dim"], c["hidden"]
    x, logits = s["x"].float(), s["logits"]
    best, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    best, ids = best[:, :k], ids[:, :k]
    p = torch.exp(best - best[:, :1])
    p = p / (p if c["renorm"] else torch.exp(logits - best[:, :1])).sum(dim=1, keepdim=True)
    if t * k < e:
        # few tokens: the experts that they use, one by one
        at = ids.flatten()
        pairs = x.repeat_interleave(k, dim=0)[:, :, None]
        gate = torch.bmm(_values(s["w1"], c["wt"], c["f16"], (e, h, d), at), pairs)
        up = torch.bmm(_values(s["w3"], c["wt"], c["f16"], (e, h, d), at), pairs)
        y = torch.bmm(_values(s["w2"], c["wt"], c["f16"], (e, d, h), at), _act(c["act"], gate) * up)
        out = (y.view(t, k, d) * p[:, :, None]).sum(dim=1)
    else:
        every = x.expand(e, t, d)
        gate = torch.bmm(every, _values(s["w1"], c["wt"], c["f16"], (e, h, d)).transpose(1, 2))
        up = torch.bmm(every, _values(s["w3"], c["wt"], c["f16"], (e, h, d)).transpose(1, 2))
        share = torch.zeros((t, e), device=x.device).scatter(1, ids, p).T[:, :, None]
        y = torch.bmm(_act(c["act"], gate) * up, _values(s["w2"], c["wt"], c["f16"], (e, d, h)).transpose(1, 2))
        out = (y * share).sum(dim=0)
    return {"out": out.to(_dtype(c["out"])), "ids": ids.to(torch.int32), "share": p}


def _plain_sample(s):
    x = s["logits"]
    n, v = x.shape
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    x, place = x.double(), torch.arange(v, device=x.device)
    top = x.amax(dim=1, keepdim=True)
    greedy = s["temperature"][:, None] == 0
    z = (x - top) / torch.where(greedy, 1.0, s["temperature"][:, None]).double()
    w = torch.exp(z).gather(1, order)
    keep = torch.ones((n, v), dtype=torch.bool, device=x.device)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (place < k) | (k == 0)
    if s["top_p"] is not None:
        mass = torch.where(keep, w, 0.0)
        before = mass.cumsum(dim=1) - mass
        p = s["top_p"].double()[:, None]
        keep &= (before < p * mass.sum(dim=1, keepdim=True)) | (p >= 1)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    score = torch.where(greedy, z, z - torch.log(s["noise"].double())).gather(1, order).masked_fill(~keep, -math.inf)
    best = score.amax(dim=1, keepdim=True)
    return torch.where(score == best, order, v).amin(dim=1)


def run(s):
    op, c = s["op"], s["case"]
    if not own:
        if op == "embed":
            return _plain_embed(s)
        if op == "rope":
            return {"q": _plain_rope_one(s, s["q"], s["qw"]), "k": _plain_rope_one(s, s["k"], s["kw"])}
        if op == "moe":
            return _plain_moe(s)
        return _plain_sample(s)
    import block_quantized_weight_q4_gb300 as qmv

    if op == "embed":
        return qmv.embed(c["wt"], qmv.SCALE_F16 if c["f16"] else qmv.SCALE_F32, c["vocab"], c["cols"], s["W"], s["ids"],
                         scale=math.sqrt(c["cols"]), out=c["out"])
    if op == "rope":
        q, k = qmv.qk_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, pairs=c["pairs"], out=c["out"])
        return {"q": q, "k": k}
    if op == "moe":
        out, ids, share = qmv.moe(s["layer"], s["x"], s["logits"], top=c["used"], renorm=c["renorm"], act=c["act"], out=c["out"], routing=True)
        return {"out": out, "ids": ids, "share": share}
    return qmv.sample(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "embed":
        per = case["cols"] * (1.0 if case["wt"] == 1 else 0.5) + case["cols"] / 32 * (2 if case["f16"] else 4)
        n = case["rows"] * case["cols"]
        # a row that is asked for again is read once
        rows = case["vocab"] * -math.expm1(case["rows"] * math.log1p(-1.0 / case["vocab"]))
        return {"bytes": rows * per + 8 * case["rows"] + size[case["out"]] * n, "flops": 2 * n}
    if op == "rope":
        n = case["rows"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": n * (size[case["x"]] + size[case["out"]]) + 4 * case["rows"], "flops": n * (3 + 4 * case["norm"])}
    if op == "moe":
        t, e, k, d, h = case["tokens"], case["experts"], case["used"], case["dim"], case["hidden"]
        used = e * (1.0 - (1.0 - k / e) ** t)  # experts that any token uses, by the routing's even spread
        weight = (1.0 if case["wt"] == 1 else 0.5) + (2 if case["f16"] else 4) / 32
        return {"bytes": 3 * used * d * h * weight + t * (d * (size[case["x"]] + size[case["out"]]) + 4 * e + 8 * k), "flops": 6 * t * k * d * h}
    n = case["rows"] * case["vocab"]
    # the random numbers of what nothing cuts off are all read, else those of the few that are left
    reads = 8 if case["kind"] == "free" else 4
    return {"bytes": reads * n + 24 * case["rows"], "flops": 4 * n}


# ---------------------------------------------------------------------------- the definition in 64 bits
def _exact_row(W, wt, f16, shape, expert):
    """One expert's matrix in float64, straight from the format: 32 weights to a block, each block a scale."""
    e, rows, cols = shape
    n = e * rows * cols
    size = n if wt == 1 else n // 2
    blocks = rows * cols // 32
    scales = W[-(-size // 64) * 64:].view(torch.float16 if f16 else torch.float32)[expert * blocks: (expert + 1) * blocks].double()
    if wt == 1:
        levels = W[expert * rows * cols: (expert + 1) * rows * cols].view(torch.int8).double().view(blocks, 32)
    else:
        b = W[expert * rows * cols // 2: (expert + 1) * rows * cols // 2].view(blocks, 16).int()
        levels = torch.empty((blocks, 32), dtype=torch.float64, device=W.device)
        levels[:, :16] = b.remainder(16) - 8
        levels[:, 16:] = b.div(16, rounding_mode="floor") - 8
    return (levels * scales[:, None]).view(rows, cols)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "embed":
        table = _exact_row(s["W"], case["wt"], case["f16"], (1, case["vocab"], case["cols"]), 0)
        return table[s["ids"]] * case["cols"] ** 0.5
    if op == "rope":
        got, rot = {}, case["rot"]
        turn = torch.polar(torch.ones((case["rows"], rot // 2), dtype=torch.float64, device="cuda"), torch.outer(s["pos"].double(), s["freq"].double()))
        for key, w in (("q", s["qw"]), ("k", s["kw"])):
            x = s[key].double()
            if w is not None:
                x = x / torch.sqrt((x ** 2).sum(dim=-1, keepdim=True) / case["dim"] + 1e-6) * w.double()
            first = x[..., : rot // 2] if case["pairs"] == "halves" else x[..., :rot][..., ::2]
            second = x[..., rot // 2: rot] if case["pairs"] == "halves" else x[..., :rot][..., 1::2]
            z = torch.complex(first.contiguous(), second.contiguous()) * turn[:, None]
            y = x.clone()
            if case["pairs"] == "halves":
                y[..., : rot // 2], y[..., rot // 2: rot] = z.real, z.imag
            else:
                y[..., :rot] = torch.view_as_real(z).flatten(-2)
            got[key] = y
        return got
    if op == "moe":
        t, e, k, d, h = case["tokens"], case["experts"], case["used"], case["dim"], case["hidden"]
        x, logits = s["x"].double(), s["logits"].double()
        p = torch.softmax(logits, dim=1)
        chosen = torch.zeros((t, e), dtype=torch.bool, device="cuda").scatter(1, torch.topk(logits, k, dim=1)[1], True)
        if case["renorm"]:
            p = torch.where(chosen, p, 0.0)
            p = p / p.sum(dim=1, keepdim=True)
        out = torch.zeros((t, d), dtype=torch.float64, device="cuda")
        for i in range(e):
            rows = chosen[:, i].nonzero()[:, 0]
            if rows.numel() == 0:
                continue
            gate = x[rows] @ _exact_row(s["w1"], case["wt"], case["f16"], (e, h, d), i).T
            up = x[rows] @ _exact_row(s["w3"], case["wt"], case["f16"], (e, h, d), i).T
            if case["act"] == "silu":
                hid = gate * torch.sigmoid(gate) * up
            else:
                hid = torch.nn.functional.gelu(gate, approximate="tanh") * up
            out[rows] += p[rows, i, None] * (hid @ _exact_row(s["w2"], case["wt"], case["f16"], (e, d, h), i).T)
        share = torch.sort(torch.where(chosen, p, -1.0), dim=1, descending=True)[0][:, :k]
        return {"out": out, "ids": None, "share": share}
    return None
