"""The operators between the products of a decode or prompt step, as cases that can be timed.

    norm     residual addition, root-mean-square norm, and the Q8_0 / f32-scale image that the
             activation-quantized product reads (or bfloat16 / float32 rows)
    write    new keys and values into the paged 8-bit cache (one scale for each page and head)
    read     tokens of that cache back as bfloat16 or float32
    attend   softmax attention of new queries over that cache: single tokens, short runs of
             tokens and whole prompt chunks, causal, with or without a sliding window
    logprobs log probabilities of given tokens, entropy and the top alternatives of a row of logits

`own` false: the plain form, elementary torch operations in float32 rounded once at the end.
`own` true: the calls of this repository's package.  Head counts, head sizes, hidden sizes and
vocabularies are those of the repository's benchmark layers (32 heads of 128 with 8 key/value
heads over 4096 columns, 1024 and 11008 columns, a vocabulary of 151936), the rest is generic.
"""
import math

import torch

own = False

GOLD = 0.6180339887498949


# ---------------------------------------------------------------------------- sizes of a case
def _lens(case):
    """Cached tokens of each sequence (its new tokens included), from the case alone."""
    n, hi, lo = case["seqs"], case["kv_max"], case["kv_min"]
    return [hi if i == 0 else int(round(lo + (hi - lo) * ((i * GOLD) % 1.0))) for i in range(n)]


def _news(case):
    """New tokens of each sequence: at most its cached tokens."""
    hi, lo = case["new_max"], case["new_min"]
    got = [hi if i == 0 else int(round(lo + (hi - lo) * ((i * GOLD + 0.5) % 1.0))) for i in range(case["seqs"])]
    return [min(a, b) for a, b in zip(got, _lens(case))]


def _reads(case):
    return [min(a, case["back"]) for a in _lens(case)]


def _pairs(case):
    """Query-key pairs that the mask leaves, over all sequences (one head)."""
    total = 0
    for length, new in zip(_lens(case), _news(case)):
        w = case["window"]
        # position p = length - new .. length - 1 sees min(p + 1, w) keys
        a, b = length - new + 1, length
        if not w or b <= w:
            total += (a + b) * new // 2
        elif a > w:
            total += w * new
        else:
            total += (a + w) * (w - a + 1) // 2 + w * (b - w)
    return total


def listed():
    return [
        # one token's hidden row between two products of a decode step: the smallest call there is
        {"name": "norm_decode_1x4096", "op": "norm", "rows": 1, "cols": 4096, "x": "f32", "out": "q8"},
        # a prompt chunk's rows, bfloat16 activations into a float32 residual stream
        {"name": "norm_prompt_2048x4096", "op": "norm", "rows": 2048, "cols": 4096, "x": "bf16", "out": "q8"},
        # a decode step of 64 sequences: one new token each (float32, as the products leave it), and
        # the pages' newest tokens read back
        {"name": "write_decode_64", "op": "write", "seqs": 64, "kv_max": 4000, "kv_min": 70, "new_max": 1, "new_min": 1,
         "back": 33, "kv_heads": 8, "dim": 128, "page": 64, "x": "f32", "out": "f32"},
        # a prompt batch of ragged lengths written page by page, and read back for a further pass
        {"name": "write_prompt_ragged_5", "op": "write", "seqs": 5, "kv_max": 4096, "kv_min": 513, "new_max": 4096,
         "new_min": 301, "back": 4096, "kv_heads": 8, "dim": 128, "page": 64, "x": "bf16", "out": "bf16"},
        # a long cache read back as bfloat16 (moving a conversation to another program)
        {"name": "read_16x16384", "op": "read", "seqs": 16, "kv_max": 16384, "kv_min": 9000, "new_max": 0, "new_min": 0,
         "back": 16384, "kv_heads": 8, "dim": 128, "page": 64, "x": "bf16", "out": "bf16"},
        # one conversation's next token: latency
        {"name": "attend_decode_1x1000", "op": "attend", "seqs": 1, "kv_max": 1000, "kv_min": 1000, "new_max": 1,
         "new_min": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "x": "bf16"},
        # a serving batch with long ragged conversations: the cache's bytes
        {"name": "attend_decode_64x16384", "op": "attend", "seqs": 64, "kv_max": 16384, "kv_min": 1200, "new_max": 1,
         "new_min": 1, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "x": "bf16"},
        # float32 rows, as many key/value heads as heads, heads of 64, small pages, a sliding window
        {"name": "attend_decode_f32_9x5001", "op": "attend", "seqs": 9, "kv_max": 5001, "kv_min": 17, "new_max": 3,
         "new_min": 1, "heads": 16, "kv_heads": 16, "dim": 64, "page": 16, "window": 2047, "x": "f32"},
        # whole prompts, ragged, nothing cached before
        {"name": "attend_prompt_3x2048", "op": "attend", "seqs": 3, "kv_max": 2048, "kv_min": 777, "new_max": 2048,
         "new_min": 2048, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "x": "bf16"},
        # a chunk of a long prompt over what was cached before it: the arithmetic
        {"name": "attend_chunk_2048_of_16384", "op": "attend", "seqs": 1, "kv_max": 16384, "kv_min": 16384, "new_max": 2048,
         "new_min": 2048, "heads": 32, "kv_heads": 8, "dim": 128, "page": 64, "window": 0, "x": "bf16"},
        # one row of logits: the sampled token's probability and its alternatives
        {"name": "logprobs_1x151936", "op": "logprobs", "rows": 1, "vocab": 151936, "given": 1, "top": 8},
        # scoring a prompt: every position's given token
        {"name": "logprobs_512x151936", "op": "logprobs", "rows": 512, "vocab": 151936, "given": 1, "top": 5},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "write", "read", "attend", "attend", "attend", "logprobs"])
    if op == "norm":
        return {"op": op, "rows": log(1, 2048), "cols": 32 * log(8, 344), "x": rng.choice(["f32", "bf16"]),
                "out": rng.choice(["q8", "q8", "bf16", "f32"])}
    if op == "logprobs":
        return {"op": op, "rows": log(1, 500), "vocab": log(1000, 151936), "given": rng.choice([1, 1, 2, 5]),
                "top": rng.choice([1, 3, 5, 8, 20])}
    heads = rng.choice([(32, 8), (32, 8), (16, 16), (14, 2), (32, 32), (8, 1)])
    case = {"op": op, "kv_heads": heads[1], "dim": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 64, 128]),
            "x": rng.choice(["bf16", "bf16", "f32"])}
    if op == "attend":
        case["heads"] = heads[0]
        case["window"] = rng.choice([0, 0, 0, log(16, 4096)])
        kind = rng.choice(["decode", "decode", "few", "prompt"])
        if kind == "prompt":
            case.update(seqs=rng.randint(1, 4), kv_max=log(64, 4096), kv_min=1, new_max=0, new_min=0, x="bf16")
            case["new_max"] = max(1, int(case["kv_max"] * rng.choice([1.0, 1.0, 0.3])))
            case["new_min"] = max(1, case["new_max"] // 3)
        else:
            case.update(seqs=log(1, 48), kv_max=log(20, 8192), kv_min=1, new_max=1 if kind == "decode" else rng.randint(2, 9), new_min=1)
        return case
    case.update(seqs=log(1, 16), kv_max=log(8, 8192), kv_min=1, out=case["x"])
    case["new_max"] = 0 if op == "read" else rng.choice([1, 1, log(2, 1024)])
    case["new_min"] = 0 if op == "read" else 1
    case["back"] = case["kv_max"] if op == "read" else max(case["page"], min(2 * case["new_max"], case["kv_max"]))
    return case


# ---------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _dtype(name):
    return torch.float32 if name == "f32" else torch.bfloat16


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _starts(counts):
    total, got = 0, [0]
    for c in counts:
        total += c
        got.append(total)
    return got


def _pool(g, pages, heads, page, dim):
    """int8 levels and float32 scales of `pages` pages of normal values with a few loud channels."""
    x = torch.randn((pages, heads, page, dim), device="cuda", generator=g)
    x *= 1.0 + 3.0 * (torch.rand((1, heads, 1, dim), device="cuda", generator=g) > 0.97)
    d = x.abs().amax(dim=(2, 3)) / 127
    x /= d[:, :, None, None]
    return x.round_().clamp_(-127, 127).to(torch.int8), d.contiguous()


def _cache(case, g):
    """The paged cache, its page table in a shuffled order, and the call's tokens."""
    page, lens = case["page"], _lens(case)
    need = [-(-n // page) for n in lens]
    width, pages = max(need), sum(need) + 3
    order = torch.randperm(pages, device="cuda", generator=g).to(torch.int32)
    at = _starts(need)
    cols = torch.arange(width, device="cuda")
    first = _ints(at[:-1], torch.int64)
    have = _ints(need, torch.int64)
    table = order[(first[:, None] + cols[None, :]).clamp(max=pages - 1)]
    table = torch.where(cols[None, :] < have[:, None], table, torch.full_like(table, -1)).contiguous()
    k, ks = _pool(g, pages, case["kv_heads"], page, case["dim"])
    v, vs = _pool(g, pages, case["kv_heads"], page, case["dim"])
    return {"k": k, "v": v, "k_scale": ks, "v_scale": vs, "table": table, "len": _ints(lens), "max_len": max(lens)}


def _handles(s, counts, key):
    """What a program keeps beside its cache: the cache's handle, and the rows of a kind of call."""
    import block_quantized_weight_q4_gb300 as qmv

    s["cache"] = qmv.KvCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    s[key] = qmv.KvBatch(s["table"], s["len"], starts=_ints(_starts(counts)), rows=sum(counts), max_rows=max(counts),
                         max_len=s["max_len"])


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case), "op": op}
    if op == "norm":
        r, c = case["rows"], case["cols"]
        s["x"] = torch.randn((r, c), device="cuda", generator=g).to(_dtype(case["x"]))
        loud = 1.0 + 20.0 * (torch.rand((1, c), device="cuda", generator=g) > 0.999)
        s["res"] = 2.0 * torch.randn((r, c), device="cuda", generator=g) * loud
        s["w"] = 1.0 + 0.1 * torch.randn((c,), device="cuda", generator=g)
        s["sum"] = torch.empty_like(s["res"])
        return s
    if op == "logprobs":
        r, v = case["rows"], case["vocab"]
        s["logits"] = 2.5 * torch.randn((r, v), device="cuda", generator=g)
        s["logits"][:, v - v // 50:] = -math.inf  # the ids that a vocabulary pads itself with
        s["given"] = torch.randint(0, v - v // 50, (r, case["given"]), device="cuda", generator=g)
        return s
    s.update(_cache(case, g))
    h, d, news = case["kv_heads"], case["dim"], _news(case)
    s["news"], s["reads"] = news, _reads(case) if op != "attend" else []
    if op == "attend":
        # the queries are a slice of a wider row, as a fused projection leaves them
        wide = torch.randn((sum(news), case["heads"] * d + 2 * h * d), device="cuda", generator=g) * 1.5
        s["wide"] = wide.to(_dtype(case["x"]))
        s["q"] = s["wide"][:, : case["heads"] * d].unflatten(1, (case["heads"], d))
    else:
        loud = 1.0 + 3.0 * (torch.rand((1, 2, h, 1), device="cuda", generator=g) > 0.7)
        s["kv"] = (torch.randn((sum(news), 2, h, d), device="cuda", generator=g) * loud).to(_dtype(case["x"]))
    if own:
        if op != "read":
            _handles(s, news, "rows")
        if op != "attend":
            _handles(s, s["reads"], "back")
    # the plain form's indices: row r of the call is token pos[r] of sequence seq[r]
    for key, counts in (("new", news), ("back", s["reads"])):
        n = _ints(counts or [0], torch.int64)
        seq = torch.repeat_interleave(torch.arange(n.numel(), device="cuda"), n)
        pos = torch.arange(seq.numel(), device="cuda") - (torch.cumsum(n, 0) - n)[seq] + (s["len"].long()[: n.numel()] - n)[seq]
        s[key + "_seq"], s[key + "_pos"] = seq, pos
        if key == "new":
            s["first"] = s["len"].long()[: n.numel()] - n
    return s


# ---------------------------------------------------------------------------- one pass
def _plain_norm(s):
    c = s["case"]
    h = s["x"].float() + s["res"]
    r = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + 1e-5)
    t = h * s["w"]
    if c["out"] != "q8":
        return {"sum": h, "y": (t * r).to(_dtype(c["out"]))}
    # the row's factor r is common to its blocks, so the levels do not depend on it: it goes to the scales
    b = t.view(c["rows"], -1, 32)
    top = b.abs().amax(dim=2, keepdim=True)
    zero = top < 1e-30
    inv = torch.where(zero, torch.zeros_like(top), 127.0 / top)
    q = torch.trunc(b * inv + torch.copysign(torch.full_like(b, 0.5), b)).clamp(-127, 127)
    d = torch.where(zero, torch.zeros_like(top), top / 127.0) * r[:, :, None]
    return {"sum": h, "y": (q * d).view(c["rows"], c["cols"])}


def _plain_write_one(s, pool, scale, x):
    """New rows x (rows, heads, dim) into one pool: the page's scale is the largest it has needed so far."""
    page = s["case"]["page"]
    seq, pos = s["new_seq"], s["new_pos"]
    slot = s["table"][seq, pos // page].long()
    heads = scale.shape[1]
    top = torch.zeros_like(scale).scatter_reduce(0, slot[:, None].expand(-1, heads), x.abs().amax(dim=2), "amax")
    want = torch.where(top < 1e-30, torch.zeros_like(top), top / 127.0)
    # pages whose first tokens were there before the call: the page of each sequence's first new token
    old = torch.zeros(scale.shape[0], dtype=torch.int64, device=x.device)
    lead = pos == s["first"][seq]
    old.scatter_reduce_(0, slot, torch.where(lead, pos % page, torch.zeros_like(pos)), "amax")
    had = torch.where(old[:, None] > 0, scale, torch.zeros_like(scale))
    new = torch.maximum(want, had)
    lead_slot = slot[lead]  # one page for each sequence with new tokens
    ratio = torch.where(new > 0, had / new, torch.ones_like(new))[lead_slot][:, :, None, None]
    levels = pool[lead_slot].float()
    moved = torch.trunc(levels * ratio + torch.copysign(torch.full_like(levels, 0.5), levels))
    raised = (new > had)[lead_slot][:, :, None, None]
    kept = torch.arange(page, device=x.device)[None, None, :, None] < old[lead_slot][:, None, None, None]
    pool[lead_slot] = torch.where(raised & kept, moved, levels).to(torch.int8)
    inv = torch.where(new > 0, 1.0 / new, torch.zeros_like(new))[slot][:, :, None]
    q = torch.trunc(x * inv + torch.copysign(torch.full_like(x, 0.5), x)).clamp(-127, 127)
    pool[slot, :, pos % page] = q.to(torch.int8)
    touched = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device)
    touched[slot] = True
    scale.copy_(torch.where(touched[:, None], new, scale))


def _plain_read(s, pool, scale):
    page = s["case"]["page"]
    seq, pos = s["back_seq"], s["back_pos"]
    slot = s["table"][seq, pos // page].long()
    return (pool[slot, :, pos % page].float() * scale[slot][:, :, None]).to(_dtype(s["case"]["out"]))


def _plain_attend(s):
    c = s["case"]
    page, h, d, group = c["page"], c["kv_heads"], c["dim"], c["heads"] // c["kv_heads"]
    seqs, width = s["table"].shape
    at = s["table"].clamp(min=0).long()

    def whole(pool, scale):  # (sequences, heads, tokens, dim)
        x = pool[at].float() * scale[at][:, :, :, None, None]
        return x.transpose(1, 2).reshape(seqs, h, width * page, d)

    k, v = whole(s["k"], s["k_scale"]), whole(s["v"], s["v_scale"])
    most = max(s["news"])
    seq, pos = s["new_seq"], s["new_pos"]
    place = pos - s["first"][seq]
    q = torch.zeros((seqs, most, c["heads"], d), device=k.device)
    q[seq, place] = s["q"].float()
    q = q.view(seqs, most, h, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, h, group * most, d)
    p = torch.matmul(q, k.transpose(2, 3))
    p *= 1.0 / math.sqrt(d)
    j = torch.arange(width * page, device=k.device)
    own_pos = s["first"][:, None] + torch.arange(most, device=k.device)[None, :]
    hide = (j[None, None, :] > own_pos[:, :, None]) | (j[None, None, :] >= s["len"].long()[:, None, None])
    if c["window"]:
        hide |= j[None, None, :] <= own_pos[:, :, None] - c["window"]
    p.view(seqs, h, group, most, -1).masked_fill_(hide[:, None, None], -math.inf)
    top = p.amax(dim=3, keepdim=True).clamp(min=-3e38)
    p -= top
    p.exp_()
    o = torch.matmul(p, v) / p.sum(dim=3, keepdim=True).clamp(min=1e-30)
    o = o.view(seqs, h, group, most, d).permute(0, 3, 1, 2, 4).reshape(seqs, most, c["heads"], d)
    return o[seq, place].to(_dtype(c["x"]))


def _plain_logprobs(s):
    x, top = s["logits"], s["case"]["top"]
    m = x.amax(dim=1, keepdim=True)
    e = torch.exp(x - m)
    z = e.sum(dim=1, keepdim=True)
    lse = m + torch.log(z)
    mean = torch.where(e > 0, e * (x - m), torch.zeros_like(e)).sum(dim=1, keepdim=True) / z
    best, ids = torch.sort(x, dim=1, descending=True, stable=True)
    return {"given": torch.gather(x, 1, s["given"]) - lse, "entropy": (torch.log(z) - mean)[:, 0],
            "top_ids": ids[:, :top].to(torch.int32), "top": best[:, :top] - lse}


def run(s):
    op, c = s["op"], s["case"]
    if not own:
        if op == "norm":
            return _plain_norm(s)
        if op == "logprobs":
            return _plain_logprobs(s)
        if op == "attend":
            return _plain_attend(s)
        if op == "write":
            _plain_write_one(s, s["k"], s["k_scale"], s["kv"][:, 0].float())
            _plain_write_one(s, s["v"], s["v_scale"], s["kv"][:, 1].float())
        return {"k": _plain_read(s, s["k"], s["k_scale"]), "v": _plain_read(s, s["v"], s["v_scale"])}
    import block_quantized_weight_q4_gb300 as qmv

    if op == "norm":
        y = qmv.rmsnorm(s["x"], s["w"], 1e-5, residual=s["res"], residual_out=s["sum"], out=c["out"])
        if c["out"] == "q8":  # the values that the 8-bit image stands for
            y = qmv.dequant(qmv.Q8_0, qmv.SCALE_F32, c["rows"], c["cols"], y)
        return {"sum": s["sum"], "y": y}
    if op == "logprobs":
        given, entropy, ids, best = qmv.logprobs(s["logits"], s["given"], top=c["top"])
        return {"given": given, "entropy": entropy, "top_ids": ids, "top": best}
    if op == "attend":
        return qmv.attend(s["cache"], s["rows"], s["q"], window=c["window"])
    if op == "write":
        qmv.kv_write(s["cache"], s["rows"], s["kv"][:, 0], s["kv"][:, 1])
    k, v = qmv.kv_read(s["cache"], s["back"], _dtype(c["out"]))
    return {"k": k, "v": v}


# ---------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    size = {"f32": 4, "bf16": 2}
    if op == "norm":
        n = case["rows"] * case["cols"]
        # x and the residual read, their sum and the row's values written, the weight once; the 8-bit
        # image (36 bytes for 32 values) is written and read where the values come from it
        out = 4 * n + 2 * (n + n // 8) if case["out"] == "q8" else size[case["out"]] * n
        return {"bytes": n * (size[case["x"]] + 8) + out + 4 * case["cols"], "flops": 6 * n}
    if op == "logprobs":
        n = case["rows"] * case["vocab"]
        return {"bytes": 4 * n + case["rows"] * (12 * case["given"] + 8 * case["top"] + 4), "flops": 6 * n}
    lens, news, h, d, page = _lens(case), _news(case), case["kv_heads"], case["dim"], case["page"]
    if op == "attend":
        w, x = case["window"], size[case["x"]]
        span = [n if not w else min(n, w + m - 1) for n, m in zip(lens, news)]
        pages = sum(-(-n // page) for n in span)
        nbytes = 2 * h * d * sum(span) + pages * (8 * h + 4) + 2 * x * sum(news) * case["heads"] * d
        return {"bytes": nbytes, "flops": 4 * _pairs(case) * case["heads"] * d}
    back = sum(_reads(case))
    pages = sum(-(-n // page) for n in _reads(case))
    nbytes = 2 * h * d * back * (1 + size[case["out"]]) + pages * (8 * h + 4)
    if op == "write":
        nbytes += 2 * h * d * sum(news) * (size[case["x"]] + 1) + 8 * h * sum(-(-n // page) for n in news)
    return {"bytes": nbytes, "flops": 2 * h * d * (back + 3 * sum(news))}


# ---------------------------------------------------------------------------- the definition in 64 bits
def _half_away(x):
    return torch.sign(x) * torch.floor(x.abs() + 0.5)


def _exact_write(s, pool, scale, x):
    """Page by page, from the definition: raise the scale if the new tokens need it, move the old levels."""
    page, table = s["case"]["page"], s["table"].tolist()
    levels, d = pool.double(), scale.double()
    row = 0
    for i, (length, new) in enumerate(zip(s["len"].tolist(), s["news"])):
        pos = length - new
        while pos < length:
            end = min(length, (pos // page + 1) * page)
            at, off = table[i][pos // page], pos % page
            new_rows = x[row: row + end - pos].transpose(0, 1)
            need = new_rows.abs().amax(dim=(1, 2))
            need = torch.where(need < 1e-30, torch.zeros_like(need), need / 127)
            had = d[at] if off else torch.zeros_like(need)
            now = torch.maximum(need, had)
            safe = torch.where(now > 0, now, torch.ones_like(now))[:, None, None]
            if off:
                moved = _half_away(levels[at, :, :off] * (had[:, None, None] / safe))
                levels[at, :, :off] = torch.where((now > had)[:, None, None], moved, levels[at, :, :off])
            q = torch.where(now[:, None, None] > 0, _half_away(new_rows / safe), torch.zeros_like(new_rows))
            levels[at, :, off: off + end - pos] = q.clamp(-127, 127)
            d[at] = now
            row, pos = row + end - pos, end
    return levels, d


def _exact_read(s, levels, d):
    page, table, got = s["case"]["page"], s["table"], []
    for i, (length, n) in enumerate(zip(s["len"].tolist(), s["reads"])):
        pages = table[i, : -(-length // page)].long()
        x = levels[pages].double() * d[pages].double()[:, :, None, None]
        got.append(x.transpose(1, 2).reshape(-1, x.shape[1], x.shape[3])[length - n: length])
    return torch.cat(got)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["res"].double()
        r = 1.0 / torch.sqrt((h ** 2).sum(dim=1, keepdim=True) / case["cols"] + 1e-5)
        y = h * r * s["w"].double()
        if case["out"] == "q8":
            blocks = y.reshape(-1, 32)
            d = blocks.abs().max(dim=1, keepdim=True).values / 127
            y = torch.where(d > 0, _half_away(blocks / d).clamp(-127, 127) * d, torch.zeros_like(blocks)).reshape(y.shape)
        return {"sum": h, "y": y}
    if op == "logprobs":
        given, entropy, top = [], [], []
        for i in range(case["rows"]):
            x = s["logits"][i].double()
            lp = x - torch.logsumexp(x, 0)
            live = lp[torch.isfinite(lp)]
            given.append(lp[s["given"][i]])
            entropy.append(-(live.exp() * live).sum())
            top.append(torch.topk(lp, case["top"]).values)
        return {"given": torch.stack(given), "entropy": torch.stack(entropy), "top_ids": None, "top": torch.stack(top)}
    if op != "attend":
        got = {}
        for i, key in enumerate(("k", "v")):
            levels, d = s[key], s[key + "_scale"]
            if op == "write":
                levels, d = _exact_write(s, levels, d, s["kv"][:, i].double())
            got[key] = _exact_read(s, levels, d)
        return got
    h, d, page, group = case["kv_heads"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    out = torch.empty((sum(s["news"]), case["heads"], d), dtype=torch.float64, device="cuda")
    row = 0
    for i, (length, n) in enumerate(zip(s["len"].tolist(), s["news"])):
        pages = s["table"][i, : -(-length // page)].long()
        for a in range(h):
            k = (s["k"][pages, a].double() * s["k_scale"][pages, a].double()[:, None, None]).reshape(-1, d)[:length]
            v = (s["v"][pages, a].double() * s["v_scale"][pages, a].double()[:, None, None]).reshape(-1, d)[:length]
            j = torch.arange(length, device="cuda")
            for lo in range(0, n, 1024):
                hi = min(n, lo + 1024)
                p = torch.arange(length - n + lo, length - n + hi, device="cuda")[:, None]
                seen = j <= p
                if case["window"]:
                    seen &= j > p - case["window"]
                for b in range(a * group, (a + 1) * group):
                    z = s["q"][row + lo: row + hi, b].double() @ k.T / math.sqrt(d)
                    w = torch.softmax(z.masked_fill(~seen, -math.inf), dim=1)
                    out[row + lo: row + hi, b] = w @ v
        row += n
    return out
