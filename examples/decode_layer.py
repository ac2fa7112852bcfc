"""A small transformer run on quantized weights and an 8-bit cache: the products of this library with the
operators between them, for a prompt and then token by token.

    python examples/decode_layer.py [--layers 2] [--tokens 12] [--experts 8] [--temperature 0.8 --top-k 50 --top-p 0.95]

Random weights (Q4_0, f16 scales): nothing is loaded, so the text it would write means nothing; what it shows
is how the calls fit together.  The tokens' rows come from a quantized table (embed); a layer is

    s += y;  xq = norm(s) in 8 bits       one rmsnorm call (the residual's addition, the norm, the quantizer)
    q, k, v = Wq xq, Wk xq, Wv xq         matvec_qx (activation-quantized products)
    norms and rotary positions of q and k qk_rope
    cache <- k, v;  o = attention         kv_write, attend
    y = Wo o                              matvec
    s += y;  xq = norm(s)                 rmsnorm
    y = W2 (silu(W1 xq) * (W3 xq))        matvec_qx, then the gated product; with --experts
    x = norm(s) in bfloat16, l = Wr x     rmsnorm, matvec (the router's logits)
    y = sum of the best experts' FFNs     moe

and the last rows go through a final norm and the classifier; sample takes the next token from the logits and
logprobs tells its log probability.
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Model:
    """Random weights of a small model, its caches, and the step that reads them."""

    def __init__(self, layers=2, dim=1024, heads=16, kv_heads=4, hidden=2048, vocab=4096, page_tokens=64, pages=64, seed=0,
                 experts=0, top=2):
        import torch
        import block_quantized_weight_q4_gb300 as qmv
        self.qmv, self.torch = qmv, torch
        self.dim, self.heads, self.kv_heads, self.hidden, self.vocab = dim, heads, kv_heads, hidden, vocab
        self.head_dim, self.experts, self.top = dim // heads, experts, min(top, max(experts, 1))
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(rows, cols):
            w = torch.randn((rows, cols), device="cuda", generator=g) / cols ** 0.5
            return qmv.quantize(qmv.Q4_0, qmv.SCALE_F16, w)[0]

        kv = kv_heads * self.head_dim
        n = max(experts, 1)  # the experts' matrices one under the other: that of all of them
        self.layers = [{"wq": matrix(dim, dim), "wk": matrix(kv, dim), "wv": matrix(kv, dim), "wo": matrix(dim, dim),
                        "w1": matrix(n * hidden, dim), "w3": matrix(n * hidden, dim), "w2": matrix(n * dim, hidden),
                        "n1": torch.ones(dim, device="cuda"), "n2": torch.ones(dim, device="cuda"),
                        "cache": qmv.KvCache.empty(pages, kv_heads, self.head_dim, page_tokens)} for _ in range(layers)]
        for w in self.layers if experts else ():
            w["router"] = matrix(experts, dim)
            w["moe"] = qmv.Moe(qmv.Q4_0, qmv.Q4_0, qmv.SCALE_F16, experts, dim, hidden, w["w1"], w["w3"], w["w2"])
        for w in self.layers:
            w["qn"], w["kn"] = (torch.ones(self.head_dim, device="cuda") for _ in range(2))
        self.emb = matrix(vocab, dim)  # of variance 1 / dim, as every matrix here
        self.cls = matrix(vocab, dim)
        self.nf = torch.ones(dim, device="cuda")
        self.freq = 10000.0 ** (-torch.arange(0, self.head_dim, 2, device="cuda", dtype=torch.float32) / self.head_dim)

    def product(self, W, rows, xq, n):
        return self.qmv.matvec_qx(self.qmv.Q4_0, self.qmv.SCALE_F16, rows, self.dim, W, xq, n)

    def ffn(self, w, s, y, n):
        """s += y, then the layer's FFN, or that of its experts."""
        qmv, torch = self.qmv, self.torch
        if self.experts:
            x = qmv.rmsnorm(y, w["n2"], residual=s, residual_out=s, out="bf16")
            logits = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, self.experts, self.dim, w["router"], x)
            return qmv.moe(w["moe"], x, logits, self.top)
        xq = qmv.rmsnorm(y, w["n2"], residual=s, residual_out=s, out="q8")
        gate_up = torch.empty((2, n, self.hidden), device="cuda")
        qmv.matvec_qx(qmv.Q4_0, qmv.SCALE_F16, self.hidden, self.dim, w["w1"], xq, n, y=gate_up[0])
        qmv.matvec_qx(qmv.Q4_0, qmv.SCALE_F16, self.hidden, self.dim, w["w3"], xq, n, y=gate_up[1])
        y = torch.empty((n, self.dim), device="cuda")
        qmv.matvec_grouped(qmv.Q4_0, qmv.SCALE_F16, [(self.dim, self.hidden, w["w2"], gate_up, y)], act="silu")
        return y

    def step(self, tokens, batch, pos):
        """One pass: tokens (rows,) int64 at positions pos (rows,) int32, the rows of `batch`.  Returns logits."""
        qmv, torch = self.qmv, self.torch
        n, h, kvh, d = tokens.numel(), self.heads, self.kv_heads, self.head_dim
        y = qmv.embed(qmv.Q4_0, qmv.SCALE_F16, self.vocab, self.dim, self.emb, tokens, scale=self.dim ** 0.5)
        s = torch.zeros((n, self.dim), device="cuda")
        for w in self.layers:
            xq = qmv.rmsnorm(y, w["n1"], residual=s, residual_out=s, out="q8")
            q = self.product(w["wq"], h * d, xq, n).view(n, h, d)
            k = self.product(w["wk"], kvh * d, xq, n).view(n, kvh, d)
            v = self.product(w["wv"], kvh * d, xq, n).view(n, kvh, d)
            q, k = qmv.qk_rope(q, k, pos, self.freq, w["qn"], w["kn"], pairs="neighbours", out="bf16")
            qmv.kv_write(w["cache"], batch, k, v.bfloat16())
            o = qmv.attend(w["cache"], batch, q)
            y = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, self.dim, self.dim, w["wo"], o.view(n, self.dim))
            y = self.ffn(w, s, y, n)
        x = qmv.rmsnorm(y, self.nf, residual=s, out="bf16")
        return qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, self.vocab, self.dim, self.cls, x)

    def prompt(self, tokens, table):
        """A whole prompt into empty caches.  Returns the logits of every position."""
        torch = self.torch
        n = tokens.numel()
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        length = torch.tensor([n], dtype=torch.int32, device="cuda")
        batch = self.qmv.KvBatch(table, length, starts=starts, rows=n, max_rows=n, max_len=n)
        return self.step(tokens, batch, torch.arange(n, device="cuda", dtype=torch.int32))


def run(layers=2, tokens=12, prompt=70, seed=0, experts=0, temperature=0.0, top_k=0, top_p=1.0):
    """A prompt, then `tokens` sampled tokens (temperature 0: the most probable ones).  Returns the tokens, the log
    probability that each had when it was chosen, and the same from one prompt pass over all of them."""
    import torch
    m = Model(layers=layers, seed=seed, experts=experts)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    table = torch.randperm(32, device="cuda", generator=g).to(torch.int32).view(1, 32)
    text = torch.randint(0, m.vocab, (prompt,), device="cuda", generator=g)
    logits = m.prompt(text, table)
    length = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    batch = m.qmv.KvBatch(table, length, max_len=prompt + tokens)
    how = {"temperature": torch.full((1,), temperature, device="cuda"), "top_p": torch.full((1,), top_p, device="cuda"),
           "top_k": torch.full((1,), top_k, dtype=torch.int32, device="cuda")}
    noise = torch.empty((1, m.vocab), device="cuda")
    chosen, picked = [], []
    for _ in range(tokens):
        ids = m.qmv.sample(logits[-1:], noise.exponential_(generator=g), **how)
        given, _, _, _ = m.qmv.logprobs(logits[-1:], ids[:, None])
        chosen.append(ids)
        picked.append(given[0, 0])
        length += 1
        logits = m.step(ids, batch, length - 1)
    text = torch.cat([text, *chosen])
    whole = m.prompt(text, 31 - table)  # other pages, from the start
    given, _, _, _ = m.qmv.logprobs(whole[prompt - 1:-1], text[prompt:, None])
    assert m.qmv.last_error() == 0
    return text[prompt:].tolist(), torch.stack(picked).cpu().numpy(), given[:, 0].cpu().numpy()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=12)
    ap.add_argument("--experts", type=int, default=0, help="experts a layer, two for each token, or the one there is (0: one FFN)")
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--top-k", type=int, default=0)
    ap.add_argument("--top-p", type=float, default=1.0)
    a = ap.parse_args()
    ids, picked, whole = run(a.layers, a.tokens, experts=a.experts, temperature=a.temperature, top_k=a.top_k, top_p=a.top_p)
    print("tokens                   ", ids)
    print("log p, token by token    ", np.round(picked, 3))
    print("log p, one prompt pass   ", np.round(whole, 3))


if __name__ == "__main__":
    main()
