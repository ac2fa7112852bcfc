"""A small transformer run on quantized weights and an 8-bit cache: the products of this library with the
operators between them, for a prompt and then token by token.

    python examples/decode_layer.py [--layers 2] [--tokens 12]

Random weights (Q4_0, f16 scales): nothing is loaded, so the text it would write means nothing; what it shows
is how the calls fit together.  A layer is

    s += y;  xq = norm(s) in 8 bits       one rmsnorm call (the residual's addition, the norm, the quantizer)
    q, k, v = Wq xq, Wk xq, Wv xq         matvec_qx (activation-quantized products)
    rotary positions on q and k           torch, elementwise
    cache <- k, v;  o = attention         kv_write, attend
    y = Wo o                              matvec
    s += y;  xq = norm(s)                 rmsnorm
    y = W2 (silu(W1 xq) * (W3 xq))        matvec_qx, then the gated product

and the last rows go through a final norm, the classifier and logprobs.
"""
import argparse
import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


class Model:
    """Random weights of a small model, its caches, and the step that reads them."""

    def __init__(self, layers=2, dim=1024, heads=16, kv_heads=4, hidden=2048, vocab=4096, page_tokens=64, pages=64, seed=0):
        import torch
        import block_quantized_weight_q4_gb300 as qmv
        self.qmv, self.torch = qmv, torch
        self.dim, self.heads, self.kv_heads, self.hidden, self.vocab = dim, heads, kv_heads, hidden, vocab
        self.head_dim = dim // heads
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def matrix(rows, cols):
            w = torch.randn((rows, cols), device="cuda", generator=g) / cols ** 0.5
            return qmv.quantize(qmv.Q4_0, qmv.SCALE_F16, w)[0]

        kv = kv_heads * self.head_dim
        self.layers = [{"wq": matrix(dim, dim), "wk": matrix(kv, dim), "wv": matrix(kv, dim), "wo": matrix(dim, dim),
                        "w1": matrix(hidden, dim), "w3": matrix(hidden, dim), "w2": matrix(dim, hidden),
                        "n1": torch.ones(dim, device="cuda"), "n2": torch.ones(dim, device="cuda"),
                        "cache": qmv.KvCache.empty(pages, kv_heads, self.head_dim, page_tokens)} for _ in range(layers)]
        self.emb = torch.randn((vocab, dim), device="cuda", generator=g)
        self.cls = matrix(vocab, dim)
        self.nf = torch.ones(dim, device="cuda")
        self.freq = 10000.0 ** (-torch.arange(0, self.head_dim, 2, device="cuda") / self.head_dim)

    def product(self, W, rows, xq, n):
        return self.qmv.matvec_qx(self.qmv.Q4_0, self.qmv.SCALE_F16, rows, self.dim, W, xq, n)

    def rotate(self, x, pos):
        """x (rows, heads, head_dim) at positions pos: pairs (2i, 2i + 1) turned by pos * freq_i."""
        t = pos[:, None, None] * self.freq
        a, b = x[..., 0::2], x[..., 1::2]
        return self.torch.stack((a * t.cos() - b * t.sin(), a * t.sin() + b * t.cos()), dim=-1).flatten(2)

    def step(self, tokens, batch, pos):
        """One pass: tokens (rows,) int64 at positions pos (rows,), the rows of `batch`.  Returns logits."""
        qmv, torch = self.qmv, self.torch
        n, h, kvh, d = tokens.numel(), self.heads, self.kv_heads, self.head_dim
        y, s = self.emb[tokens], torch.zeros((n, self.dim), device="cuda")
        for w in self.layers:
            xq = qmv.rmsnorm(y, w["n1"], residual=s, residual_out=s, out="q8")
            q = self.product(w["wq"], h * d, xq, n).view(n, h, d)
            k = self.product(w["wk"], kvh * d, xq, n).view(n, kvh, d)
            v = self.product(w["wv"], kvh * d, xq, n).view(n, kvh, d)
            qmv.kv_write(w["cache"], batch, self.rotate(k, pos), v)
            o = qmv.attend(w["cache"], batch, self.rotate(q, pos).bfloat16())
            y = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, self.dim, self.dim, w["wo"], o.view(n, self.dim))
            xq = qmv.rmsnorm(y, w["n2"], residual=s, residual_out=s, out="q8")
            gate_up = torch.empty((2, n, self.hidden), device="cuda")
            qmv.matvec_qx(qmv.Q4_0, qmv.SCALE_F16, self.hidden, self.dim, w["w1"], xq, n, y=gate_up[0])
            qmv.matvec_qx(qmv.Q4_0, qmv.SCALE_F16, self.hidden, self.dim, w["w3"], xq, n, y=gate_up[1])
            y = torch.empty((n, self.dim), device="cuda")
            qmv.matvec_grouped(qmv.Q4_0, qmv.SCALE_F16, [(self.dim, self.hidden, w["w2"], gate_up, y)], act="silu")
        x = qmv.rmsnorm(y, self.nf, residual=s, out="bf16")
        return qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, self.vocab, self.dim, self.cls, x)

    def prompt(self, tokens, table):
        """A whole prompt into empty caches.  Returns the logits of every position."""
        torch = self.torch
        n = tokens.numel()
        starts = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        length = torch.tensor([n], dtype=torch.int32, device="cuda")
        batch = self.qmv.KvBatch(table, length, starts=starts, rows=n, max_rows=n, max_len=n)
        return self.step(tokens, batch, torch.arange(n, device="cuda", dtype=torch.float32))


def run(layers=2, tokens=12, prompt=70, seed=0):
    """A prompt, then `tokens` greedy tokens.  Returns the tokens, the log probability that each had when it was
    chosen, and the same from one prompt pass over all of them."""
    import torch
    m = Model(layers=layers, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    table = torch.randperm(32, device="cuda", generator=g).to(torch.int32).view(1, 32)
    text = torch.randint(0, m.vocab, (prompt,), device="cuda", generator=g)
    logits = m.prompt(text, table)
    length = torch.tensor([prompt], dtype=torch.int32, device="cuda")
    batch = m.qmv.KvBatch(table, length, max_len=prompt + tokens)
    chosen, picked = [], []
    for _ in range(tokens):
        _, entropy, ids, best = m.qmv.logprobs(logits[-1:], top=4)
        chosen.append(ids[0, :1].long())
        picked.append(best[0, 0])
        length += 1
        logits = m.step(chosen[-1], batch, length.float() - 1)
    text = torch.cat([text, *chosen])
    whole = m.prompt(text, 31 - table)  # other pages, from the start
    given, _, _, _ = m.qmv.logprobs(whole[prompt - 1:-1], text[prompt:, None])
    assert m.qmv.last_error() == 0
    return text[prompt:].tolist(), torch.stack(picked).cpu().numpy(), given[:, 0].cpu().numpy()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=12)
    a = ap.parse_args()
    ids, picked, whole = run(a.layers, a.tokens)
    print("tokens                   ", ids)
    print("log p, token by token    ", np.round(picked, 3))
    print("log p, one prompt pass   ", np.round(whole, 3))


if __name__ == "__main__":
    main()
