"""The operators of a decode step run together: ids -> embed -> layers of norms, products, qk_rope, the cache, attention and
experts -> the classifier -> sample -> the next step's ids, eagerly and as one replayed graph."""
import os
import sys

import numpy as np
import pytest

import oracle
import step_ref

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def qmv():
    from block_quantized_weight_q4_gb300.build import build
    import block_quantized_weight_q4_gb300 as q
    build()
    q.load_library()
    yield q
    assert q.last_error() == 0


def _model(experts, **more):
    import decode_layer
    return decode_layer.Model(layers=2, dim=512, heads=8, kv_heads=2, hidden=256, vocab=1000, page_tokens=16, experts=experts, **more)


class Loop:
    """Two sequences, a token a step: every tensor of a step is written in place, so that it can be captured."""

    def __init__(self, qmv, m, seed):
        import torch
        self.qmv, self.m = qmv, m
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.ids = torch.tensor([3, 998], device="cuda")
        self.length = torch.zeros(2, dtype=torch.int32, device="cuda")
        table = torch.randperm(16, device="cuda", generator=g).to(torch.int32).view(2, 8)
        self.batch = qmv.KvBatch(table, self.length, max_len=128)
        self.noise = torch.empty((40, 2, m.vocab), device="cuda").exponential_(generator=g)
        self.how = {"temperature": torch.tensor([0.9, 1.2], device="cuda"), "top_p": torch.tensor([0.9, 1.0], device="cuda"),
                    "top_k": torch.tensor([0, 40], dtype=torch.int32, device="cuda"), "min_p": torch.tensor([0.0, 0.01], device="cuda")}
        self.now = self.noise[0].clone()

    def step(self):
        self.length += 1
        self.logits = self.m.step(self.ids, self.batch, self.length - 1)
        self.qmv.sample(self.logits, self.now, ids=self.ids, **self.how)

    def eager(self, steps):
        out = []
        for i in range(steps):
            self.now.copy_(self.noise[i])
            self.step()
            out.append(self.ids.tolist())
        return out


@pytest.mark.parametrize("experts", [0, 8])
def test_a_captured_step_gives_the_eager_ids(qmv, experts):
    import torch
    m = _model(experts)
    eager = Loop(qmv, m, 5).eager(40)
    loop = Loop(qmv, m, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # workspaces of the stream that is captured
        loop.step()
        loop.ids.copy_(torch.tensor([3, 998], device="cuda"))
        loop.length.zero_()
        for w in m.layers:
            w["cache"].k_scale.zero_()
            w["cache"].v_scale.zero_()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            loop.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    got = []
    for i in range(40):
        loop.now.copy_(loop.noise[i])
        graph.replay()
        got.append(loop.ids.tolist())
    assert got == eager
    assert len({tuple(t) for t in got}) > 20 and all(0 <= v < m.vocab for t in got for v in t)


def test_each_operator_of_a_step_against_its_formula(qmv):
    """The step's operators by hand on one layer, each result against the 64-bit formula of the tensors that it was given."""
    import torch
    m = _model(8)
    w, n, d = m.layers[0], 5, m.dim
    ids = torch.tensor([7, 999, 0, 7, -1], device="cuda")  # the same token twice, and a padded row
    y = qmv.embed(qmv.Q4_0, qmv.SCALE_F16, m.vocab, d, m.emb, ids, scale=d ** 0.5)
    table = oracle.dequant(m.emb.cpu().numpy(), qmv.Q4_0, qmv.SCALE_F16, m.vocab, d).reshape(m.vocab, d)
    want = np.where((ids.cpu().numpy() >= 0)[:, None], table[ids.cpu().numpy()] * F(d ** 0.5), F(0))
    assert np.array_equal(y.cpu().numpy(), want)
    s = torch.zeros_like(y)
    xq = qmv.rmsnorm(y, w["n1"], residual=s, residual_out=s, out="q8")
    q, k = m.product(w["wq"], 512, xq, n).view(n, 8, 64), m.product(w["wk"], 128, xq, n).view(n, 2, 64)
    v = m.product(w["wv"], 128, xq, n).view(n, 2, 64)
    pos = torch.tensor([0, 31, 2, 1 << 20, 4], dtype=torch.int32, device="cuda")
    qr, kr = qmv.qk_rope(q, k, pos, m.freq, w["qn"], w["kn"], pairs="neighbours", out="bf16")
    for x, r in ((q, qr), (k, kr)):
        want, mag = step_ref.qk_rope(x.cpu().numpy(), np.ones(64, F), 1e-6, pos.cpu().numpy(), m.freq.cpu().numpy(), False)
        # half a step of bfloat16, and 2^-19 of the pair for the norm's and the rotation's float32 steps
        assert np.all(np.abs(r.float().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * mag)
    length = torch.tensor([5], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    batch = qmv.KvBatch(torch.tensor([[9]], dtype=torch.int32, device="cuda"), length, starts=starts, rows=5, max_rows=5, max_len=5)
    qmv.kv_write(w["cache"], batch, kr, v.bfloat16())
    o = qmv.attend(w["cache"], batch, qr)
    y = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, d, d, w["wo"], o.view(n, d))
    x = qmv.rmsnorm(y, w["n2"], residual=s, residual_out=s, out="bf16")
    logits = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, 8, d, w["router"], x)
    out, who, shares = qmv.moe(w["moe"], x, logits, 2, routing=True)
    w1, w3 = (oracle.dequant(w[i].cpu().numpy(), qmv.Q4_0, qmv.SCALE_F16, 8 * 256, d).reshape(8, 256, d) for i in ("w1", "w3"))
    w2 = oracle.dequant(w["w2"].cpu().numpy(), qmv.Q4_0, qmv.SCALE_F16, 8 * d, 256).reshape(8, d, 256)
    want, bound, wi, ws, rel = step_ref.moe(w1, w3, w2, x.float().cpu().numpy(), logits.cpu().numpy(), 2, True, 1.0, "silu", 2)
    assert np.array_equal(who.cpu().numpy(), wi) and np.all(np.abs(shares.cpu().numpy() - ws) <= rel * ws)
    assert np.all(np.abs(out.cpu().numpy() - want) <= bound + 2.0 ** -22 * np.abs(want) + 1e-30)
    x = qmv.rmsnorm(out, m.nf, residual=s, out="bf16")
    logits = qmv.matvec(qmv.Q4_0, qmv.SCALE_F16, m.vocab, d, m.cls, x)
    noise = torch.empty_like(logits).exponential_()
    p = np.array([0.9, 1.0, 0.5, 0.99, 0.9], F)
    got = qmv.sample(logits, noise, top_p=torch.from_numpy(p).cuda()).cpu().numpy()
    for r in range(n):
        assert int(got[r]) in step_ref.sample(logits[r].cpu().numpy(), noise[r].cpu().numpy(), 1.0, 0, p[r], 0.0)
    lp, _, _, _ = qmv.logprobs(logits, torch.from_numpy(got).cuda()[:, None])
    assert torch.isfinite(lp).all()


@pytest.mark.parametrize("how", [{}, {"experts": 4}, {"temperature": 0.8, "top_k": 50, "top_p": 0.95}])
def test_the_example_runs(qmv, how):
    import decode_layer
    ids, picked, whole = decode_layer.run(layers=1, tokens=4, **how)
    assert len(ids) == 4 and np.isfinite(picked).all() and np.isfinite(whole).all()
