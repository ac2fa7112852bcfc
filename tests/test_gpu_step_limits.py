"""sample, embed, qk_rope and moe at the far ends of what their documentation allows: long rows, offsets past 32 bits, calls at
once, padded and extreme tokens."""
import numpy as np
import pytest

import oracle
import step_ref
from block_quantized_weight_q4_gb300 import inputs
from helpers import dev_x
from test_gpu_moe import Layer, _check as check_moe, _x
from test_gpu_sample import _logits, _settings

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def qmv():
    import torch
    from block_quantized_weight_q4_gb300.build import build
    import block_quantized_weight_q4_gb300 as q
    assert torch.cuda.is_available()
    build()
    q.load_library()
    yield q
    assert q.last_error() == 0


def _cuda(a):
    import torch
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


@pytest.mark.parametrize("vocab", [262145, 300001, 1000003])
@pytest.mark.parametrize("kind", ["flat", "sharp", "near", "equal"])
@pytest.mark.parametrize("cuts", ["all", "p", "free"])
def test_sample_long_rows(qmv, vocab, kind, cuts):
    """Rows of more chunks than the chunk maxima have places: longer chunks."""
    rng = np.random.default_rng([vocab, len(kind), len(cuts)])
    rows = 2
    x, e = _logits(rng, rows, vocab, kind), rng.exponential(size=(rows, vocab)).astype(F)
    s = _settings(rng, rows, cuts)
    got = qmv.sample(_cuda(x), _cuda(e), *[_cuda(a) for a in s]).cpu().numpy()
    for r in range(rows):
        t, k, p, m = (d if a is None else a[r] for a, d in zip(s, (1.0, 0, 1.0, 0.0)))
        assert int(got[r]) in step_ref.sample(x[r], e[r], t, k, p, m), (r, got[r])


def test_sample_rows_far_apart(qmv):
    """Rows 2^31 bytes and more apart, at every start of a 16-byte piece; the noise the logits' own tensor."""
    import torch
    vocab, stride = 5001, (1 << 30) + 1
    base = torch.empty(2 * stride + vocab, device="cuda")
    rng = np.random.default_rng(3)
    x = np.abs(_logits(rng, 3, vocab - 1, "flat"))
    x[np.isinf(x)] = 0.25
    x = np.concatenate([x, np.full((3, 1), 0.5, F)], axis=1)
    for r in range(3):
        base[r * stride:r * stride + vocab] = _cuda(x[r])
    view = base.as_strided((3, vocab), (stride, 1))
    p = np.array([0.9, 0.5, 1.0], F)
    got = qmv.sample(view, view, top_p=_cuda(p)).cpu().numpy()
    for r in range(3):
        assert int(got[r]) in step_ref.sample(x[r], x[r], 1.0, 0, p[r], 0.0)


def test_rope_rows_far_apart_and_many(qmv):
    import torch
    stride = (1 << 30) + 64
    base = torch.empty(2 * stride + 256, dtype=torch.bfloat16, device="cuda")
    view = base.as_strided((3, 2, 128), (stride, 128, 1))
    x = torch.randn((3, 2, 128), device="cuda").bfloat16()
    view.copy_(x)
    pos = torch.tensor([5, -7, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    freq = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float32) / 64)
    want = qmv.qk_rope(x, None, pos, freq)[0]
    assert torch.equal(qmv.qk_rope(view, None, pos, freq)[0], want)
    qmv.qk_rope(view, None, pos, freq, q_out=view)
    assert torch.equal(view, want)
    del base, view
    x = torch.randn((70001, 1, 64), device="cuda")
    pos = torch.arange(70001, dtype=torch.int32, device="cuda")
    w = torch.randn(64, device="cuda")
    got = qmv.qk_rope(x, None, pos, freq[:32].contiguous(), q_weight=w)[0].cpu().numpy()
    at = np.array([0, 1, 7, 8, 65535, 65536, 69999, 70000])
    want, mag = step_ref.qk_rope(x.cpu().numpy()[at], w.cpu().numpy(), 1e-6, at, freq[:32].cpu().numpy(), True)
    assert np.all(np.abs(got[at] - want) <= 2.0 ** -19 * mag)
    some = torch.from_numpy(at).cuda()  # every row as in a call of its own
    again = qmv.qk_rope(x[some], None, pos[some], freq[:32].contiguous(), q_weight=w)[0].cpu().numpy()
    assert np.array_equal(got[at], again)


def test_moe_weights_past_32_bits(qmv):
    """Matrices of more than 2^32 bytes, of which only some experts' rows hold anything but zeros."""
    import torch
    experts, dim, hidden = 256, 4096, 4352
    total = [torch.zeros(qmv.weight_bytes(1, 1, experts * r, c), dtype=torch.uint8, device="cuda") for r, c in ((hidden, dim), (hidden, dim), (dim, hidden))]
    some = Layer(qmv, 1, 1, 1, 1, dim, hidden, seed=31)
    for W, part, (r, c) in zip(total, (some.dev.W1, some.dev.W3, some.dev.W2), ((hidden, dim), (hidden, dim), (dim, hidden))):
        off, part_off, n = qmv.scale_offset(1, 1, experts * r, c), qmv.scale_offset(1, 1, r, c), r * c
        W[255 * n:256 * n] = part[:n]
        W[off + 255 * n // 16:off + 256 * n // 16] = part[part_off:part_off + n // 16]
    layer = qmv.Moe(1, 1, 1, experts, dim, hidden, *total)
    rng = np.random.default_rng(32)
    x, xd = _x(rng, 3, dim, True)
    logits = np.full((3, experts), -5, F)
    logits[:, 255], logits[1, 254] = 1.0, 4.0
    out, ids, _ = qmv.moe(layer, xd, dev_x(logits), 1, routing=True)
    assert ids[:, 0].tolist() == [255, 254, 255]
    # (the sums' order follows from the sizes and the routing, so the small layer's own call may differ in its last bits: the bound, then)
    want, bound, _, _, _ = step_ref.moe(some.w1, some.w3, some.w2, x, np.zeros((3, 1), F), 1, True, 1.0, "silu", 2)
    err = np.abs(out.cpu().numpy() - want)
    assert np.all(err[[0, 2]] <= (bound + 2.0 ** -22 * np.abs(want) + 1e-30)[[0, 2]]) and not out[1].any()


@pytest.mark.parametrize("wt,sf,bf16,out", [(2, 0, False, "f32"), (2, 0, True, "bf16"), (1, 0, False, "f32"), (2, 1, False, "bf16")])
@pytest.mark.parametrize("tokens,dim,hidden", [(5, 16448, 64), (4, 64, 16448), (3, 8256, 4160)])
def test_moe_long_sides(qmv, wt, sf, bf16, out, tokens, dim, hidden):
    """Columns that do not stay in shared memory, units of fewer tokens, many chunks a warp."""
    rng = np.random.default_rng([dim, wt, sf])
    layer = Layer(qmv, wt, wt, sf, 2, dim, hidden, seed=33)
    x, xd = _x(rng, tokens, dim, bf16, 0.3)
    logits = rng.standard_normal((tokens, 2)).astype(F)
    got = qmv.moe(layer.dev, xd, dev_x(logits), 1, act="gelu", out=out, routing=True)
    check_moe(layer, got, x, logits, 1, True, 1.0, "gelu", out == "bf16")


@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_moe_tokens_of_one_expert(qmv, out):
    rng = np.random.default_rng(34)
    layer = Layer(qmv, 2, 2, 1, 5, 192, 128, seed=35)
    for tokens in (63, 64, 65, 129):
        x, xd = _x(rng, tokens, 192, True)
        logits = np.zeros((tokens, 5), F)
        logits[:, 3] = 2
        got = qmv.moe(layer.dev, xd, dev_x(logits), 1, out=out, routing=True)
        check_moe(layer, got, x, logits, 1, True, 1.0, "silu", out == "bf16")


def test_moe_extreme_tokens_keep_to_themselves(qmv):
    """Padded tokens (zeros), NaN, infinities and values at the types' ends: the other tokens' bits do not change."""
    import torch
    layer = Layer(qmv, 2, 2, 1, 4, 256, 128, seed=36)
    x = torch.randn((9, 256), device="cuda")
    logits = torch.randn((9, 4), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        for out in ("f32", "bf16"):
            plain = qmv.moe(layer.dev, x.to(dtype), logits, 2, out=out)
            y = x.clone()
            y[1], y[3, 7], y[4, 200], y[6, :100], y[8] = 0, np.nan, np.inf, 3e38, 1e-40
            got = qmv.moe(layer.dev, y.to(dtype), logits, 2, out=out)
            for t in (0, 2, 5, 7):
                assert torch.equal(got[t], plain[t])
            assert not got[1].any() and got[3].isnan().all() and torch.isfinite(got[8].float()).all()


def test_calls_at_once(qmv):
    """Every operator on three streams at once, each with its own tensors."""
    import torch
    m = inputs.make_matrix(2, 1, 500, 256, seed=3)
    W = torch.from_numpy(m.W).cuda()
    layer = Layer(qmv, 2, 2, 1, 6, 256, 128, seed=37)
    freq = torch.rand(32, device="cuda")
    ids = [torch.randint(0, 500, (40,), device="cuda") for _ in range(3)]
    gates = [torch.randn((40, 6), device="cuda") for _ in range(3)]
    logits = [torch.randn((40, 30000), device="cuda") for _ in range(3)]
    noise = [torch.empty_like(t).exponential_() for t in logits]
    p = torch.full((40,), 0.95, device="cuda")
    k = torch.full((40,), 100, dtype=torch.int32, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")

    def run(i):
        x = qmv.embed(2, 1, 500, 256, W, ids[i])
        q, _ = qmv.qk_rope(x.view(40, 4, 64), None, pos, freq)
        y = qmv.moe(layer.dev, q.view(40, 256), gates[i], 2)
        return x, q, y, qmv.sample(logits[i], noise[i], top_k=k, top_p=p), qmv.sample(logits[i], noise[i])

    want = [run(i) for i in range(3)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [[] for _ in range(3)]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(run(i))
    torch.cuda.synchronize()
    for i in range(3):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_embed_more_than_2_31_values(qmv):
    import torch
    m = inputs.make_matrix(2, 1, 300, 4096, seed=4)
    W = torch.from_numpy(m.W).cuda()
    n = 2 ** 19 + 70
    ids = torch.arange(n, device="cuda") % 301  # 300 is outside
    y = qmv.embed(2, 1, 300, 4096, W, ids, out="bf16")
    table = torch.from_numpy(oracle.dequant(m.W, 2, 1, 300, 4096)).cuda().bfloat16()
    table = torch.cat([table, torch.zeros_like(table[:1])])
    for at in (0, 299, 2 ** 19 - 1, n - 40):
        assert torch.equal(y[at:at + 40], table[ids[at:at + 40]])


def test_embed_more_than_2_31_pieces(qmv):
    """An output of more than 2^31 pieces of 16 bytes: launches over parts of the rows."""
    import torch
    m = inputs.make_matrix(1, 0, 50, 32, seed=5)
    W = torch.from_numpy(m.W).cuda()
    n = 2 ** 29 + 1000
    ids = torch.arange(n, device="cuda").remainder_(51)
    y = qmv.embed(1, 0, 50, 32, W, ids, out="bf16")
    table = torch.from_numpy(oracle.dequant(m.W, 1, 0, 50, 32)).cuda().bfloat16()
    table = torch.cat([table, torch.zeros_like(table[:1])])
    for at in (0, 2 ** 28 - 50, 2 ** 29 - 400, 2 ** 29 - 200, n - 100):
        assert torch.equal(y[at:at + 100], table[ids[at:at + 100]])
    del y, ids
    torch.cuda.empty_cache()


def test_sample_2_30_ids(qmv):
    """A row of more than 2^30 ids: a few stand out, at its ends and at the borders of whole pieces."""
    import torch
    n = 2 ** 30 + 5
    x = torch.full((1, n), -20.0, device="cuda")
    e = torch.ones((1, n), device="cuda")
    at = torch.tensor([n - 1, 0, 2 ** 30 - 1, 2 ** 30, 77777777], device="cuda")
    x[0, at] = torch.tensor([1.0, 0.5, 0.75, 0.25, 0.0], device="cuda")

    def one(**how):
        types = {"top_k": torch.int32}
        return qmv.sample(x, e, **{k: torch.tensor([v], dtype=types.get(k, torch.float32), device="cuda") for k, v in how.items()}).item()

    assert one(temperature=0.0) == n - 1 and one() == n - 1
    e[0, 2 ** 30] = 1e-3  # 0.25 + 6.9: ahead of the others, where it is kept
    assert one() == 2 ** 30 and one(top_k=4) == 2 ** 30 and one(top_k=3) == n - 1 and one(min_p=0.4) == 2 ** 30 and one(min_p=0.5) == n - 1
    e[0, n - 3] = 1e-15  # -20 + 34.5: ahead of all, where nothing is cut off
    assert one() == n - 3 and one(temperature=2.0) == n - 3
    assert one(top_k=1000) == 2 ** 30  # of equal logits the lowest ids are kept
    assert one(min_p=0.1) == 2 ** 30 and one(top_k=5, min_p=0.4) == 2 ** 30
    x[0, 12345] = float("nan")
    assert one() == -1 and one(top_k=5) == -1
    del x, e
    torch.cuda.empty_cache()
