"""qmv_embed: rows of a quantized table, bit for bit."""
import numpy as np
import pytest

import oracle
from block_quantized_weight_q4_gb300 import inputs

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


def _bf16(x):
    import torch
    return torch.from_numpy(x).bfloat16().float().numpy()


@pytest.mark.parametrize("wt", [1, 2])
@pytest.mark.parametrize("sf", [0, 1])
@pytest.mark.parametrize("vocab,cols,rows", [(1, 32, 1), (5, 32, 9), (7, 96, 3), (100, 1024, 1), (33, 4096, 70), (1000, 352, 257)])
def test_rows(qmv, wt, sf, vocab, cols, rows):
    import torch
    m = inputs.make_matrix(wt, sf, vocab, cols, seed=vocab + cols)
    table = oracle.dequant(m.W, wt, sf, vocab, cols)
    W = torch.from_numpy(m.W).cuda()
    rng = np.random.default_rng(rows)
    ids = rng.integers(0, vocab, rows)
    ids[0], ids[-1] = vocab - 1, 0
    dev = torch.from_numpy(ids).cuda()
    for scale in (1.0, 32.0, float(F(cols) ** F(0.5)), 0.0, -1.5):
        want = (table[ids] * F(scale)).astype(F)
        got = qmv.embed(wt, sf, vocab, cols, W, dev, scale=scale)
        assert np.array_equal(got.cpu().numpy().view(np.uint32), want.view(np.uint32))
        got = qmv.embed(wt, sf, vocab, cols, W, dev, scale=scale, out="bf16")
        assert np.array_equal(got.float().cpu().numpy(), _bf16(want))


def test_ids_outside_and_shapes(qmv):
    import torch
    m = inputs.make_matrix(2, 1, 50, 64, seed=1)
    W = torch.from_numpy(m.W).cuda()
    table = oracle.dequant(m.W, 2, 1, 50, 64)
    ids = torch.tensor([[3, -1, 50], [2 ** 62, 49, -2 ** 63]], device="cuda")
    y = torch.full((2, 3, 64), 9.0, device="cuda")
    got = qmv.embed(2, 1, 50, 64, W, ids, y=y)
    assert got.data_ptr() == y.data_ptr()
    want = np.zeros((2, 3, 64), F)
    want[0, 0], want[1, 1] = table[3], table[49]
    assert np.array_equal(y.cpu().numpy(), want)
    none = qmv.embed(2, 1, 50, 64, W, torch.empty(0, dtype=torch.int64, device="cuda"))
    assert none.shape == (0, 64)
    for bad in (dict(ids=ids.int()), dict(W=W[:-1]), dict(out="q8"), dict(y=y[:1]), dict(y=y.bfloat16()), dict(ids=ids.cpu())):
        with pytest.raises(ValueError):
            qmv.embed(**{**dict(wtype=2, scale_dtype=1, vocab=50, cols=64, W=W, ids=ids), **bad})


def test_offsets_past_32_bits(qmv):
    """A table of more than 2^32 bytes: rows at its end."""
    import torch
    vocab, cols = 2 ** 20 + 5, 4096
    size = qmv.weight_bytes(1, 0, vocab, cols)
    W = torch.zeros(size, dtype=torch.uint8, device="cuda")
    off = qmv.scale_offset(1, 0, vocab, cols)
    ids = torch.tensor([vocab - 1, 2 ** 20 + 1], device="cuda")
    for i, r in enumerate(ids.tolist()):
        W[r * cols:(r + 1) * cols] = torch.arange(cols, device="cuda").remainder(100).to(torch.uint8) + i
        W[off + r * cols // 8: off + (r + 1) * cols // 8].view(torch.float32).fill_(0.5)
    got = qmv.embed(1, 0, vocab, cols, W, ids)
    want = torch.arange(cols, device="cuda").remainder(100).float() * 0.5
    assert torch.equal(got[0], want) and torch.equal(got[1], want + 0.5)


def test_graph_reads_ids_when_it_runs(qmv):
    import torch
    m = inputs.make_matrix(1, 1, 64, 256, seed=2)
    W, ids = torch.from_numpy(m.W).cuda(), torch.arange(4, device="cuda")
    table = torch.from_numpy(oracle.dequant(m.W, 1, 1, 64, 256)).cuda()
    y = qmv.embed(1, 1, 64, 256, W, ids)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qmv.embed(1, 1, 64, 256, W, ids, y=y)
    ids.add_(60)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, table[60:])
