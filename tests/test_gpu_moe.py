"""qmv_moe against 64 bits: sizes, types, routings with ties and masks, blocks of tokens, streams and graphs."""
import numpy as np
import pytest

import oracle
import step_ref
from block_quantized_weight_q4_gb300 import inputs
from helpers import dev_x

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


class Layer:
    def __init__(self, qmv, wt13, wt2, sf, experts, dim, hidden, seed):
        import torch
        self.args = (wt13, wt2, sf, experts, dim, hidden)
        ms = [inputs.make_matrix(wt13, sf, experts * hidden, dim, seed=seed), inputs.make_matrix(wt13, sf, experts * hidden, dim, seed=seed + 1),
              inputs.make_matrix(wt2, sf, experts * dim, hidden, seed=seed + 2)]
        self.w1, self.w3 = (oracle.dequant(m.W, wt13, sf, experts * hidden, dim).reshape(experts, hidden, dim) for m in ms[:2])
        self.w2 = oracle.dequant(ms[2].W, wt2, sf, experts * dim, hidden).reshape(experts, dim, hidden)
        self.dev = qmv.Moe(*self.args, *[torch.from_numpy(m.W).cuda() for m in ms])


def _x(rng, tokens, dim, bf16, amp=1.0):
    # products of about unit size: the weights of make_matrix are a few hundredths
    x = (amp * rng.standard_normal((tokens, dim))).astype(F)
    if bf16:
        code = (x.view(np.uint32) >> 16).astype(np.uint16)
        return (code.astype(np.uint32) << 16).view(F), dev_x(code)
    return x, dev_x(x)


def _check(layer, got, x, logits, top, renorm, scale, act, bf16_out):
    y, ids, shares = got
    want, bound, wi, ws, rel = step_ref.moe(layer.w1, layer.w3, layer.w2, x, logits, top, renorm, scale, act, 1 if bf16_out else 2)
    assert np.array_equal(ids.cpu().numpy(), wi)
    s = shares.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(s), np.isnan(ws)) and np.all((np.abs(s - ws) <= rel * ws + 1e-38) | np.isnan(ws))
    y = y.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(y), np.isnan(want))
    live = ~np.isnan(want)
    bound = bound + (2.0 ** -8 * np.abs(want) if bf16_out else 2.0 ** -22 * np.abs(want)) + 1e-30
    err = np.abs(y - want)
    assert np.all(err[live] <= bound[live]), float(np.max(err[live] / bound[live]))


@pytest.mark.parametrize("tokens,experts,top,dim,hidden", [
    (1, 1, 1, 64, 64), (1, 4, 2, 256, 128), (2, 5, 5, 128, 192), (3, 32, 4, 1024, 64), (5, 8, 2, 320, 256), (8, 2, 1, 512, 320), (9, 3, 2, 192, 448),
    (17, 16, 8, 256, 64), (33, 7, 3, 448, 128), (64, 4, 2, 128, 256), (65, 6, 2, 64, 64), (150, 3, 3, 64, 128), (2, 256, 16, 64, 64), (64, 256, 16, 64, 64),
    (1, 2, 2, 2112, 1088)])
@pytest.mark.parametrize("wt,sf,bf16,out", [(2, 1, True, "f32"), (2, 1, True, "bf16"), (2, 0, False, "f32"), (1, 0, True, "bf16"), (1, 1, False, "bf16"),
                                            (1, 0, False, "f32")])
def test_sizes_and_types(qmv, tokens, experts, top, dim, hidden, wt, sf, bf16, out):
    import torch
    rng = np.random.default_rng(tokens * 7 + experts + dim)
    layer = Layer(qmv, wt, wt, sf, experts, dim, hidden, seed=experts)
    x, xd = _x(rng, tokens, dim, bf16)
    logits = (1.5 * rng.standard_normal((tokens, experts))).astype(F)
    renorm, act = bool(tokens & 1), "silu" if hidden % 128 == 0 else "gelu"
    got = qmv.moe(layer.dev, xd, torch.from_numpy(logits).cuda(), top, renorm=renorm, scale=1.5, act=act, out=out, routing=True)
    _check(layer, got, x, logits, top, renorm, 1.5, act, out == "bf16")


@pytest.mark.parametrize("wt13,wt2", [(2, 1), (1, 2)])
def test_mixed_files(qmv, wt13, wt2):
    import torch
    rng = np.random.default_rng(2)
    layer = Layer(qmv, wt13, wt2, 1, 6, 256, 192, seed=3)
    x, xd = _x(rng, 4, 256, True)
    logits = rng.standard_normal((4, 6)).astype(F)
    got = qmv.moe(layer.dev, xd, torch.from_numpy(logits).cuda(), 2, routing=True)
    _check(layer, got, x, logits, 2, True, 1.0, "silu", False)


@pytest.mark.parametrize("renorm", [True, False])
def test_routing(qmv, renorm):
    """Equal logits, masked experts, tokens without experts, NaN and infinity, all tokens with one expert."""
    import torch
    rng = np.random.default_rng(8)
    layer = Layer(qmv, 2, 2, 1, 40, 128, 64, seed=9)
    tokens = 20
    x, xd = _x(rng, tokens, 128, True)
    logits = rng.standard_normal((tokens, 40)).astype(F)
    logits[0] = 0.0
    logits[1] = np.round(logits[1])
    logits[2, 5:] = -np.inf
    logits[2, :3] = -np.inf  # two are left
    logits[3] = -np.inf
    logits[4, 7] = np.nan
    logits[5, 7] = np.inf
    logits[6] = np.finfo(F).min
    logits[7] *= 100
    logits[8, ::2] = 0.0
    logits[8, 1::2] = -0.0
    logits[9:, 33] = 50.0  # an expert that eleven tokens use
    got = qmv.moe(layer.dev, xd, torch.from_numpy(logits).cuda(), 6, renorm=renorm, routing=True)
    _check(layer, got, x, logits, 6, renorm, 1.0, "silu", False)
    assert not got[0][3].any()


def test_a_token_does_not_depend_on_timing(qmv):
    import torch
    rng = np.random.default_rng(12)
    layer = Layer(qmv, 2, 2, 1, 8, 1024, 512, seed=5)
    x, xd = _x(rng, 40, 1024, True)
    logits = torch.from_numpy(rng.standard_normal((40, 8)).astype(F)).cuda()
    first = qmv.moe(layer.dev, xd, logits, 2)
    for _ in range(20):
        assert torch.equal(first, qmv.moe(layer.dev, xd, logits, 2))


def test_strides_streams_and_graphs(qmv):
    import torch
    rng = np.random.default_rng(13)
    layer = Layer(qmv, 2, 2, 1, 8, 512, 256, seed=6)
    x, xd = _x(rng, 5, 512, True)
    wide = torch.from_numpy(rng.standard_normal((5, 13)).astype(F)).cuda()
    logits = wide[:, 2:10]
    a = qmv.moe(layer.dev, xd, logits, 3)
    assert torch.equal(a, qmv.moe(layer.dev, xd, logits.contiguous(), 3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = qmv.moe(layer.dev, xd, logits, 3, stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    # two graphs with scratch memory of their own, replayed at once on two streams; the routing is read when they run
    ys, graphs, keep = [], [], []
    for _ in range(2):
        y, scratch = torch.zeros_like(a), torch.empty(qmv.moe_scratch_bytes(5, 3, 256), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmv.moe(layer.dev, xd, logits, 3, y=y, scratch=scratch)
        ys.append(y), graphs.append(g), keep.append(scratch)
    wide.copy_(torch.from_numpy(rng.standard_normal((5, 13)).astype(F)))
    torch.cuda.synchronize()
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    want = qmv.moe(layer.dev, xd, logits, 3)
    assert torch.equal(ys[0], want) and torch.equal(ys[1], want) and not torch.equal(want, a)


def test_nothing_to_do_and_refusals(qmv):
    import torch
    layer = Layer(qmv, 2, 2, 1, 4, 64, 64, seed=1)
    x, logits = torch.zeros((2, 64), device="cuda"), torch.zeros((2, 4), device="cuda")
    assert qmv.moe(layer.dev, x[:0], logits[:0], 2).shape == (0, 64)
    for bad in (dict(x=x[:, :32]), dict(x=x[:1]), dict(logits=logits.double()), dict(act="relu"), dict(out="q8"),
                dict(scratch=torch.empty(16, dtype=torch.uint8, device="cuda")), dict(y=x.bfloat16()), dict(logits=logits.cpu())):
        with pytest.raises(ValueError):
            qmv.moe(**{**dict(layer=layer.dev, x=x, logits=logits, top=2), **bad})
    with pytest.raises(TypeError):
        qmv.moe(layer.dev, x.half(), logits, 2)
    for top in (0, 5):
        with pytest.raises(qmv.QmvError):
            qmv.moe(layer.dev, x, logits, top)
    with pytest.raises(ValueError):
        qmv.Moe(2, 2, 1, 4, 64, 128, layer.dev.W1, layer.dev.W3, layer.dev.W2)


@pytest.mark.parametrize("sf", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("wt", [0, 1])
def test_float32_outputs_are_float32(qmv, wt, sf, bf16):
    """Float32 outputs hold the accuracy of float32 sums, for either type of x: about 16 roundings of 2^-24 (8 steps of a block on the tensor
    core, the warps' and blocks' sums) of values up to twice the result, each of gate, up and down: sqrt(3) sqrt(16) 2 2^-24 = 2^-20.2 of
    the output's norm, where the errors' signs are by chance."""
    wt = (qmv.Q4_0, qmv.Q8_0)[wt]
    layer = Layer(qmv, wt, wt, sf, 8, 1024, 512, seed=91)
    rng = np.random.default_rng(92)
    x, xd = _x(rng, 5, 1024, bf16)
    logits = rng.standard_normal((5, 8)).astype(F)
    y = qmv.moe(layer.dev, xd, dev_x(logits), 3).cpu().numpy().astype(np.float64)
    want, _, _, _, _ = step_ref.moe(layer.w1, layer.w3, layer.w2, x, logits, 3, True, 1.0, "silu", 2)
    assert np.linalg.norm(y - want) <= 2.0 ** -20 * np.linalg.norm(want)
