"""qmv_moe's results beside what their types hold: how often an output is another one than the rounded formula's."""
import numpy as np
import pytest

import step_ref
from helpers import dev_x
from test_gpu_moe import Layer, _check, _x

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


@pytest.mark.parametrize("sf", [0, 1])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("wt", [1, 2])
def test_bfloat16_outputs_are_rounded_once(qmv, wt, sf, bf16):
    """A bfloat16 output is the formula's, rounded, but where the formula's lies as close to the middle of two as the sums are off.
    Those are float32's, 2^-20 of the outputs' norm (16 roundings of 2^-24 of values up to twice the result, of gate, up and down), and
    for Q4_0 the tensor core's products of levels as bits, 2^-18 each of gate, up and down, by chance of sign: below 2^-17 together.
    An error of E root mean square changes an output whose bfloat16 neighbours are u apart with probability 0.8 E / u at most."""
    import torch
    tokens, dim, hidden = 12, 1024, 512
    layer = Layer(qmv, wt, wt, sf, 8, dim, hidden, seed=61)
    rng = np.random.default_rng(62)
    x, xd = _x(rng, tokens, dim, bf16)
    logits = rng.standard_normal((tokens, 8)).astype(F)
    y = qmv.moe(layer.dev, xd, dev_x(logits), 3, out="bf16").double().cpu().numpy()
    want = step_ref.moe(layer.w1, layer.w3, layer.w2, x, logits, 3, True, 1.0, "silu", 2)[0]
    near = torch.from_numpy(want).bfloat16().double().numpy()
    e = (2.0 ** -17 if wt == 2 else 2.0 ** -20) * np.sqrt((want ** 2).mean(axis=1, keepdims=True))
    gap = 2.0 ** (np.floor(np.log2(np.abs(want))) - 7)
    most = np.minimum(1, 0.8 * e / gap).sum()
    assert (y != near).sum() <= most + 6 * np.sqrt(most) + 3


def _scaled(qmv, wt, experts, dim, hidden, seed, *by):
    """A layer of float32 scales whose W1, W3 and W2 are those of make_matrix times 2^by."""
    import torch
    layer = Layer(qmv, wt, wt, 0, experts, dim, hidden, seed=seed)
    images = []
    for name, W, b, rows, cols in (("w1", layer.dev.W1, by[0], hidden, dim), ("w3", layer.dev.W3, by[1], hidden, dim), ("w2", layer.dev.W2, by[2], dim, hidden)):
        off = qmv.scale_offset(wt, 0, experts * rows, cols)
        W = W.clone()
        d = W[off:off + experts * rows * cols // 8].view(torch.float32) * 2.0 ** b
        assert d.isfinite().all() and ((d == 0) | (d.abs() >= 2.0 ** -126)).all()  # (else they would be rounded)
        W[off:off + experts * rows * cols // 8] = d.view(torch.uint8)
        images.append(W)
        setattr(layer, name, getattr(layer, name).astype(np.float64) * 2.0 ** b)
    layer.dev = qmv.Moe(wt, wt, 0, experts, dim, hidden, *images)
    return layer


@pytest.mark.parametrize("wt", [1, 2])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("amp,by,act", [
    (119, (-112, -113, 0), "silu"),   # x at the top of the range
    (124, (-114, -115, -8), "gelu"),
    (60, (0, 0, -114), "silu"),       # act(gate) * up there: 2^123 at most for Q4_0, but 2^131, past the range, for Q8_0
    (56, (0, 0, -112), "silu"),
    (-120, (96, 96, 47), "gelu"),     # x at the bottom
    (-130, (94, 92, 76), "silu"),     # (subnormal numbers)
    (-58, (0, 0, 99), "silu"),        # act(gate) * up there
])
def test_ends_of_the_range(qmv, wt, bf16, out, amp, by, act):
    """Finite results stay what the formula says where activations or act(gate) * up come near float32's ends.  Float32 outputs: 2^-20 of
    their norm, as sums of 16 roundings of gate, up and down by chance of sign.  bfloat16 ones: 2^-8 of each for its rounding, and 2^-17 of the norm before it."""
    tokens, dim, hidden = 5, 512, 256
    layer = _scaled(qmv, wt, 4, dim, hidden, 71, *by)
    rng = np.random.default_rng(72)
    x, xd = _x(rng, tokens, dim, bf16, 2.0 ** amp)
    logits = rng.standard_normal((tokens, 4)).astype(F)
    y = qmv.moe(layer.dev, xd, dev_x(logits), 2, act=act, out=out).double().cpu().numpy()
    want = step_ref.moe(layer.w1, layer.w3, layer.w2, x, logits, 2, True, 1.0, act, 2)[0]
    norm = np.linalg.norm(want)
    if amp == 60 and wt == 1:
        assert not np.isfinite(y).all()
        return
    assert np.isfinite(norm) and norm > 1e-30 and np.isfinite(y).all()
    assert np.linalg.norm(y - want) <= (2.0 ** -20 if out == "f32" else 2.0 ** -8 + 2.0 ** -17) * norm


def test_blocks_of_both_ends(qmv):
    """One token's blocks of 32 from 2^-140 to 2^120: each at a power of two of its own."""
    layer = _scaled(qmv, 2, 1, 512, 64, 73, -100, -100, 60)
    rng = np.random.default_rng(74)
    amps = np.repeat(2.0 ** np.linspace(-140, 120, 16), 32)
    for only in (None, 15):  # all blocks, the largest alone
        x = (rng.standard_normal((2, 512)) * amps).astype(F)
        if only is not None:
            x[:, :32 * only] = 0
        for out in ("f32", "bf16"):
            y = qmv.moe(layer.dev, dev_x(x), dev_x(np.zeros((2, 1), F)), 1, out=out).double().cpu().numpy()
            want = step_ref.moe(layer.w1, layer.w3, layer.w2, x, np.zeros((2, 1), F), 1, True, 1.0, "silu", 2)[0]
            assert np.isfinite(want).all()
            assert np.linalg.norm(y - want) <= (2.0 ** -20 if out == "f32" else 2.0 ** -8 + 2.0 ** -17) * np.linalg.norm(want)


def test_a_layer_does_not_grow(qmv):
    """Calls of many counts of tokens leave nothing behind in the layer."""
    import torch
    layer = Layer(qmv, 2, 2, 1, 4, 64, 64, seed=81).dev

    def held():
        return sum(len(v) for v in vars(layer).values() if isinstance(v, (dict, list, tuple, set)))

    def call(n, top, out):
        return qmv.moe(layer, torch.ones((n, 64), device="cuda"), torch.zeros((n, 4), device="cuda"), top, out=out)

    call(1, 1, "f32")
    before = held()
    for n in range(1, 70):
        call(n, 1 + n % 4, "bf16" if n % 3 else "f32")
    assert held() == before
    assert torch.equal(call(66, 2, "f32"), call(66, 2, "f32"))


@pytest.mark.parametrize("wt,sf", [(1, 0), (1, 1), (2, 0), (2, 1)])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("tokens,experts,top,dim,hidden", [
    (48, 256, 16, 64, 64), (49, 256, 16, 64, 64), (48, 3, 3, 128, 320), (47, 12, 2, 192, 64), (3, 2, 2, 320, 128), (112, 4, 2, 64, 128), (113, 2, 1, 64, 64),
    (31, 16, 1, 64, 64), (33, 16, 1, 64, 64), (48, 5, 3, 2112, 64), (40, 4, 2, 64, 2112)])
def test_units_and_blocks(qmv, wt, sf, out, tokens, experts, top, dim, hidden):
    """Units of 2 and of 4 tokens on both sides of what chooses them, with the most tokens and places that they take, and blocks of both sizes."""
    rng = np.random.default_rng([tokens, experts, dim])
    layer = Layer(qmv, wt, wt, sf, experts, dim, hidden, seed=83)
    x, xd = _x(rng, tokens, dim, out == "bf16")
    logits = rng.standard_normal((tokens, experts)).astype(F)
    _check(layer, qmv.moe(layer.dev, xd, dev_x(logits), top, out=out, routing=True), x, logits, top, True, 1.0, "silu", out == "bf16")
