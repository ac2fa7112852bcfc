"""qmv_moe's results beside what their types hold: how often an output is another one than the rounded formula's."""
import numpy as np
import pytest

import step_ref
from helpers import dev_x
from test_gpu_moe import Layer, _x

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
