"""qmv_qk_rope against 64 bits: norms, both pairings, partial rotation, far positions, strides, updates in place."""
import numpy as np
import pytest

import step_ref
from helpers import dev_x

pytestmark = pytest.mark.gpu
F = np.float32
# cos and sin of an angle rounded to 2^-25 half turns (2^-23.3 radians), their own 2 ulp, the factor's product, two products and a sum:
# at most 16 units of 2^-24 of |a| + |b|.  The norm: squares' chain of 8 and 5 steps, mean, root, two products: 16 more.
TURN, NORM = 16 * 2.0 ** -24, 16 * 2.0 ** -24


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


def _make(rng, rows, heads, dim, bf16):
    x = (1.5 * rng.standard_normal((rows, heads, dim))).astype(F)
    if bf16:
        code = (x.view(np.uint32) >> 16).astype(np.uint16)
        return (code.astype(np.uint32) << 16).view(F), dev_x(code)
    return x, dev_x(x)


def _check(got, want, mag, normed, bf16_out):
    got = got.float().cpu().numpy().astype(np.float64)
    bound = (TURN + (NORM if normed else 0)) * mag + (2.0 ** -8 * np.abs(want) if bf16_out else 0) + 1e-37
    assert np.all(np.abs(got - want) <= bound), float(np.max(np.abs(got - want) / bound))


@pytest.mark.parametrize("rows,heads,kv_heads,dim,rot", [(1, 32, 8, 128, 128), (3, 5, 5, 64, 64), (17, 14, 2, 64, 32), (2, 8, 1, 256, 256),
                                                         (5, 1, 1, 256, 16), (260, 4, 2, 128, 64), (2, 130, 3, 128, 128), (1, 1, 1, 64, 48)])
@pytest.mark.parametrize("halves", [True, False])
@pytest.mark.parametrize("bf16,out_bf16", [(False, False), (False, True), (True, True), (True, False)])
@pytest.mark.parametrize("normed", [True, False])
def test_rotation(qmv, rows, heads, kv_heads, dim, rot, halves, bf16, out_bf16, normed):
    import torch
    rng = np.random.default_rng(rows + heads * dim + rot)
    q, qd = _make(rng, rows, heads, dim, bf16)
    k, kd = _make(rng, rows, kv_heads, dim, bf16)
    qw, kw = ((1 + 0.2 * rng.standard_normal(dim)).astype(F) for _ in range(2)) if normed else (None, None)
    pos = rng.integers(0, 2 ** 20, rows).astype(np.int32)
    freq = (500000.0 ** (-np.arange(0, rot, 2) / rot)).astype(F)
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()  # noqa: E731
    gq, gk = qmv.qk_rope(qd, kd, up(pos), up(freq), q_weight=up(qw), k_weight=up(kw), eps=1e-5, pairs="halves" if halves else "neighbours",
                         factor=1.25, out="bf16" if out_bf16 else "f32")
    for got, x, w in ((gq, q, qw), (gk, k, kw)):
        want, mag = step_ref.qk_rope(x, w, float(F(1e-5)), pos, freq, halves, 1.25)
        _check(got, want, mag, normed, out_bf16)


def test_far_and_negative_positions_and_frequencies(qmv):
    import torch
    rng = np.random.default_rng(4)
    pos = np.array([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31, 131071, 10 ** 6 + 3], np.int32)
    q, qd = _make(rng, len(pos), 3, 64, False)
    freq = np.concatenate([[0.0, 1.0, -1.0, 3.5, 100.25, 1e-30], rng.random(26)]).astype(F)
    got, none = qmv.qk_rope(qd, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda())
    assert none is None
    want, mag = step_ref.qk_rope(q, None, 0, pos, freq, True)
    _check(got, want, mag, False, False)


def test_norm_alone_one_weight_and_extremes(qmv):
    import torch
    rng = np.random.default_rng(6)
    q, qd = _make(rng, 4, 6, 128, False)
    k, kd = _make(rng, 4, 2, 128, False)
    w = (1 + 0.2 * rng.standard_normal(128)).astype(F)
    gq, gk = qmv.qk_rope(qd, kd, None, None, k_weight=torch.from_numpy(w).cuda(), eps=1e-6)
    assert torch.equal(gq, qd)
    want, mag = step_ref.qk_rope(k, w, float(F(1e-6)), None, None, True)
    _check(gk, want, mag, True, False)
    z = torch.zeros((2, 6, 128), device="cuda")
    gz, _ = qmv.qk_rope(z, None, None, None, q_weight=torch.from_numpy(w).cuda(), eps=1e-6)
    assert torch.equal(gz, z)
    empty, _ = qmv.qk_rope(qd[:0], None, None, None)
    assert empty.shape == (0, 6, 128)


@pytest.mark.parametrize("halves", ["halves", "neighbours"])
def test_slices_in_place_streams_and_graphs(qmv, halves):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, h, kvh, d = 9, 12, 4, 128
    wide = torch.randn((rows, (h + 2 * kvh) * d + 8), device="cuda", generator=g)
    q, k = wide[:, :h * d].unflatten(1, (h, d)), wide[:, h * d:(h + kvh) * d].unflatten(1, (kvh, d))
    keep = wide.clone()
    pos = torch.arange(rows, dtype=torch.int32, device="cuda") * 1000
    freq = torch.rand(d // 2, device="cuda", generator=g)
    w = torch.rand(d, device="cuda", generator=g)
    a, b = qmv.qk_rope(q, k, pos, freq, q_weight=w, k_weight=w, pairs=halves)
    assert torch.equal(wide, keep)
    a2, b2 = qmv.qk_rope(q.contiguous(), k.contiguous(), pos, freq, q_weight=w, k_weight=w, pairs=halves)
    assert torch.equal(a, a2) and torch.equal(b, b2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a3, b3 = qmv.qk_rope(q, k, pos, freq, q_weight=w, k_weight=w, pairs=halves, stream=side)
    side.synchronize()
    assert torch.equal(a, a3) and torch.equal(b, b3)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmv.qk_rope(q, k, pos, freq, q_weight=w, k_weight=w, pairs=halves, q_out=q, k_out=k)
    assert torch.equal(wide, keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(wide[:, (h + kvh) * d:], keep[:, (h + kvh) * d:])  # the values and what lies behind are as they were
    for bad in (dict(pos=None), dict(pos=pos.long()), dict(freq=freq.double()), dict(q_weight=w[:64]), dict(pairs="both"), dict(out="f16"),
                dict(k=k.bfloat16()), dict(q=q.transpose(1, 2)), dict(q_out=a.bfloat16()), dict(k=None, k_weight=w)):
        with pytest.raises(ValueError):
            qmv.qk_rope(**{**dict(q=q, k=k, pos=pos, freq=freq), **bad})
