"""qmv_qk_rope's cosines and sines themselves: heads of (1, 0) pairs."""
import numpy as np
import pytest

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


def _turn(qmv, pos, freq):
    """cos and sin (rows, freq.size) as the call turns them, and of the exact angles."""
    import torch
    half = freq.size
    x = torch.zeros((pos.size, 1, 2 * half), device="cuda")
    x[..., :half] = 1.0
    y = qmv.qk_rope(x, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda())[0][:, 0].cpu().numpy()
    t = pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)  # (exact: 31 and 24 bits)
    return y[:, :half], y[:, half:], np.cos(t), np.sin(t)


@pytest.mark.parametrize("far", [2 ** 12, 2 ** 20, 2 ** 31 - 1])
@pytest.mark.parametrize("sign", [1, -1])
def test_angles(qmv, far, sign):
    """An angle is off by 2 units of 2^-64 turns for each position, 2^-29.3 radians at the farthest (and by 2^-43 for the square of what its
    first 24 bits leave).  sincospif's values are off by 2 of their own last places, 4 2^-24 of themselves, the turn by the rest rounds once
    more.  So near the axes, where a value is small, it is nearly exact."""
    rng = np.random.default_rng(far)
    pos = rng.integers(-far, far, 4000).astype(np.int32)
    freq = (sign * np.concatenate([rng.random(100), 500000.0 ** (-np.arange(28) / 28)])).astype(F)
    c, s, want_c, want_s = _turn(qmv, pos, freq)
    for got, want in ((c, want_c), (s, want_s)):
        err = np.abs(got - want).astype(np.float64)
        size = np.abs(want).astype(np.float64)
        assert (size < 2.0 ** -10).sum() > 100
        bound = 2.0 ** -29 * max(far / 2 ** 31, 2.0 ** -10) + 2.0 ** -43 + 5.0 * 2.0 ** -24 * size
        assert np.all(err <= bound), float(np.max(err / bound))


@pytest.mark.parametrize("halves", [True, False])
def test_frequencies_without_an_angle(qmv, halves):
    """Frequencies that are not finite, or 2^40 and more, give NaN in their pairs and change nothing else; those below are exact."""
    import torch
    bad = np.array([np.nan, np.inf, -np.inf, 2.0 ** 40, -3e38], F)
    fine = np.array([np.nextafter(F(2.0 ** 40), F(0)), -1e9, 12345.678, 0.0, -0.0, 1e-45, 0.25, 1.5, 7.0, 3e11, -1e12], F)
    freq = np.concatenate([fine[:5], bad, fine[5:]])
    pos = np.array([0, 1, -1, 77, 2 ** 31 - 1, -2 ** 31], np.int32)
    half = freq.size
    x = torch.zeros((pos.size, 2, 64), device="cuda")
    x[:, 1], x[:, 0, 2 * half:] = 3.0, 5.0
    a = slice(0, half) if halves else slice(0, 2 * half, 2)
    b = slice(half, 2 * half) if halves else slice(1, 2 * half, 2)
    x[:, 0, a] = 1.0
    y = qmv.qk_rope(x, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda(), pairs="halves" if halves else "neighbours")[0].cpu().numpy()
    none = np.isin(np.arange(half), np.arange(5, 10))
    for part in (a, b):
        assert np.isnan(y[:, :, part][..., none]).all() and np.isfinite(y[:, :, part][..., ~none]).all()
    assert np.all(y[:, 0, 2 * half:] == 5.0) and np.all(y[:, 1, 2 * half:] == 3.0)
    t = pos.astype(np.longdouble)[:, None] * freq[~none].astype(np.longdouble)  # (55 bits: exact)
    assert np.all(np.abs(y[:, 0, a][:, ~none] - np.cos(t)) <= 2.0 ** -28 + 5.0 * 2.0 ** -24)
    assert np.all(np.abs(y[:, 0, b][:, ~none] - np.sin(t)) <= 2.0 ** -28 + 5.0 * 2.0 ** -24)
