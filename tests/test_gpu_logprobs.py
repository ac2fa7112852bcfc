"""qmv_logprobs against 64 bits: given ids, entropy, the top alternatives with ties and masked ids."""
import numpy as np
import pytest

import ops_ref

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


def run(qmv, x, given, top, pad=0, offset=0):
    """x in a wider buffer: rows `pad` apart more than they are long, the first `offset` floats in."""
    import torch
    rows, n = x.shape
    buf = torch.full((rows, n + pad + offset), 1e30, device="cuda")
    view = buf[:, offset:offset + n]
    view.copy_(torch.from_numpy(x))
    got = qmv.logprobs(view, torch.from_numpy(given).cuda(), top=top)
    return [None if t is None else t.cpu().numpy() for t in got]


def check(x, given, top, got):
    lp, h = ops_ref.logprobs(x)
    glp, ent, ids, tlp = got
    # x - m and its logarithm's sum: a few roundings of values up to span, float32 sums of n terms
    finite = np.where(np.isfinite(x) & (lp > -1e4), np.abs(x), 0.0).astype(np.float64)
    span = 1 + 2 * finite.max(axis=1, keepdims=True)
    tol = (span * 4 + 16 + np.sqrt(x.shape[1])) * 2.0 ** -24
    ref = np.take_along_axis(lp, given, axis=1)
    live = np.isfinite(ref)
    assert np.array_equal(np.isneginf(ref), np.isneginf(glp))
    with np.errstate(invalid="ignore"):
        err = np.abs(glp.astype(np.float64) - ref)
    assert np.all(err[live] <= (np.broadcast_to(tol, ref.shape) + 2.0 ** -23 * np.abs(np.where(live, ref, 0)))[live])
    assert np.all(np.abs(ent - h) <= tol[:, 0] * (4 + np.abs(h) * 2))
    if top:
        want = ops_ref.top_ids(x, top)
        assert np.array_equal(ids, want)
        ref = np.take_along_axis(lp, want.astype(np.int64), axis=1)
        live = np.isfinite(ref)
        assert np.array_equal(np.isneginf(ref), np.isneginf(tlp))
        with np.errstate(invalid="ignore"):
            err = np.abs(tlp.astype(np.float64) - ref)
        assert np.all(err[live] <= (np.broadcast_to(tol, ref.shape) + 2.0 ** -23 * np.abs(np.where(live, ref, 0)))[live])


@pytest.mark.parametrize("rows,n", [(1, 1), (3, 2), (2, 31), (1, 1000), (5, 4097), (64, 3001), (1, 151936), (9, 32003), (200, 777)])
@pytest.mark.parametrize("top", [0, 1, 8, 32])
def test_random_rows(qmv, rows, n, top):
    rng = np.random.default_rng(n + rows)
    top = min(top, n)
    x = (3 * rng.standard_normal((rows, n))).astype(F)
    given = rng.integers(0, n, (rows, 3))
    check(x, given, top, run(qmv, x, given, top))


@pytest.mark.parametrize("pad,offset", [(1, 0), (0, 1), (3, 2), (4, 4), (128, 3)])
def test_strides_and_alignment(qmv, pad, offset):
    rng = np.random.default_rng(pad)
    x = (2 * rng.standard_normal((4, 5003))).astype(F)
    given = rng.integers(0, 5003, (4, 1))
    check(x, given, 5, run(qmv, x, given, 5, pad, offset))


def test_ties_go_to_the_lower_id(qmv):
    rng = np.random.default_rng(0)
    x = rng.integers(-3, 4, (6, 20000)).astype(F)      # thousands of equal logits
    x[1] = 0.0
    x[1, ::2] = -0.0                                    # +0 and -0 are equal
    x[2] = np.arange(20000)                             # ascending: every element enters the list
    x[3] = -np.arange(20000)
    x[4, :] = -5
    x[4, -3:] = 2
    given = np.zeros((6, 1), np.int64)
    check(x, given, 32, run(qmv, x, given, 32))


def test_masked_ids(qmv):
    """-infinity and the type's lowest value as masks, rows with one id left and with none."""
    rng = np.random.default_rng(1)
    x = (2 * rng.standard_normal((6, 3000))).astype(F)
    x[0, ::3] = -np.inf
    x[1, 5:] = np.finfo(F).min
    x[2] = -np.inf
    x[2, 1234] = 3.0
    x[3] = -np.inf
    x[4] = np.finfo(F).min
    x[5, :2990] = -np.inf
    given = np.array([[0, 1, 2], [0, 4, 5], [1234, 0, 2999], [0, 1, 2], [7, 8, 9], [0, 2995, 2999]])
    check(x, given, 20, run(qmv, x, given, 20))


def test_nan_infinity_and_ids_outside(qmv):
    import torch
    rng = np.random.default_rng(1)
    x = (2 * rng.standard_normal((3, 900))).astype(F)
    x[0, 17] = np.nan
    x[1, 30] = np.inf
    glp, ent, ids, tlp = run(qmv, x, np.array([[1, 2], [1, 2], [-1, 900]]), 3)
    assert np.isnan(glp).all() and np.isnan(ent[:2]).all() and np.isnan(tlp[:2]).all()
    assert ids[0, 0] == 17 and ids[1, 0] == 30
    assert np.isfinite(ent[2]) and np.isfinite(tlp[2]).all()
    got = qmv.logprobs(torch.zeros((0, 50), device="cuda"), top=2)
    assert got[0] is None and got[2].shape == (0, 2)
    got = qmv.logprobs(torch.zeros((2, 50), device="cuda"), entropy=False, top=2)
    assert got[1] is None and got[2].tolist() == [[0, 1], [0, 1]]


def test_another_stream_and_repeat(qmv):
    import torch
    x = torch.randn((3, 50000), device="cuda")
    given = torch.zeros((3, 1), dtype=torch.int64, device="cuda")
    a = qmv.logprobs(x, given, top=6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = qmv.logprobs(x, given, top=6)
        c = qmv.logprobs(x, given, top=6)
    s.synchronize()
    for u, v, w in zip(a, b, c):
        assert torch.equal(u, v) and torch.equal(u, w)


@pytest.mark.parametrize("warm", [False, True])
def test_in_a_graph(qmv, warm):
    """Captured on a stream without a workspace (rows are not cut) and on one with it."""
    import torch
    x = (2 * np.random.default_rng(3).standard_normal((2, 60001))).astype(F)
    xd = torch.zeros((2, 60001), device="cuda")
    given = torch.tensor([[5], [60000]], device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if warm:
        qmv.logprobs(xd, given, top=3, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        got = qmv.logprobs(xd, given, top=3)
    xd.copy_(torch.from_numpy(x))
    g.replay()
    torch.cuda.synchronize()
    check(x, given.cpu().numpy(), 3, [t.cpu().numpy() for t in got])


@pytest.mark.parametrize("at", [1e5, -1e6, 3e7, "lowest"])
@pytest.mark.parametrize("n", [3000, 60001])
def test_large_maximum_keeps_log_z(qmv, at, n):
    """Rows whose logits are large beside their differences: (x - m) - log Z.  x - m is exact where x and m lie within a
    factor of two (else rounded once), the sum of n exponentials carries sqrt(n) 2^-24 and 2^-22 an exponential, the
    logarithm and the two differences a rounding each of at most |lp| 2^-23."""
    rng = np.random.default_rng(n)
    if at == "lowest":
        x = np.full((2, n), np.finfo(F).min, F)
        x[1, ::3] = -np.inf
    else:
        x = (at + 3 * rng.standard_normal((2, n))).astype(F)
    given = np.array([[0, 1, n - 1], [1, 2, n - 2]])
    got = run(qmv, x, given, 20)
    lp, h = ops_ref.logprobs(x)

    def close(a, b):
        live = np.isfinite(b)
        assert np.array_equal(np.isneginf(a), np.isneginf(b))
        tol = np.sqrt(n) * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -23 * np.abs(np.where(live, b, 0))
        assert np.all(np.abs(np.where(live, a, 0).astype(np.float64) - np.where(live, b, 0)) <= tol)

    close(got[0], np.take_along_axis(lp, given, axis=1))
    ids = ops_ref.top_ids(x, 20)
    assert np.array_equal(got[2], ids)
    close(got[3], np.take_along_axis(lp, ids.astype(np.int64), axis=1))
    # a term of the entropy is an exponential's error times its difference to the maximum, the quotient's and log Z's errors
    span = np.abs(np.where(np.isfinite(x), x.astype(np.float64) - x.max(axis=1, keepdims=True), 0)).max(axis=1)
    assert np.all(np.abs(got[1] - h) <= (np.sqrt(n) + 8) * 2.0 ** -23 * (1 + span + np.abs(h)))
