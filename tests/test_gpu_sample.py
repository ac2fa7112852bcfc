"""qmv_sample against the definition in 64 bits: cuts, ties, masks, sizes, strides, streams and graphs, and what it draws."""
import numpy as np
import pytest

import step_ref

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


def _logits(rng, rows, vocab, kind):
    x = (2.2 * rng.standard_normal((rows, vocab))).astype(F)
    if kind == "sharp":
        at = rng.integers(0, vocab, (rows, min(40, vocab)))
        np.put_along_axis(x, at, (8 + 8 * rng.random(at.shape)).astype(F), axis=1)
    elif kind == "steps":  # few values: many equal logits
        x = np.round(x * 2) / 2
    elif kind == "equal":
        x[:] = 1.25
    elif kind == "near":  # all within one bucket, few of them equal
        x = (3 + 1e-4 * rng.random((rows, vocab))).astype(F)
    if kind != "equal" and vocab > 8:
        x[:, vocab - vocab // 8:] = -np.inf
    return x.astype(F)


def _settings(rng, rows, kind):
    pick = lambda v: rng.choice(v, rows)  # noqa: E731
    t = pick([0.6, 0.9, 1.0, 1.5]).astype(F)
    k = pick([0, 1, 2, 7, 40, 1000, 5000]).astype(np.int32)
    p = pick([1.0, 0.3, 0.9, 0.999]).astype(F)
    m = pick([0.0, 0.01, 0.2]).astype(F)
    if kind == "k":
        return t, k, None, None
    if kind == "p":
        return t, None, p, None
    if kind == "m":
        return t, None, None, m
    if kind == "free":
        return t, None, None, None
    if kind == "none":
        return None, None, None, None
    t[rng.random(rows) < 0.1] = 0
    return t, k, p, m


def _run(qmv, x, e, s, **more):
    import torch
    dev = [None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in s]
    got = qmv.sample(torch.from_numpy(x).cuda(), torch.from_numpy(e).cuda(), *dev, **more)
    return got.cpu().numpy()


def _check(x, e, s, got):
    for i in range(x.shape[0]):
        v = [d if a is None else a[i] for a, d in zip(s, (F(1), 0, F(1), F(0)))]
        may = step_ref.sample(x[i], e[i], *v)
        assert int(got[i]) in may, (i, int(got[i]), may, v)


@pytest.mark.parametrize("rows,vocab", [(1, 1), (2, 2), (3, 5), (2, 31), (7, 1000), (5, 4099), (1, 8192), (2, 32000), (1, 151936),
                                        (200, 2050), (400, 517), (80, 20001)])
@pytest.mark.parametrize("kind", ["flat", "sharp"])
@pytest.mark.parametrize("cuts", ["all", "k", "p", "m", "free", "none"])
def test_sizes_and_cuts(qmv, rows, vocab, kind, cuts):
    rng = np.random.default_rng(rows * 1000 + vocab)
    x, e = _logits(rng, rows, vocab, kind), rng.exponential(size=(rows, vocab)).astype(F)
    s = _settings(rng, rows, cuts)
    _check(x, e, s, _run(qmv, x, e, s))


@pytest.mark.parametrize("kind", ["steps", "equal", "near"])
@pytest.mark.parametrize("vocab", [3000, 30011])
def test_borders_among_equal_logits(qmv, kind, vocab):
    """More equal or nearly equal logits than are collected at a time."""
    rng = np.random.default_rng(vocab)
    s = [(0.8, 2500, 1.0, 0.0), (1.0, 0, 0.5, 0.0), (1.3, 2900, 0.7, 0.0), (1.0, 2048, 0.999, 0.1), (0.7, 2049, 0.2, 0.0), (2.0, 2, 0.9, 0.0)]
    t, k, p, m = (np.array(a) for a in zip(*s))
    x, e = _logits(rng, len(s), vocab, kind), rng.exponential(size=(len(s), vocab)).astype(F)
    s = (t.astype(F), k.astype(np.int32), p.astype(F), m.astype(F))
    _check(x, e, s, _run(qmv, x, e, s))


def test_kept_sets(qmv):
    """The kept set itself: with noise that puts one id ahead of all others, that id comes out where it is kept, and only there."""
    rng = np.random.default_rng(5)
    vocab, k, p = 5000, 60, 0.8
    x = _logits(rng, 1, vocab, "flat")
    order = step_ref.prefix_order(x[0])
    w = np.exp((x[0].astype(np.float64) - x[0].max()) / 0.9)[order]
    mass = np.where(np.arange(vocab) < k, w, 0)
    n = int((np.cumsum(mass) - mass < np.float64(F(p)) * mass.sum()).sum())
    assert 2 < n < k
    rows = 64
    e = np.ones((rows, vocab), F)
    for i in range(rows):
        e[i, order[i]] = 1e-30
    s = (np.full(rows, 0.9, F), np.full(rows, k, np.int32), np.full(rows, p, F), None)
    got = _run(qmv, np.repeat(x, rows, 0), e, s)
    assert np.array_equal(got[:n], order[:n])
    assert np.all(got[n:] == order[0])  # the others are cut off; among equal noise the largest logit wins


def test_special_rows(qmv):
    rng = np.random.default_rng(9)
    x = _logits(rng, 12, 4001, "flat")
    e = rng.exponential(size=x.shape).astype(F)
    x[0, 77] = np.nan
    x[1] = -np.inf
    x[2] = -np.inf
    x[2, 4000] = -3e38  # the only id
    x[3, [5, 9]] = np.inf
    x[4] = np.finfo(F).min
    x[5, :] = 0.0
    x[5, ::2] = -0.0  # equal to +0
    e[6] = 0.0  # nothing can be chosen: the largest
    e[7] = np.nan
    e[8, :2000] = 0.0
    e[9] = 1e-45  # subnormal, all equal
    x[10] = np.finfo(F).max
    x[11, 3] = 3e38
    s = (np.full(12, 1.0, F), np.array([0, 0, 4, 0, 30, 10, 0, 3, 0, 7, 100, 2], np.int32), np.full(12, 0.9, F), None)
    _check(x, e, s, _run(qmv, x, e, s))
    s = (np.full(12, 0.7, F), None, None, None)
    _check(x, e, s, _run(qmv, x, e, s))


def test_settings_outside_their_range(qmv):
    rng = np.random.default_rng(10)
    x = _logits(rng, 10, 3001, "sharp")
    e = rng.exponential(size=x.shape).astype(F)
    t = np.array([-1, np.nan, 0, 1e-38, 1e30, np.inf, 1, 1, 1, 1], F)
    k = np.array([0, 0, 0, 0, 5, 5, -3, 4000, 2 ** 31 - 1, 0], np.int32)
    p = np.array([1, 1, 1, 1, 1, 1, 2, np.nan, 1, -1], F)
    m = np.array([0, 0, 0, 0, 0, 0, -1, np.nan, 5, 0], F)
    got = _run(qmv, x, e, (t, k, p, m))
    first = np.array([step_ref.prefix_order(r)[0] for r in x])
    assert np.array_equal(got[[0, 1, 2, 3, 8, 9]], first[[0, 1, 2, 3, 8, 9]])
    for i in (6, 7):  # nothing is cut off
        assert int(got[i]) in step_ref.sample(x[i], e[i])
    for i in (4, 5):  # everything weighs the same: the smallest noise among the first five
        ids = step_ref.prefix_order(x[i])[:5]
        assert got[i] == ids[np.argmin(e[i][ids])]


def test_draws_follow_the_weights(qmv):
    """Frequencies of 40000 draws within 6 standard deviations of the kept weights' shares."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.tensor([0.0, 1.0, -1.0, 2.5, 2.5, -3.0, 0.5, 1.5] + [-20.0] * 100, device="cuda")
    n = 40000
    e = torch.empty((n, x.numel()), device="cuda").exponential_(generator=g)
    for t, k, share in ((0.7, 0, None), (1.3, 5, None), (1.0, 3, None)):
        got = qmv.sample(x.expand(n, -1).contiguous(), e, torch.full((n,), t, device="cuda"), torch.full((n,), k, dtype=torch.int32, device="cuda"))
        w = torch.exp(x.double().cpu() / t)
        if k:
            keep = torch.topk(x.cpu(), k)[1]
            w = torch.zeros_like(w).scatter(0, keep, w[keep])
        p = (w / w.sum()).numpy()
        c = torch.bincount(got.cpu(), minlength=x.numel()).numpy()
        assert np.all(np.abs(c - n * p) <= 6 * np.sqrt(n * p * (1 - p)) + 1)


def test_strides_streams_and_graphs(qmv):
    import torch
    rng = np.random.default_rng(11)
    rows, vocab = 6, 9001
    wide = torch.from_numpy(_logits(rng, rows, vocab + 7, "sharp")).cuda()
    noise = torch.from_numpy(rng.exponential(size=(rows, vocab + 2)).astype(F)).cuda()
    s = [torch.from_numpy(a).cuda() for a in _settings(rng, rows, "all")]
    views = [(wide[:, i:i + vocab], noise[:, j:j + vocab]) for i in range(4) for j in (0, 1)]  # every 4-byte alignment
    for x, e in views:
        _check(x.cpu().numpy(), e.cpu().numpy(), [a.cpu().numpy() for a in s], qmv.sample(x, e, *s).cpu().numpy())
        assert torch.equal(qmv.sample(x, e), qmv.sample(x.contiguous(), e.contiguous()))
    x, e = views[1]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = qmv.sample(x, e, *s, stream=side)
    side.synchronize()
    assert torch.equal(a, qmv.sample(x, e, *s))
    # two captured graphs, replayed on two streams at once: nothing is shared between calls
    outs = [torch.empty(rows, dtype=torch.int64, device="cuda") for _ in range(2)]
    graphs = []
    for o in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            qmv.sample(x, e, *s, ids=o)
        graphs.append(g)
    s[1].fill_(3)  # read when the graph runs
    torch.cuda.synchronize()
    for _ in range(5):
        graphs[0].replay()
        with torch.cuda.stream(side):
            graphs[1].replay()
    torch.cuda.synchronize()
    want = qmv.sample(x, e, *s)
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


def test_no_rows_and_refusals(qmv):
    import torch
    x = torch.zeros((0, 10), device="cuda")
    assert qmv.sample(x, x).shape == (0,)
    y = torch.zeros((3, 10), device="cuda")
    for bad in (dict(noise=y[:2]), dict(noise=y.double()), dict(temperature=torch.ones(2, device="cuda")), dict(top_k=torch.ones(3, device="cuda")),
                dict(noise=y.t().contiguous().t()), dict(ids=torch.zeros(3, dtype=torch.int32, device="cuda")), dict(temperature=torch.ones(3))):
        with pytest.raises(ValueError):
            qmv.sample(**{**dict(logits=y, noise=y), **bad})
