"""qmv_sample's special rows and the borders of what it keeps, probed id by id."""
import numpy as np
import pytest

from test_gpu_sample import _logits

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


@pytest.mark.parametrize("vocab", [3, 5000, 300001])
@pytest.mark.parametrize("shift", [0, 1])
def test_infinity_whatever_its_noise(qmv, vocab, shift):
    """A row with +infinity gives the lowest id of those, uncut or cut, the noise where it is and at another alignment than the logits."""
    import torch
    rng = np.random.default_rng(vocab)
    bad = [np.nan, -1.0, np.inf, 0.0, 1.0]
    x = rng.standard_normal((len(bad), vocab)).astype(F)
    e = np.zeros((len(bad), vocab + shift), F)
    e[:, shift:] = rng.exponential(size=x.shape)
    at = [vocab // 2, vocab - 1, 0, vocab // 3, vocab - 2]
    for r, (a, v) in enumerate(zip(at, bad)):
        x[r, [a, vocab - 1]] = np.inf
        e[r, [shift + a, shift + vocab - 1]] = v
    logits, noise = torch.from_numpy(x).cuda(), torch.from_numpy(e).cuda()[:, shift:]
    p = torch.full((len(bad),), 0.9, device="cuda")
    assert qmv.sample(logits, noise).tolist() == at
    assert qmv.sample(logits, noise, top_p=p).tolist() == at
    assert qmv.sample(logits, noise, top_k=torch.full((len(bad),), 2, dtype=torch.int32, device="cuda"), min_p=p).tolist() == at


@pytest.mark.parametrize("vocab", [7, 3000, 300001])
def test_scores_past_float32(qmv, vocab):
    """Where the largest logits' noise rules them out, the best of the others is chosen, however low its score: temperatures and
    logits whose quotients pass float32's range."""
    import torch
    rng = np.random.default_rng(vocab)
    x = np.stack([rng.standard_normal(vocab), rng.standard_normal(vocab), -3e38 + 1e37 * rng.random(vocab), 1e20 * rng.standard_normal(vocab)]).astype(F)
    x[2, vocab // 2] = 3e38
    t = np.array([1e-20, 2.0 ** -99, 1.0, 1e-18], F)
    e = rng.exponential(size=x.shape).astype(F)
    want = []
    for r, bad in enumerate((0.0, np.nan, -1.0, np.inf)):
        order = np.lexsort((np.arange(vocab), -x[r]))
        e[r, order[:2]] = bad
        z = (x[r].astype(np.float64) - x[r].max()) / np.float64(t[r])
        ids = order[2:]  # (of different logits; their noise decides nothing at these distances, but among the close ones of row 2)
        want.append(int(ids[np.argmax(z[ids] - np.log(e[r, ids].astype(np.float64)))]))
    up = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    assert qmv.sample(up(x), up(e), up(t)).tolist() == want
    k = np.array([5, 1000, 4, 2500], np.int32)
    assert qmv.sample(up(x), up(e), up(t), up(k))[[0, 1, 3]].tolist() == [want[i] for i in (0, 1, 3)]
    e[:] = rng.choice(np.array([0.0, -2.0, np.nan, np.inf], F), e.shape)  # none that can be chosen: the largest
    for cut in (None, up(k)):
        assert qmv.sample(up(x), up(e), up(t), cut).tolist() == x.argmax(axis=1).tolist()


def _kept(x, t, k, p, m):
    """The row's ids in descending order, and how many of the first are kept: lo at least, hi at most, by the documentation's slack.
    Top-p's: each weight off by (1 + ln 1/w) 2^-21 of itself and 2^-32 of the largest, so as far off the mass above an id and the
    kept mass; a row's sum by float32 additions of vocab / 4096 terms in a thread and 5 + 8 steps of joining.  Min-p's: 64 bits'."""
    x64 = x.astype(np.float64) + 0.0
    order = np.lexsort((np.arange(x.size), -x64))
    n = int(np.isfinite(x).sum())
    z = (x64[order[:n]] - x64[order[0]]) / np.float64(F(t))
    if 0 < k < n:
        n = k
    z = z[:n]
    w = np.exp(z)
    lo = hi = n
    if p < 1:
        eps = (1 - z) * 2.0 ** -21 * w + 2.0 ** -32
        before, off = np.cumsum(w) - w, np.cumsum(eps) - eps
        total, far = w.sum(), eps.sum() + w.sum() * (x.size / 4096 + 13) * 2.0 ** -24
        lo = max(1, int((before + off < np.float64(F(p)) * (total - far)).sum()))
        hi = max(1, int((before - off < np.float64(F(p)) * (total + far)).sum()))
    if m > 0:
        m = min(np.float64(F(m)), 1.0)
        off = 2.0 ** -45 if m < 1 else 0.0
        lo, hi = min(lo, int((w >= m * (1 + off)).sum())), min(hi, int((w >= m * (1 - off)).sum()))
    return order, np.exp(z), max(lo, 1), max(hi, 1)


# logits, their count, and the settings: what places the border is on the right
ROUTES = [
    ("flat", 5000, 0.9, 60, 0.8, 0.0),        # the list holds everything kept
    ("sharp", 30011, 0.8, 0, 0.95, 0.0),
    ("sharp", 30011, 0.8, 50, 0.9, 0.05),
    ("flat", 30011, 0.9, 0, 0.5, 0.0),        # top-p: a bucket is collected
    ("flat", 30011, 1.1, 0, 0.9, 0.0),
    ("flat", 30011, 0.7, 0, 0.999, 0.0),
    ("flat", 151936, 0.9, 0, 0.95, 0.0),
    ("flat", 30011, 1.0, 2049, 1.0, 0.0),     # top-k past the list: a bucket
    ("flat", 30011, 0.8, 20000, 1.0, 0.0),
    ("flat", 3000, 1.0, 2500, 1.0, 0.0),
    ("flat", 30011, 1.0, 2500, 0.7, 0.0),     # both: the k-th logit, then the mass above it
    ("flat", 30011, 1.3, 20000, 0.9, 0.0),
    ("flat", 30011, 0.6, 5000, 0.999, 0.0),
    ("steps", 30011, 1.0, 0, 0.7, 0.0),       # equal logits: the bucket is cut again by the keys' bits
    ("steps", 30011, 0.9, 9000, 1.0, 0.0),
    ("steps", 30011, 0.9, 9000, 0.8, 0.0),
    ("equal", 3000, 1.0, 0, 0.5, 0.0),
    ("equal", 30011, 0.8, 0, 0.9, 0.0),
    ("equal", 30011, 0.8, 2500, 1.0, 0.0),
    ("equal", 30011, 1.3, 20000, 0.7, 0.0),
    ("near", 3000, 1.3, 2900, 0.7, 0.0),
    ("near", 30011, 1.0, 0, 0.5, 0.0),
    ("near", 30011, 1.0, 20000, 1.0, 0.0),
    ("near", 30011, 1.0, 20000, 0.3, 0.0),
    ("flat", 30011, 0.9, 0, 0.9, 0.02),       # min-p after them
    ("flat", 30011, 1.1, 0, 0.99, 0.001),
    ("flat", 30011, 1.0, 5000, 1.0, 0.01),
    ("flat", 30011, 1.0, 20000, 0.95, 0.003),
    ("near", 30011, 1.0, 20000, 1.0, 1.0),
    ("sharp", 30011, 1.0, 0, 1.0, 0.1),       # min-p alone
    ("flat", 30011, 1.0, 0, 1.0, 0.05),
    ("flat", 30011, 1.2, 0, 1.0, 1e-4),
    ("flat", 151936, 0.9, 0, 1.0, 1e-6),
    ("flat", 30011, 0.6, 0, 1.0, 1e-8),
    ("equal", 30011, 1.0, 0, 1.0, 1.0),
    ("flat", 300001, 1.0, 0, 0.9, 0.0),       # rows of more chunks than there are places for
    ("flat", 300001, 1.0, 100000, 0.9, 0.0),
    ("sharp", 300001, 0.9, 0, 0.9, 1e-5),
    ("near", 300001, 1.0, 0, 0.7, 0.0),
    ("steps", 300001, 1.0, 100000, 1.0, 0.0),
    ("flat", 1000003, 1.0, 0, 0.9, 0.0),
]


@pytest.mark.parametrize("kind,vocab,t,k,p,m", ROUTES)
def test_borders(qmv, kind, vocab, t, k, p, m):
    """Of ids around the border one at a time gets noise that puts it ahead of all others: it comes out where it is kept, else the
    largest logit does.  In one call for all of them, and for some in a call of their own (more CTAs a row)."""
    import torch
    rng = np.random.default_rng([vocab, len(kind), k, int(1000 * p)])
    x = _logits(rng, 1, vocab, kind)[0]
    order, w, lo, hi = _kept(x, t, k, p, m)
    finite = int(np.isfinite(x).sum())
    assert hi - lo <= 2 + 2.0 ** -7 * hi  # (what the slack leaves open)
    at = sorted({i for i in (0, 1, lo // 2, lo - 3, lo - 2, lo - 1) if 0 <= i < lo} | {i for i in (hi, hi + 1, hi + 2, hi + 100, finite - 1) if hi <= i < finite})
    assert w[[i for i in at if i < lo]].min() > 1e-25  # (the noise outweighs that)
    rows = len(at)
    e = torch.ones((rows, vocab), device="cuda")
    e[torch.arange(rows), torch.from_numpy(order[at]).cuda()] = 1e-30
    logits = torch.from_numpy(x).cuda().repeat(rows, 1)
    how = dict(temperature=torch.full((rows,), t, device="cuda"), top_k=torch.full((rows,), k, dtype=torch.int32, device="cuda"),
               top_p=torch.full((rows,), p, device="cuda"), min_p=torch.full((rows,), m, device="cuda"))
    want = [int(order[i]) if i < lo else int(order[0]) for i in at]
    assert qmv.sample(logits, e, **how).tolist() == want
    for r in range(max(0, sum(i < lo for i in at) - 2), min(rows, sum(i < lo for i in at) + 2)):
        assert qmv.sample(logits[r:r + 1], e[r:r + 1], **{n: v[r:r + 1] for n, v in how.items()}).item() == want[r]


def test_min_p_to_the_last_bit(qmv):
    """The smallest float32 logit of min-p's weight is kept, the one below it is not, whatever min-p, temperature and maximum."""
    import torch
    rng = np.random.default_rng(21)
    n = 400
    t, m = rng.uniform(0.3, 2.0, n).astype(F), (10.0 ** rng.uniform(-12, -0.05, n)).astype(F)
    top = (rng.standard_normal(n) * 10.0 ** rng.uniform(-3, 2, n)).astype(F)
    t[:4], m[:4] = [2.0 ** 100, 2.0 ** -60, 1.0, 1.0], [1e-3, 0.9, 1e-45, 1.0]
    least = top.astype(np.float64) + t.astype(np.float64) * np.log(m.astype(np.float64))
    kept = least.astype(F)
    kept = np.where(kept < least, np.nextafter(kept, F(np.inf)), kept)
    kept[3] = top[3]
    for off in (0, 1):
        x = np.full((n, 9), F(-3e38))
        x[:, 7], x[:, 5 - off] = top, kept if off == 0 else np.nextafter(kept, F(-np.inf))
        e = np.ones((n, 9), F)
        e[:, 5 - off] = 1e-38
        clear = (x[:, 5 - off] > x[:, 0]) & (x[:, 5 - off] < top) & (t * 80 > top - x[:, 5 - off])  # (the noise outweighs the distance)
        assert clear.sum() > n - 10
        got = qmv.sample(*(torch.from_numpy(a).cuda() for a in (x, e, t)), min_p=torch.from_numpy(m).cuda()).cpu().numpy()
        assert np.array_equal(got[clear], np.full(n, 5 if off == 0 else 7)[clear])


@pytest.mark.parametrize("vocab", [5, 3001, 32000])
def test_rows_that_are_one(qmv, vocab):
    """Logits, noise or both expanded to rows: as if they had been copied into each."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(vocab)
    rows = 37
    x, e = torch.randn((1, vocab), device="cuda", generator=g), torch.empty((rows, vocab), device="cuda").exponential_(generator=g)
    t, p = torch.rand(rows, device="cuda", generator=g) + 0.5, torch.rand(rows, device="cuda", generator=g)
    for how in ({}, dict(temperature=t, top_p=p)):
        assert torch.equal(qmv.sample(x.expand(rows, -1), e, **how), qmv.sample(x.repeat(rows, 1), e, **how))
        assert torch.equal(qmv.sample(x.repeat(rows, 1), e[:1].expand(rows, -1), **how), qmv.sample(x.repeat(rows, 1), e[:1].repeat(rows, 1), **how))
        assert torch.equal(qmv.sample(x.expand(rows, -1), e[:1].expand(rows, -1), **how), qmv.sample(x.repeat(rows, 1), e[:1].repeat(rows, 1), **how))


def test_the_longest_row(qmv):
    """2^31 - 4097 ids, the most that there may be: a few stand out, at the row's ends."""
    import torch
    n = 2 ** 31 - 4097
    x = torch.full((1, n), -30.0, device="cuda")
    e = torch.ones((1, n), device="cuda")
    x[0, [n - 1, n - 2, 0, 2 ** 30 + 3]] = torch.tensor([0.5, 1.0, 0.75, 0.25], device="cuda")

    def one(**how):
        return qmv.sample(x, e, **{k: torch.tensor([v], dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in how.items()}).item()

    assert one() == one(temperature=0.0) == one(top_k=4) == one(top_p=0.9) == n - 2
    e[0, n - 1] = 1e-3
    assert one() == one(top_k=3) == one(top_k=5000) == one(min_p=0.5) == one(top_p=0.9999) == n - 1
    assert one(top_k=2) == one(min_p=0.7) == one(top_p=0.5) == n - 2  # (1 of 2.86 of the weight, 1.78 with the next)
    e[0, n - 3] = 1e-25  # -30 + 57.6: ahead of all where nothing is cut off
    assert one() == n - 3 and one(top_k=5000) == n - 1
    assert one(top_k=n - 1) == n - 1 and one(top_k=n) == n - 3  # (the highest id of the lowest logit is the last in order)
    del x, e
    torch.cuda.empty_cache()
