"""qmv_sample's special rows and the borders of what it keeps, probed id by id."""
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
