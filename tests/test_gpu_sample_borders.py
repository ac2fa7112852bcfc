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
