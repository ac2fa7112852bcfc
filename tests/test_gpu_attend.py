"""qmv_attend against softmax attention in 64 bits over the cache's own values."""
import numpy as np
import pytest

import ops_ref
from helpers import dev_x
from test_gpu_kv import batch_of, ints, make

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


def filled(qmv, lens, heads, dim, page, seed):
    """A cache whose pages hold random levels and scales over a wide range; what lies past a
    sequence's tokens is loud, and unused pages' scales are NaN."""
    import torch
    cache, twin, table, td = make(qmv, lens, heads, dim, page, seed)
    rng = np.random.default_rng(seed)
    for i in range(2):
        twin.lev[i][:] = rng.integers(-127, 128, twin.lev[i].shape, dtype=np.int8)
        twin.scale[i][:] = (2.0 ** rng.uniform(-9, -5, twin.scale[i].shape)).astype(F)
    used = {int(p) for s, n in enumerate(lens) for p in table[s, :-(-n // page)]}
    for i in range(2):
        twin.scale[i][[p for p in range(cache.n_pages) if p not in used]] = np.nan
    for t, a in ((cache.k, twin.lev[0]), (cache.v, twin.lev[1]), (cache.k_scale, twin.scale[0]), (cache.v_scale, twin.scale[1])):
        t.copy_(torch.from_numpy(a))
    return cache, twin, table, td


def queries(rng, rows, heads, dim, bf16, amp=1.0):
    x = (amp * rng.standard_normal((rows, heads, dim))).astype(F)
    if not bf16:
        return x, dev_x(x)
    code = (x.view(np.uint32) >> 16).astype(np.uint16)
    return ops_ref.f32_of_bf16(code), dev_x(code)


def check(twin, table, lens, counts, qf, got, scale, causal, window, bf16, what="", halves=False):
    got = got.float().cpu().numpy().astype(np.float64)
    row = 0
    for s, n in enumerate(counts):
        if n == 0:
            continue
        k, v = twin.values(0, table[s], lens[s]), twin.values(1, table[s], lens[s])
        ref, mag, amp = ops_ref.attend(qf[row:row + n], k, v, lens[s] - n, scale, causal, window)
        bound = ops_ref.attend_bound(mag, amp, ref, k.shape[2], lens[s], bf16)
        if halves:
            pages = np.asarray(table[s][: -(-lens[s] // twin.page)], np.int64)
            lev = np.moveaxis(twin.lev[1][pages], 1, 2).reshape(-1, v.shape[1], v.shape[2])[:lens[s]]
            sv = np.repeat(twin.scale[1][pages], twin.page, axis=0)[:lens[s]]
            bound = bound + ops_ref.half_weights(qf[row:row + n], k, lev, sv, lens[s] - n, scale, causal, window)
        err = np.abs(got[row:row + n] - ref)
        bad = ~(err <= bound)
        assert not bad.any(), (what, s, lens[s], n, int(bad.sum()), np.argwhere(bad)[0], float((err / bound).max()))
        row += n


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("heads,kvh,dim,page", [(32, 8, 128, 64), (4, 4, 64, 16), (14, 2, 64, 32), (8, 1, 128, 128),
                                                (2, 2, 256, 64), (16, 1, 128, 16), (24, 1, 64, 64), (12, 2, 256, 32)])
def test_single_tokens(qmv, heads, kvh, dim, page, bf16):
    """Lengths around pages and tiles, from one key on."""
    rng = np.random.default_rng(dim + heads)
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 700, 1531]
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=page)
    qf, qd = queries(rng, len(lens), heads, dim, bf16)
    b = qmv.KvBatch(td, ints(lens), max_len=max(lens))
    got = qmv.attend(cache, b, qd)
    check(twin, table, lens, [1] * len(lens), qf, got, dim ** -0.5, True, 0, bf16)
    again = qmv.attend(cache, b, qd)
    assert bool((got == again).all())  # no order of arrival in the result


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 5), (True, 100), (False, 0), (False, 33)])
@pytest.mark.parametrize("heads,kvh,dim,page", [(8, 2, 128, 64), (6, 6, 64, 16), (4, 1, 256, 32)])
def test_runs_of_tokens(qmv, heads, kvh, dim, page, causal, window, bf16):
    """Short and long runs of rows over cached tokens, ragged, one sequence without rows."""
    rng = np.random.default_rng(heads + window)
    lens = [5, 200, 64, 0, 333, 130]
    counts = [5, 3, 64, 0, 150, 129]
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=window)
    qf, qd = queries(rng, sum(counts), heads, dim, bf16)
    got = qmv.attend(cache, batch_of(qmv, td, lens, counts), qd, causal=causal, window=window)
    check(twin, table, lens, counts, qf, got, dim ** -0.5, causal, window, bf16)


@pytest.mark.parametrize("n,length", [(1, 20011), (4, 9000), (700, 2500), (257, 257), (128, 128), (1024, 1100)])
@pytest.mark.parametrize("dim", [64, 128])
def test_long(qmv, n, length, dim):
    rng = np.random.default_rng(n)
    cache, twin, table, td = filled(qmv, [length], 2, dim, 64, seed=n)
    qf, qd = queries(rng, n, 8, dim, True)
    got = qmv.attend(cache, batch_of(qmv, td, [length], [n]), qd)
    check(twin, table, [length], [n], qf, got, dim ** -0.5, True, 0, True)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 200), (False, 0), (False, 77)])
@pytest.mark.parametrize("heads,kvh,dim,page,lens,counts", [
    (32, 8, 128, 64, [700], [640]),                        # a chunk over cached tokens
    (16, 16, 64, 16, [513, 300, 0, 650, 1], [513, 299, 0, 400, 1]),
    (64, 8, 128, 128, [129, 257, 20], [129, 200, 20]),
    (24, 8, 64, 32, [1100, 900], [400, 500]),              # a group of three heads
])
def test_prompts(qmv, heads, kvh, dim, page, lens, counts, causal, window):
    """Many rows a sequence, ragged, with rows that fill no tile of 128."""
    rng = np.random.default_rng(dim + window)
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=page)
    qf, qd = queries(rng, sum(counts), heads, dim, True)
    b = batch_of(qmv, td, lens, counts)
    got = qmv.attend(cache, b, qd, causal=causal, window=window)
    check(twin, table, lens, counts, qf, got, dim ** -0.5, causal, window, True)
    again = qmv.attend(cache, b, qd, causal=causal, window=window)
    assert bool((got == again).all())


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1500), (False, 0)])
@pytest.mark.parametrize("heads,kvh,dim,page,lens,counts", [
    (8, 2, 128, 64, [5000], [256]),             # few blocks over many keys: each cut along them
    (32, 8, 64, 16, [2900], [130]),
    (8, 1, 128, 128, [3000, 40, 2111], [200, 40, 33]),
    (64, 16, 128, 64, [2100], [700]),           # whole blocks, and the rest cut
])
def test_prompts_cut_along_the_keys(qmv, heads, kvh, dim, page, lens, counts, causal, window):
    rng = np.random.default_rng(dim + window)
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=page)
    qf, qd = queries(rng, sum(counts), heads, dim, True)
    b = batch_of(qmv, td, lens, counts)
    got = qmv.attend(cache, b, qd, causal=causal, window=window)
    check(twin, table, lens, counts, qf, got, dim ** -0.5, causal, window, True)
    for _ in range(3):
        again = qmv.attend(cache, b, qd, causal=causal, window=window)
        assert bool((got == again).all())


def test_cut_prompts_in_captures(qmv):
    """Captured on a stream that has no workspace the blocks stay whole; after a call on the stream they are
    cut, in the capture too."""
    import torch
    rng = np.random.default_rng(21)
    lens, counts = [3000], [150]
    cache, twin, table, td = filled(qmv, lens, 2, 64, 64, seed=9)
    qf, qd = queries(rng, 150, 8, 64, True)
    b = batch_of(qmv, td, lens, counts)
    s = torch.cuda.Stream()
    got = []
    for _ in range(2):
        out = torch.empty_like(qd)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qmv.attend(cache, b, qd, out=out, stream=s)
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        check(twin, table, lens, counts, qf, out, 64 ** -0.5, True, 0, True)
        got.append(out)
        with torch.cuda.stream(s):
            again = qmv.attend(cache, b, qd, stream=s)
        torch.cuda.synchronize()
    assert bool((got[1] == again).all())


def test_many_sequences(qmv):
    """More sequences than a CTA scans at once, empty ones among them, on both kernels."""
    rng = np.random.default_rng(12)
    lens = [int(x) for x in rng.integers(0, 90, 300)]
    cache, twin, table, td = filled(qmv, lens, 2, 64, 16, seed=5)
    counts = [min(n, 1 + i % 3) for i, n in enumerate(lens)]
    qf, qd = queries(rng, sum(counts), 6, 64, True)
    got = qmv.attend(cache, batch_of(qmv, td, lens, counts), qd)
    check(twin, table, lens, counts, qf, got, 0.125, True, 0, True)
    lens = [int(x) for x in rng.integers(30, 200, 75)]
    counts = [min(n, 40) if i % 7 else 0 for i, n in enumerate(lens)]
    cache, twin, table, td = filled(qmv, lens, 8, 128, 64, seed=6)
    qf, qd = queries(rng, sum(counts), 64, 128, True)
    got = qmv.attend(cache, batch_of(qmv, td, lens, counts), qd)
    check(twin, table, lens, counts, qf, got, 128 ** -0.5, True, 0, True)


def test_nothing_to_do(qmv):
    """Sequences of length zero, and no rows at all."""
    import torch
    cache, twin, table, td = filled(qmv, [0, 40], 2, 64, 16, seed=5)
    out = torch.full((2, 4, 64), 3.0, device="cuda")
    b = batch_of(qmv, td, [0, 40], [0, 2])
    q = torch.zeros_like(out)
    qmv.attend(cache, b, q, out=out)
    v = torch.from_numpy(twin.values(1, table[1], 40)).cuda()
    want = torch.stack([v[:39].mean(0), v.mean(0)]).repeat_interleave(2, dim=1)
    assert float((out - want).abs().max()) < 1e-5  # equal scores: the mean of the values
    none = batch_of(qmv, td, [0, 40], [0, 0], max_rows=0)
    assert qmv.attend(cache, none, q[:0]).shape == (0, 4, 64)
    qmv.kv_write(cache, none, q[:0, :2], q[:0, :2])
    assert qmv.kv_read(cache, none)[0].shape == (0, 2, 64)


@pytest.mark.parametrize("scale", [-0.2, 2.0])
def test_prompts_scale_strides_and_growing_scores(qmv, scale):
    """Scores that grow along the keys (the running maximum moves at every tile), a negative scale, q and
    out as slices of wider rows."""
    import torch
    rng = np.random.default_rng(3)
    heads, kvh, dim, lens, counts = 32, 8, 128, [900, 640], [640, 640]
    cache, twin, table, td = filled(qmv, lens, kvh, dim, 32, seed=1)
    for s, n in enumerate(lens):
        for p in range(-(-n // 32)):
            twin.scale[0][table[s, p]] = 2.0 ** -12 * 1.3 ** p
    cache.k_scale.copy_(torch.from_numpy(twin.scale[0]))
    qf, qd = queries(rng, sum(counts), heads + 3, dim, True)
    out = torch.full((sum(counts), heads + 1, dim), 5.0, device="cuda", dtype=torch.bfloat16)
    qmv.attend(cache, batch_of(qmv, td, lens, counts), qd[:, 2:2 + heads], out=out[:, :heads], scale=scale)
    check(twin, table, lens, counts, qf[:, 2:2 + heads], out[:, :heads], scale, True, 0, True, halves=True)
    assert bool((out[:, heads:] == 5).all())


@pytest.mark.parametrize("bf16", [True, False])
def test_strides_scale_and_streams(qmv, bf16):
    """q a slice of a wider row, out a slice too, a scale of its own, another stream."""
    import torch
    rng = np.random.default_rng(8)
    lens, counts, dim = [100, 41], [33, 1], 64
    cache, twin, table, td = filled(qmv, lens, 2, dim, 32, seed=4)
    qf, qd = queries(rng, 34, 12, dim, bf16)
    out = torch.full((34, 10, dim), 7.0, device="cuda", dtype=qd.dtype)
    s = torch.cuda.Stream()
    b = batch_of(qmv, td, lens, counts)
    s.wait_stream(torch.cuda.current_stream())
    qmv.attend(cache, b, qd[:, 4:8], out=out[:, 2:6], scale=0.3, stream=s)
    s.synchronize()
    check(twin, table, lens, counts, qf[:, 4:8], out[:, 2:6], 0.3, True, 0, bf16)
    assert bool((out[:, :2] == 7).all()) and bool((out[:, 6:] == 7).all())


@pytest.mark.parametrize("bf16", [True, False])
@pytest.mark.parametrize("n", [1, 40])
def test_extreme_scales(qmv, bf16, n):
    """Pages whose values differ by powers of ten, all-zero pages, loud queries and one dominant key."""
    import torch
    rng = np.random.default_rng(2)
    lens = [310]
    cache, twin, table, td = filled(qmv, lens, 1, 128, 16, seed=6)
    used = table[0, :20]
    twin.scale[1][used[:, None], 0] = (10.0 ** rng.uniform(-12, 3, (20, 1))).astype(F)
    twin.scale[0][used[3]] = 0
    twin.scale[1][used[5]] = 0
    twin.lev[1][used[5]] = 0
    cache.k_scale.copy_(torch.from_numpy(twin.scale[0]))
    cache.v_scale.copy_(torch.from_numpy(twin.scale[1]))
    cache.v.copy_(torch.from_numpy(twin.lev[1]))
    for amp in (1e-6, 1.0, 20.0):
        qf, qd = queries(rng, n, 4, 128, bf16, amp)
        got = qmv.attend(cache, batch_of(qmv, td, lens, [n]), qd)
        check(twin, table, lens, [n], qf, got, 128 ** -0.5, True, 0, bf16, amp)
    twin.scale[1][used[:, None], 0] = 0
    twin.lev[1][used] = 0
    cache.v_scale.copy_(torch.from_numpy(twin.scale[1]))
    cache.v.copy_(torch.from_numpy(twin.lev[1]))
    assert not qmv.attend(cache, batch_of(qmv, td, lens, [n]), qd).any()


@pytest.mark.parametrize("warm", [False, True])
def test_in_a_graph(qmv, warm):
    """Captured on a stream that the library has not seen, or has (with its workspace), replayed after
    the lengths moved on."""
    import torch
    rng = np.random.default_rng(5)
    lens = [900, 77]
    cache, twin, table, td = filled(qmv, lens, 2, 128, 64, seed=8)
    qf, qd = queries(rng, 2, 8, 128, True)
    now = ints([850, 50])
    b = qmv.KvBatch(td, now, max_len=1000)
    out = torch.empty_like(qd)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    if warm:
        qmv.attend(cache, b, qd, out=out, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        qmv.attend(cache, b, qd, out=out)
    for ls in ([850, 50], lens):
        now.copy_(ints(ls))
        g.replay()
        torch.cuda.synchronize()
        check(twin, table, ls, [1, 1], qf, out, 128 ** -0.5, True, 0, True)


def hide(cache, twin, table, td, lens, counts, window, page, how):
    """What a server does with pages that a sliding window has left behind: their table entries cleared, or the pages
    given to something else (here scales that are no numbers).  Returns the table of the call."""
    import torch
    td = td.clone()
    for s, (n, m) in enumerate(zip(lens, counts)):
        gone = max(0, n - m - window + 1) // page  # pages that end before any row's first key
        if how == "cleared":
            td[s, :gone] = -1
        else:
            for scale in (cache.k_scale, cache.v_scale):
                scale[torch.from_numpy(table[s, :gone].astype(np.int64)).cuda()] = float(how)
    return td


@pytest.mark.parametrize("how", ["cleared", "nan", "inf"])
@pytest.mark.parametrize("window", [1, 20, 50, 100, 161, 300])
@pytest.mark.parametrize("heads,kvh,dim,page,lens,counts", [
    (8, 2, 128, 16, [40, 77, 330, 1000, 18, 551], [1, 1, 1, 1, 1, 1]),
    (4, 4, 64, 16, [300, 555, 1111, 90], [3, 1, 5, 2]),
    (4, 2, 256, 32, [200, 390, 1300], [1, 4, 9]),
    (8, 1, 128, 64, [333, 1000], [2, 1]),
    (32, 8, 128, 64, [900], [300]),              # from here on the prompt kernel
    (16, 16, 64, 16, [901, 500], [400, 300]),
    (32, 8, 64, 32, [1100], [333]),
    (64, 8, 128, 128, [1000, 700], [300, 200]),
])
def test_pages_that_the_window_hides(qmv, heads, kvh, dim, page, lens, counts, window, how):
    """Pages that no row of a sequence sees into may be anything: neither their table entries nor their scales count."""
    rng = np.random.default_rng(window)
    for bf16 in (True, False):
        cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=window)
        td = hide(cache, twin, table, td, lens, counts, window, page, how)
        qf, qd = queries(rng, sum(counts), heads, dim, bf16)
        got = qmv.attend(cache, batch_of(qmv, td, lens, counts), qd, window=window)
        assert qmv.last_error() == 0
        check(twin, table, lens, counts, qf, got, dim ** -0.5, True, window, bf16)


@pytest.mark.parametrize("how", ["cleared", "nan"])
def test_pages_that_the_window_hides_from_cut_prompts(qmv, how):
    """The same where the blocks are cut along the keys."""
    rng = np.random.default_rng(4)
    lens, counts, window, page = [4000], [130], 1500, 16
    cache, twin, table, td = filled(qmv, lens, 8, 128, page, seed=4)
    td = hide(cache, twin, table, td, lens, counts, window, page, how)
    qf, qd = queries(rng, 130, 32, 128, True)
    got = qmv.attend(cache, batch_of(qmv, td, lens, counts), qd, window=window)
    assert qmv.last_error() == 0
    check(twin, table, lens, counts, qf, got, 128 ** -0.5, True, window, True)


SCALE_SHAPES = [
    (16, 4, 128, 16, [1100], [500]),         # whole blocks on the prompt kernel
    (32, 8, 64, 64, [900, 700], [400, 300]),
    (8, 2, 128, 64, [5000], [256]),          # blocks cut along the keys
    (8, 2, 128, 128, [300, 64, 5], [1, 2, 1]),  # the kernel for few rows
]


@pytest.mark.parametrize("heads,kvh,dim,page,lens,counts", SCALE_SHAPES)
@pytest.mark.parametrize("amp,lo,hi", [(1e-6, -12, 3), (1.0, -12, 3), (20.0, -12, 3), (1.0, -25, -22), (1.0, 3, 20)])
@pytest.mark.parametrize("levels", [False, True])
def test_v_scales_decades_apart_and_zero_pages(qmv, heads, kvh, dim, page, lens, counts, amp, lo, hi, levels):
    """V scales over many powers of ten, down to values of 1e-23; pages of zero K, and of zero V with and without levels
    left in them: what a page of scale 0 holds is 0, and its keys weigh in the sum only."""
    import torch
    rng = np.random.default_rng(7)
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=3)
    for s, n in enumerate(lens):
        used = table[s, :-(-n // page)]
        twin.scale[1][used] = (10.0 ** rng.uniform(lo, hi, (used.size, kvh))).astype(F)
        for i, p in enumerate(used):
            if i % 5 == 2:
                twin.scale[1][p] = 0
                if not levels:
                    twin.lev[1][p] = 0
            if i % 7 == 3:
                twin.scale[0][p] = 0
    for t, a in ((cache.v, twin.lev[1]), (cache.k_scale, twin.scale[0]), (cache.v_scale, twin.scale[1])):
        t.copy_(torch.from_numpy(a))
    qf, qd = queries(rng, sum(counts), heads, dim, True, amp)
    b = batch_of(qmv, td, lens, counts)
    got = qmv.attend(cache, b, qd)
    check(twin, table, lens, counts, qf, got, dim ** -0.5, True, 0, True, halves=True)
    assert bool((got == qmv.attend(cache, b, qd)).all())


@pytest.mark.parametrize("heads,kvh,dim,page,lens,counts", SCALE_SHAPES)
def test_nothing_but_zero_pages(qmv, heads, kvh, dim, page, lens, counts):
    """Every V scale 0, the levels not: the output is 0 exactly."""
    rng = np.random.default_rng(8)
    cache, twin, table, td = filled(qmv, lens, kvh, dim, page, seed=3)
    cache.v_scale.zero_()
    _, qd = queries(rng, sum(counts), heads, dim, True)
    assert not qmv.attend(cache, batch_of(qmv, td, lens, counts), qd).any()
