"""qmv_kv_write and qmv_kv_read: the page rule bit for bit, appended tokens, ragged rows, strides, bad tables."""
import numpy as np
import pytest

import ops_ref
from helpers import dev_x

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


def make(qmv, lens, heads, dim, page, seed, extra=2):
    """An empty cache, its numpy twin and a shuffled table."""
    import torch
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + extra, max(max(need), 1) + 1
    order = np.random.default_rng(seed).permutation(pages)
    table = np.full((len(lens), width), -7, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return qmv.KvCache.empty(pages, heads, dim, page), ops_ref.Cache(pages, heads, page, dim), table, \
        torch.from_numpy(table).cuda()


def ints(v):
    import torch
    return torch.tensor(list(v), dtype=torch.int32, device="cuda")


def batch_of(qmv, td, lens, counts, max_rows=None, max_len=None):
    starts = np.concatenate([[0], np.cumsum(counts)])
    return qmv.KvBatch(td, ints(lens), starts=ints(starts), rows=int(starts[-1]),
                       max_rows=max(counts) if max_rows is None else max_rows,
                       max_len=max(lens) if max_len is None else max_len)


def rows_of(rng, n, heads, dim, bf16, amp=1.0):
    x = (amp * rng.standard_normal((n, heads, dim)) * (1 + 5 * (rng.random((n, heads, 1)) > 0.8))).astype(F)
    if not bf16:
        return x, dev_x(x)
    code = (x.view(np.uint32) >> 16).astype(np.uint16)
    return ops_ref.f32_of_bf16(code), dev_x(code)


def same(cache, twin):
    for i, (lev, sc) in enumerate(((cache.k, cache.k_scale), (cache.v, cache.v_scale))):
        assert np.array_equal(sc.cpu().numpy(), twin.scale[i])
        assert np.array_equal(lev.cpu().numpy(), twin.lev[i])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("dim,heads", [(64, 3), (128, 8), (256, 1)])
@pytest.mark.parametrize("bf16", [False, True])
def test_prompt_then_single_tokens(qmv, page, dim, heads, bf16):
    """A ragged prompt (a sequence without rows among them), then tokens one by one with growing
    magnitudes, so that pages are raised again and again."""
    rng = np.random.default_rng(page + dim)
    lens = [page * 2 + 5, 1, 0, page, page - 1]
    final = [n + 6 for n in lens]
    cache, twin, table, td = make(qmv, final, heads, dim, page, seed=dim)
    n = sum(lens)
    (k, kd), (v, vd) = rows_of(rng, n, heads, dim, bf16), rows_of(rng, n, heads, dim, bf16, 0.01)
    qmv.kv_write(cache, batch_of(qmv, td, lens, lens), kd, vd)
    twin.write(table, lens, lens, k, v)
    same(cache, twin)
    now = ints(lens)
    step = qmv.KvBatch(td, now, max_len=max(final))
    for t in range(6):
        lens = [x + 1 for x in lens]
        now += 1  # the batch's lengths are read when the call runs
        (k, kd), (v, vd) = rows_of(rng, 5, heads, dim, bf16, 1.3 ** t), rows_of(rng, 5, heads, dim, bf16, 0.01 * 2.0 ** -t)
        qmv.kv_write(cache, step, kd, vd)
        twin.write(table, lens, [1] * 5, k, v)
        same(cache, twin)
    # read back: everything, and the last tokens
    for counts in (lens, [min(x, 3) for x in lens]):
        for dtype in ("float32", "bfloat16"):
            import torch
            got = qmv.kv_read(cache, batch_of(qmv, td, lens, counts), getattr(torch, dtype))
            for which in range(2):
                ref = np.concatenate([twin.values(which, table[s], lens[s])[lens[s] - c:] for s, c in enumerate(counts)])
                if dtype == "bfloat16":
                    ref = torch.from_numpy(ref).bfloat16().float().numpy()
                assert np.array_equal(got[which].float().cpu().numpy(), ref)


@pytest.mark.parametrize("counts", [[40, 3], [1, 1], [0, 7]])
def test_rows_that_continue_a_page_and_strides(qmv, counts):
    """Rows that begin inside a page and end inside another; k and v as slices of a wider row."""
    import torch
    rng = np.random.default_rng(1)
    page, heads, dim = 16, 2, 64
    lens = [9, 30]
    final = [a + b for a, b in zip(lens, counts)]
    cache, twin, table, td = make(qmv, final, heads, dim, page, seed=2)
    for size, ls, amp in ((lens, lens, 1.0), (counts, final, 4.0)):
        n = sum(size)
        x = (amp * rng.standard_normal((n, 5 * heads, dim))).astype(F)
        xd = torch.from_numpy(x).cuda()
        qmv.kv_write(cache, batch_of(qmv, td, ls, size), xd[:, heads:2 * heads], xd[:, 3 * heads:4 * heads])
        twin.write(table, ls, size, x[:, heads:2 * heads], x[:, 3 * heads:4 * heads])
        same(cache, twin)


def test_round_trip_error_and_special_rows(qmv):
    """One raise moves an earlier value by half a step of the new scale at most; zero and tiny rows."""
    import torch
    page, heads, dim = 64, 2, 128
    cache, twin, table, td = make(qmv, [64], heads, dim, page, seed=9)
    rng = np.random.default_rng(4)
    xs = [np.zeros((4, heads, dim), F), np.full((1, heads, dim), 1e-35, F),
          rng.standard_normal((10, heads, dim)).astype(F), (3 * rng.standard_normal((10, heads, dim))).astype(F)]
    length, raises = 0, 0
    for x in xs:
        length += len(x)
        had = cache.k_scale.clone()
        qmv.kv_write(cache, batch_of(qmv, td, [length], [len(x)]), torch.from_numpy(x).cuda(), torch.from_numpy(-x).cuda())
        twin.write(table, [length], [len(x)], x, -x)
        same(cache, twin)
        raises += int((cache.k_scale > had).any())
    k, v = qmv.kv_read(cache, batch_of(qmv, td, [length], [length]), torch.float32)
    x = np.concatenate(xs)
    step = cache.k_scale.cpu().numpy()[table[0, 0]][None, :, None]
    assert raises == 2
    assert np.all(np.abs(k.cpu().numpy() - x) <= step * (0.5 * raises + 1e-4))
    assert torch.equal(v, -k)


def test_bad_tables_are_recorded_and_not_followed(qmv):
    import torch
    cache, twin, table, td = make(qmv, [40, 40], 2, 64, 16, seed=3)
    x = torch.ones((80, 2, 64), device="cuda")
    bad = td.clone()
    bad[0, 1] = cache.n_pages          # a page past the cache
    bad[1, 2] = -1
    good = batch_of(qmv, td, [40, 40], [40, 40])
    cases = [batch_of(qmv, bad, [40, 40], [40, 40]),
             batch_of(qmv, td, [40, 41], [40, 40], max_len=40),             # longer than stated
             batch_of(qmv, td, [40, 40], [40, 40], max_rows=39),            # more rows than stated
             batch_of(qmv, td, [40, 100], [40, 40], max_len=200),           # longer than its table
             batch_of(qmv, td, [40, 39], [40, 40]),                         # fewer tokens than rows
             batch_of(qmv, td, [-1, 40], [40, 40])]
    for b in cases:
        qmv.kv_write(cache, b, x, x)
        assert qmv.last_error() == 4
        qmv.kv_read(cache, b, torch.float32)
        assert qmv.last_error() == 4
        qmv.attend(cache, b, x.view(80, 2, 64))
        assert qmv.last_error() == 4
    b = batch_of(qmv, td, [40, 40], [40, 40])
    b.starts[2] = 81                                                        # rows past the call's
    qmv.kv_write(cache, b, x, x)
    assert qmv.last_error() == 4
    # pages that no row of the batch uses stayed as they were
    used = set(table[0, :3]) | set(table[1, :3])
    rest = [p for p in range(cache.n_pages) if p not in used]
    assert not cache.k[rest].any() and not cache.k_scale[rest].any()
    qmv.kv_write(cache, good, x, x)
    assert qmv.last_error() == 0


def test_long_cache_offsets_pass_32_bits(qmv):
    """Pages past 2^31 bytes of the pool, on a stream of their own."""
    import torch
    page, heads, dim = 128, 8, 256
    pages = (1 << 31) // (page * heads * dim) + 3
    cache = qmv.KvCache.empty(pages, heads, dim, page)
    td = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    x = torch.randn((130, heads, dim), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = batch_of(qmv, td, [130], [130])
    s.wait_stream(torch.cuda.current_stream())
    qmv.kv_write(cache, b, x, x, stream=s)
    k = torch.empty_like(x)
    v = torch.empty_like(x)
    s.wait_stream(torch.cuda.current_stream())
    qmv.kv_read(cache, b, k=k, v=v, stream=s)
    s.synchronize()
    step = float(cache.k_scale.max())
    assert float((k - x).abs().max()) <= step * 0.501 and torch.equal(k, v)
    assert not cache.k[1].any() and not cache.k[pages - 2].any()


@pytest.mark.parametrize("bf16", [False, True])
def test_scales_that_no_rows_give(qmv, bf16):
    """A page whose scale was set below 2^-110, and rows too small for one of their own: no levels."""
    import torch
    page, heads, dim = 32, 2, 128
    cache, twin, table, td = make(qmv, [12], heads, dim, page, seed=3)
    cache.k_scale.fill_(2.0 ** -120)
    cache.v_scale.fill_(2.0 ** -140)
    x = torch.full((8, heads, dim), 1e-31, device="cuda", dtype=torch.bfloat16 if bf16 else torch.float32)
    at = int(table[0, 0])
    for lev in (cache.k, cache.v):
        lev[at] = 5
    qmv.kv_write(cache, batch_of(qmv, td, [12], [8]), x, x)
    for lev, sc, d in ((cache.k, cache.k_scale, 2.0 ** -120), (cache.v, cache.v_scale, 2.0 ** -140)):
        assert bool((lev[at, :, 4:12] == 0).all()) and bool((lev[at, :, :4] == 5).all()) and bool((lev[at, :, 12:] == 5).all())
        assert bool((sc[at] == d).all())


def test_loose_bounds(qmv):
    """max_rows far above the call's rows (up to the type's largest), max_len the largest that is accepted."""
    import torch
    page, heads, dim = 16, 2, 64
    lens, counts = [700, 40, 1], [33, 1, 1]
    rng = np.random.default_rng(6)
    cache, twin, table, td = make(qmv, lens, heads, dim, page, seed=7)
    (k, kd), (v, vd) = rows_of(rng, 35, heads, dim, False), rows_of(rng, 35, heads, dim, False)
    qmv.kv_write(cache, batch_of(qmv, td, lens, counts), kd, vd)
    twin.write(table, lens, counts, k, v)
    same(cache, twin)
    tight = batch_of(qmv, td, lens, counts)
    want = qmv.kv_read(cache, tight, torch.float32)
    out = qmv.attend(cache, tight, kd)
    for max_rows, max_len in ((2 ** 31 - 1, 700), (2147483000, 2 ** 31 - 1025), (36, 2 ** 31 - 1025)):
        b = batch_of(qmv, td, lens, counts, max_rows=max_rows, max_len=max_len)
        qmv.kv_write(cache, b, kd, vd)  # the same rows again: nothing changes
        same(cache, twin)
        got = qmv.kv_read(cache, b, torch.float32)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert float((qmv.attend(cache, b, kd) - out).abs().max()) < 1e-4 * float(out.abs().max())
    assert qmv.last_error() == 0


@pytest.mark.parametrize("page,heads,dim", [(16, 2, 64), (64, 3, 128), (128, 1, 256)])
def test_levels_at_half_steps(qmv, page, heads, dim):
    """Values whose level depends on the product's own rounding: the rule rounds it before the half is added."""
    import torch
    rng = np.random.default_rng(page)
    cache, twin, table, td = make(qmv, [page], heads, dim, page, seed=1)
    k = np.empty((page, heads, dim), F)
    for h in range(heads):
        x = []
        while len(x) == 0:
            top = F(rng.uniform(0.5, 50))
            x = ops_ref.near_half(F(1) / F(top * F(1 / 127)))
        k[:, h] = rng.choice(np.concatenate([x, -x]), (page, dim))
        k[rng.integers(page), h, rng.integers(dim)] = top
    v = -k
    qmv.kv_write(cache, batch_of(qmv, td, [page], [page]), torch.from_numpy(k).cuda(), torch.from_numpy(v).cuda())
    twin.write(table, [page], [page], k, v)
    same(cache, twin)
