"""qmv_rmsnorm: float32, bfloat16 and 8-bit outputs against 64 bits and the runtime's quantizer rule."""
import numpy as np
import pytest

import ops_ref
from block_quantized_weight_q4_gb300 import inputs
from helpers import dev_x

pytestmark = pytest.mark.gpu
F = np.float32
# y against 64 bits: the rounding of s, of s w and of the last product (2^-24 each), and r's: a float32
# chain of at most 32 squares, 5 + 32 tree and warp additions, one division and one root
Y_TOL = (3 + (32 + 37) / 2 + 3) * 2.0 ** -24


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


def _case(rows, cols, bf16, seed, res=True, amp=1.0):
    r = np.random.default_rng(seed)
    x = (amp * r.standard_normal((rows, cols))).astype(F)
    if bf16:
        code = (x.view(np.uint32) >> 16).astype(np.uint16)
        xf, xd = ops_ref.f32_of_bf16(code), dev_x(code)
    else:
        xf, xd = x, dev_x(x)
    rs = (2 * amp * r.standard_normal((rows, cols))).astype(F) if res else None
    w = (1 + 0.2 * r.standard_normal(cols)).astype(F)
    return xf, xd, rs, w


def _image(qmv, y, rows, cols):
    raw = y.cpu().numpy()
    off = qmv.scale_offset(qmv.Q8_0, qmv.SCALE_F32, rows, cols)
    assert not raw[rows * cols:off].any()
    return raw[:rows * cols].view(np.int8).reshape(rows, cols), raw[off:].view(F).reshape(rows, cols // 32)


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 4096), (3, 96), (5, 1024), (2, 11008), (33, 256), (2, 16384 + 32),
                                       (1, 32768), (7, 8192)])
@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("out", ["f32", "bf16", "q8"])
def test_norm(qmv, rows, cols, bf16, out):
    import torch
    xf, xd, rs, w = _case(rows, cols, bf16, 7 * rows + cols)
    rd, wd = torch.from_numpy(rs).cuda(), torch.from_numpy(w).cuda()
    so = torch.full_like(rd, 9.0)
    y = qmv.rmsnorm(xd, wd, 1e-5, residual=rd, residual_out=so, out=out)
    s32 = (xf + rs).astype(F)
    assert np.array_equal(so.cpu().numpy(), s32)
    assert np.array_equal(rd.cpu().numpy(), rs)
    _, ref = ops_ref.rmsnorm(xf, rs, w, 1e-5)
    tol = Y_TOL
    if out == "q8":
        lev, d = _image(qmv, y, rows, cols)
        t = (s32 * w).astype(F).reshape(rows, -1, 32)
        top = np.abs(t).max(axis=2, keepdims=True)
        assert np.array_equal(lev.reshape(t.shape), ops_ref.q8_levels(t, (F(127) * (F(1) / top)).astype(F)))
        s = xf.astype(np.float64) + rs
        r = 1 / np.sqrt((s ** 2).mean(axis=1) + 1e-5)
        want = top[:, :, 0].astype(np.float64) / 127 * r[:, None]
        assert np.all(np.abs(d - want) <= Y_TOL * want)
        return
    got = y.float().cpu().numpy().astype(np.float64)
    bound = tol * np.abs(ref) + (2.0 ** -8 * np.abs(ref) if out == "bf16" else 0) + 1e-37
    assert np.all(np.abs(got - ref) <= bound)


@pytest.mark.parametrize("out", ["f32", "q8"])
def test_norm_without_residual_in_place_and_streams(qmv, out):
    import torch
    xf, xd, rs, w = _case(6, 512, False, 3)
    wd = torch.from_numpy(w).cuda()
    a = qmv.rmsnorm(xd, wd, 1e-6, out=out)
    z = torch.zeros_like(xd)
    b = qmv.rmsnorm(xd, wd, 1e-6, residual=z, residual_out=z, out=out)
    assert torch.equal(a, b) and torch.equal(z, xd)  # the update in place
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    c = qmv.rmsnorm(xd, wd, 1e-6, out=out, stream=s)
    s.synchronize()
    assert torch.equal(a, c)


def test_norm_zero_rows_and_blocks(qmv):
    import torch
    x = torch.zeros((3, 64), device="cuda")
    x[1, :32] = 1.5
    w = torch.ones(64, device="cuda")
    lev, d = _image(qmv, qmv.rmsnorm(x, w, 0.0, out="q8"), 3, 64)
    assert not lev[0].any() and not d[0].any() and not lev[2].any() and not d[2].any()
    assert (lev[1, :32] == 127).all() and not lev[1, 32:].any() and d[1, 1] == 0
    assert abs(d[1, 0] * 127 - 2 ** 0.5) < 1e-6
    assert qmv.rmsnorm(x[:0], w, out="f32").shape == (0, 64)


def test_norm_image_feeds_the_quantized_product(qmv):
    """The image is what matvec_qx reads: the product equals that of the dequantized rows."""
    import torch
    xf, xd, rs, w = _case(4, 1024, True, 11)
    rd, wd = torch.from_numpy(rs).cuda(), torch.from_numpy(w).cuda()
    xq = qmv.rmsnorm(xd, wd, residual=rd, out="q8")
    m = inputs.make_matrix(2, 1, 96, 1024, seed=5)
    Wd = torch.from_numpy(m.W).cuda()
    y = qmv.matvec_qx(2, 1, 96, 1024, Wd, xq, 4).cpu().double()
    a = qmv.dequant(qmv.Q8_0, qmv.SCALE_F32, 4, 1024, xq).cpu().double()
    wm = qmv.dequant(2, 1, 96, 1024, Wd).cpu().double()
    ref, mag = a @ wm.T, a.abs() @ wm.abs().T
    assert bool(((y - ref).abs() <= 1e-3 * mag).all())


def test_weights_written_before_the_norm(qmv):
    """Weights written by one kernel (a norm's 8-bit image is a Q8_0 / f32 matrix), a norm of the activations, then a product
    that asks for its weights early: it reads the new ones."""
    import torch
    rows, cols = 8192, 4096
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    src = [torch.randn((rows, cols), device="cuda", generator=g) for _ in range(2)]
    x = torch.randn((1, cols), device="cuda", generator=g)
    w = torch.ones(cols, device="cuda")
    h = qmv.rmsnorm(x, w, out="bf16")
    W = qmv.rmsnorm(src[0], w)
    want = []
    for s in src:
        qmv.rmsnorm(s, w, y=W)
        torch.cuda.synchronize()
        want.append(qmv.matvec(qmv.Q8_0, qmv.SCALE_F32, rows, cols, W, h))
        torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    got = [torch.empty((1, rows), device="cuda") for _ in range(100)]
    for i, y in enumerate(got):
        qmv.rmsnorm(src[i & 1], w, y=W)
        qmv.rmsnorm(x, w, out="bf16", y=h)
        qmv.matvec_grouped(qmv.Q8_0, qmv.SCALE_F32, [(rows, cols, W, h, y)], overlap=True)
    for i, y in enumerate(got):
        assert torch.equal(y, want[i & 1]), i


def test_image_levels_at_half_steps(qmv):
    """Values whose level depends on the product's own rounding: the rule rounds it before the half is added."""
    import torch
    rng = np.random.default_rng(2)
    rows, cols = 16, 1024
    x = np.empty((rows, cols // 32, 32), F)
    for r in range(rows):
        for b in range(cols // 32):
            near = []
            while len(near) == 0:
                top = F(rng.uniform(0.5, 50))
                near = ops_ref.near_half(F(127) * (F(1) / top))
            x[r, b] = rng.choice(np.concatenate([near, -near]), 32)
            x[r, b, 0] = top
    lev, _ = _image(qmv, qmv.rmsnorm(torch.from_numpy(x.reshape(rows, cols)).cuda(), torch.ones(cols, device="cuda")), rows, cols)
    inv = (F(127) * (F(1) / np.abs(x).max(axis=2, keepdims=True))).astype(F)
    assert np.array_equal(lev.reshape(x.shape), ops_ref.q8_levels(x, inv))
