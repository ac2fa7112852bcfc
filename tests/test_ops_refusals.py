"""The refusals of the operators between the products, on the host: every call here fails its checks or
has nothing to do, so nothing is launched."""
import ctypes

import pytest

from block_quantized_weight_q4_gb300 import binding
from block_quantized_weight_q4_gb300.build import build

OK, FORMAT, SHAPE, ARG, ALIGN = 0, 2, 3, 4, 5
P = 1 << 20  # an aligned address that nothing follows


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


@pytest.mark.parametrize("change,want", [
    (dict(x_dtype=2), FORMAT), (dict(out_dtype=5), FORMAT), (dict(rows=-1), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(cols=48), SHAPE), (dict(cols=0), SHAPE),
    (dict(cols=32800), SHAPE), (dict(rows=2 ** 40), SHAPE), (dict(x=None), ARG), (dict(weight=None), ARG),
    (dict(out=None), ARG), (dict(x=P + 8), ALIGN), (dict(residual=P + 4), ALIGN), (dict(residual_out=P + 4), ALIGN),
    (dict(weight=P + 4), ALIGN), (dict(out=P + 8), ALIGN), (dict(rows=0), OK), (dict(rows=0, x=None), OK)])
def test_rmsnorm(lib, change, want):
    a = dict(x_dtype=0, rows=2, cols=64, x=P, residual=P, residual_out=P, weight=P, eps=1e-5, out_dtype=16, out=P)
    a.update(change)
    assert lib.qmv_rmsnorm(a["x_dtype"], a["rows"], a["cols"], a["x"], a["residual"], a["residual_out"], a["weight"],
                           a["eps"], a["out_dtype"], a["out"], None) == want


def kv(change):
    cache = dict(k=P, v=P, k_scale=P, v_scale=P, n_pages=10, kv_heads=2, head_dim=64, page_tokens=16)
    batch = dict(page_table=P, table_stride=4, table_pages=4, kv_len=P, starts=P, n_seq=2, rows=5, max_rows=4, max_len=60)
    for key, v in change.items():
        (cache if key in cache else batch)[key] = v
    c, b = binding._KvCacheC(*cache.values()), binding._KvBatchC(*batch.values())
    return c, b


KV = [(dict(page_tokens=24), SHAPE), (dict(page_tokens=256), SHAPE), (dict(head_dim=96), SHAPE), (dict(head_dim=32), SHAPE),
      (dict(kv_heads=0), SHAPE), (dict(kv_heads=1025), SHAPE), (dict(n_pages=-1), SHAPE), (dict(n_pages=2 ** 31), SHAPE),
      (dict(n_seq=-1), ARG), (dict(rows=-1), ARG), (dict(max_rows=-1), ARG), (dict(max_len=-1), ARG),
      (dict(table_pages=-1), ARG), (dict(table_stride=3), SHAPE), (dict(n_seq=70000), SHAPE), (dict(rows=2 ** 31), SHAPE),
      (dict(starts=None), SHAPE), (dict(n_seq=0), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(k_scale=None), ARG),
      (dict(v_scale=None), ARG), (dict(page_table=None), ARG), (dict(kv_len=None), ARG), (dict(k=P + 8), ALIGN),
      (dict(v=P + 8), ALIGN), (dict(k_scale=P + 2), ALIGN), (dict(page_table=P + 2), ALIGN), (dict(kv_len=P + 2), ALIGN),
      (dict(starts=P + 1), ALIGN), (dict(rows=0), OK), (dict(max_rows=0), OK), (dict(rows=0, k=None), OK)]


@pytest.mark.parametrize("change,want", KV)
def test_cache_and_rows(lib, change, want):
    c, b = kv(change)
    cp, bp = ctypes.addressof(c), ctypes.addressof(b)
    stride = c.kv_heads * c.head_dim
    assert lib.qmv_kv_write(cp, bp, 0, P, max(stride, 128), P, max(stride, 128), None) == want
    assert lib.qmv_kv_read(cp, bp, 1, P, P, None) == want
    heads = 4 * c.kv_heads if c.kv_heads else 4
    assert lib.qmv_attend(cp, bp, heads, 1, P, heads * 256, 0.1, 1, 0, P, heads * 256, None) == want


def test_write_read_attend_arguments(lib):
    c, b = kv({})
    cp, bp = ctypes.addressof(c), ctypes.addressof(b)
    w = lambda xd=0, k=P, ks=128, v=P, vs=128, cc=cp, bb=bp: lib.qmv_kv_write(cc, bb, xd, k, ks, v, vs, None)  # noqa: E731
    assert w(xd=2) == FORMAT and w(cc=None) == ARG and w(bb=None) == ARG and w(k=None) == ARG and w(v=None) == ARG
    assert w(ks=127) == SHAPE and w(vs=64) == SHAPE and w(ks=2 ** 62) == SHAPE and w(k=P + 4) == ALIGN and w(ks=130) == ALIGN
    assert w(xd=1, ks=132) == ALIGN
    r = lambda od=0, k=P, v=P: lib.qmv_kv_read(cp, bp, od, k, v, None)  # noqa: E731
    assert r(od=16) == FORMAT and r(k=None) == ARG and r(v=P + 8) == ALIGN
    a = lambda heads=8, xd=1, q=P, qs=512, sc=0.1, win=0, o=P, os=512: lib.qmv_attend(  # noqa: E731
        cp, bp, heads, xd, q, qs, sc, 1, win, o, os, None)
    assert a(xd=2) == FORMAT and a(heads=3) == SHAPE and a(heads=0) == SHAPE and a(heads=70000) == SHAPE
    assert a(q=None) == ARG and a(o=None) == ARG and a(win=-1) == ARG and a(sc=float("inf")) == ARG and a(sc=float("nan")) == ARG
    c2, b2 = kv(dict(rows=2 ** 30, max_rows=1))
    assert lib.qmv_attend(ctypes.addressof(c2), ctypes.addressof(b2), 8, 1, P, 512, 0.1, 1, 0, P, 512, None) == SHAPE
    assert a(qs=500) == SHAPE and a(os=8) == SHAPE and a(q=P + 2) == ALIGN and a(qs=516) == ALIGN and a(o=P + 8) == ALIGN


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), ARG), (dict(n_given=-1), ARG), (dict(n_top=-1), ARG), (dict(vocab=0), SHAPE), (dict(vocab=2 ** 31), SHAPE),
    (dict(stride=99), SHAPE), (dict(n_top=33), SHAPE), (dict(vocab=3, n_top=4), SHAPE), (dict(n_given=65), SHAPE),
    (dict(logits=None), ARG), (dict(given=None), ARG), (dict(glp=None), ARG), (dict(ids=None), ARG), (dict(tlp=None), ARG),
    (dict(logits=P + 2), ALIGN), (dict(given=P + 4), ALIGN), (dict(glp=P + 2), ALIGN), (dict(ent=P + 1), ALIGN),
    (dict(ids=P + 2), ALIGN), (dict(tlp=P + 2), ALIGN), (dict(rows=0), OK), (dict(rows=2 ** 40), SHAPE)])
def test_logprobs(lib, change, want):
    a = dict(rows=2, vocab=100, logits=P, stride=100, given=P, n_given=1, glp=P, ent=P, n_top=4, ids=P, tlp=P)
    a.update(change)
    assert lib.qmv_logprobs(a["rows"], a["vocab"], a["logits"], a["stride"], a["given"], a["n_given"], a["glp"], a["ent"],
                            a["n_top"], a["ids"], a["tlp"], None) == want


def test_binding_checks_shapes():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        binding.KvCache(z((2, 1, 16, 64)), z((2, 1, 16, 64)), z((2, 1)), z((2, 1)))
    k = z((2, 1, 16, 64), dtype=torch.int8)
    with pytest.raises(ValueError):
        binding.KvCache(k, k, z((2, 2)), z((2, 1)))
    cache = binding.KvCache(k, k.clone(), z((2, 1)), z((2, 1)))
    i = lambda *s: z(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        binding.KvBatch(z((1, 2)), i(1))
    with pytest.raises(ValueError):
        binding.KvBatch(i(1, 2), i(2))
    with pytest.raises(ValueError):
        binding.KvBatch(i(1, 2), i(1), starts=i(2))  # rows missing
    b = binding.KvBatch(i(1, 2), i(1), starts=i(2), rows=3)
    with pytest.raises(ValueError):
        binding.kv_write(cache, b, z((3, 1, 64)), z((3, 1, 64)).bfloat16())
    with pytest.raises(ValueError):
        binding.kv_write(cache, b, z((2, 1, 64)), z((2, 1, 64)))
    with pytest.raises(ValueError):
        binding.attend(cache, b, z((3, 1, 128)))
    with pytest.raises(ValueError):
        binding.attend(cache, b, z((3, 64, 2)).transpose(1, 2))
    with pytest.raises(ValueError):
        binding.logprobs(z((2, 5), dtype=torch.float64))
    with pytest.raises(ValueError):
        binding.rmsnorm(z((2, 64)), z(63))
    with pytest.raises(ValueError):
        binding.rmsnorm(z((2, 64)), z(64), out="int8")
    with pytest.raises(ValueError):
        binding.rmsnorm(z((2, 64)), z(64), out="f32")  # not CUDA tensors
    with pytest.raises(TypeError):
        binding.rmsnorm(z((2, 64), dtype=torch.float16), z(64), out="f32")


@pytest.mark.parametrize("name", ["attend", "attend_prompt", "kv_cache", "logprobs", "norm"])
def test_dependents_start_after_the_wait(name):
    """QMV_FLAG_OVERLAP lets a product read its weights before it waits, so an operator that released it before its own wait
    would let it read weights that the kernel before the operator is still writing."""
    import os
    import re
    from block_quantized_weight_q4_gb300.build import CSRC
    text = open(os.path.join(CSRC, name + ".cu")).read()
    calls = re.findall(r"griddep_(wait|launch_dependents)\(\);", text)
    kernels = text.count("__global__")
    assert calls == ["wait", "launch_dependents"] * kernels


def test_operands_on_other_devices():
    """A tensor on the host, or on a device that is not the call's or not current, is refused before anything is launched:
    its address would be followed.  (Tensors that say they are on a device, so that this runs without one.)"""
    import torch

    class On(torch.Tensor):
        index = 0

        def get_device(self):
            return type(self).index

    class OnOther(On):
        index = 1

    def z(*shape, dtype=torch.float32, on=On):
        t = torch.zeros(shape, dtype=dtype)
        return t if on is None else t.as_subclass(on)

    i32 = torch.int32
    for bad in (None, OnOther):
        k = z(2, 1, 16, 64, dtype=torch.int8)
        with pytest.raises(ValueError, match="device"):
            binding.KvCache(k, z(2, 1, 16, 64, dtype=torch.int8, on=bad), z(2, 1), z(2, 1))
        with pytest.raises(ValueError, match="device"):
            binding.KvCache(k, k, z(2, 1), z(2, 1, on=bad))
        with pytest.raises(ValueError, match="device"):
            binding.KvBatch(z(1, 2, dtype=i32), z(1, dtype=i32, on=bad))
        with pytest.raises(ValueError, match="device"):
            binding.KvBatch(z(1, 2, dtype=i32), z(1, dtype=i32), starts=z(2, dtype=i32, on=bad), rows=3)
        cache = binding.KvCache(k, k, z(2, 1), z(2, 1))
        batch = binding.KvBatch(z(1, 2, dtype=i32), z(1, dtype=i32), starts=z(2, dtype=i32), rows=3)
        far = binding.KvBatch(z(1, 2, dtype=i32, on=bad), z(1, dtype=i32, on=bad), starts=z(2, dtype=i32, on=bad), rows=3)
        fc = binding.KvCache(*[t if bad is None else t.as_subclass(bad) for t in
                               (torch.zeros((2, 1, 16, 64), dtype=torch.int8), torch.zeros((2, 1, 16, 64), dtype=torch.int8),
                                torch.zeros(2, 1), torch.zeros(2, 1))])
        x, xb = z(3, 1, 64), z(3, 1, 64, on=bad)
        for call in (lambda: binding.kv_write(cache, batch, x, xb), lambda: binding.kv_write(cache, far, x, x),
                     lambda: binding.kv_write(fc, batch, x, x), lambda: binding.kv_read(cache, batch, k=x, v=xb),
                     lambda: binding.kv_read(cache, far, k=x, v=x), lambda: binding.attend(cache, far, x, out=x),
                     lambda: binding.attend(fc, batch, x, out=x), lambda: binding.attend(cache, batch, x, out=xb),
                     lambda: binding.rmsnorm(z(2, 64), z(64, on=bad), y=z(256, dtype=torch.uint8)),
                     lambda: binding.rmsnorm(z(2, 64), z(64), residual=z(2, 64, on=bad), y=z(256, dtype=torch.uint8)),
                     lambda: binding.rmsnorm(z(2, 64), z(64), residual_out=z(2, 64, on=bad), y=z(256, dtype=torch.uint8)),
                     lambda: binding.rmsnorm(z(2, 64), z(64), y=z(256, dtype=torch.uint8, on=bad)),
                     lambda: binding.logprobs(z(2, 5), z(2, 1, dtype=torch.int64, on=bad))):
            with pytest.raises(ValueError, match="one CUDA device"):
                call()


def test_operands_on_a_device_that_is_not_current(monkeypatch):
    import torch

    class On(torch.Tensor):
        def get_device(self):
            return 1

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    t = torch.zeros(2, 64).as_subclass(On)
    with pytest.raises(ValueError, match="current"):
        binding.rmsnorm(t, t[0], out="f32", y=t)
