"""The refusals of the operators around a decode step's products, on the host: every call here fails its checks or has nothing
to do, so nothing is launched."""
import ctypes

import pytest

from block_quantized_weight_q4_gb300 import binding
from block_quantized_weight_q4_gb300.build import build

OK, FORMAT, SHAPE, ARG, ALIGN = 0, 2, 3, 4, 5
P = 1 << 20  # an aligned address that nothing follows
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.load_library()


@pytest.mark.parametrize("change,want", [
    (dict(rows=-1), ARG), (dict(vocab=0), SHAPE), (dict(vocab=-5), SHAPE), (dict(vocab=2 ** 31 - 4096, stride=2 ** 31, ns=2 ** 31), SHAPE),
    (dict(stride=99), SHAPE), (dict(ns=99), SHAPE), (dict(rows=2 ** 29), SHAPE), (dict(stride=2 ** 62), SHAPE), (dict(ns=2 ** 62), SHAPE),
    (dict(logits=None), ARG), (dict(noise=None), ARG), (dict(ids=None), ARG), (dict(logits=P + 2), ALIGN), (dict(noise=P + 1), ALIGN),
    (dict(t=P + 2), ALIGN), (dict(k=P + 2), ALIGN), (dict(p=P + 2), ALIGN), (dict(m=P + 2), ALIGN), (dict(ids=P + 4), ALIGN), (dict(rows=0), OK),
    (dict(rows=0, logits=None), OK)])
def test_sample(lib, change, want):
    a = dict(rows=2, vocab=100, logits=P, stride=100, noise=P, ns=100, t=P, k=P, p=P, m=P, ids=P)
    a.update(change)
    assert lib.qmv_sample(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(wt=3), FORMAT), (dict(sd=2), FORMAT), (dict(od=16), FORMAT), (dict(vocab=0), SHAPE), (dict(cols=48), SHAPE), (dict(cols=0), SHAPE),
    (dict(vocab=2 ** 40, cols=2 ** 30), SHAPE), (dict(rows=-1), ARG), (dict(scale=INF), ARG), (dict(scale=NAN), ARG), (dict(W=None), ARG),
    (dict(ids=None), ARG), (dict(out=None), ARG), (dict(W=P + 8), ALIGN), (dict(ids=P + 4), ALIGN), (dict(out=P + 8), ALIGN), (dict(rows=2 ** 62), SHAPE),
    (dict(rows=2 ** 40), SHAPE), (dict(rows=0), OK), (dict(rows=0, W=None), OK)])
def test_embed(lib, change, want):
    a = dict(wt=2, sd=1, vocab=100, cols=64, W=P, ids=P, rows=3, scale=1.0, od=0, out=P)
    a.update(change)
    assert lib.qmv_embed(*a.values(), None) == want


@pytest.mark.parametrize("change,want", [
    (dict(xd=2), FORMAT), (dict(od=16), FORMAT), (dict(pairs=2), FORMAT), (dict(rows=-1), ARG), (dict(eps=-1.0), ARG), (dict(eps=NAN), ARG),
    (dict(eps=INF), ARG), (dict(factor=NAN), ARG), (dict(factor=INF), ARG), (dict(heads=0), SHAPE), (dict(heads=65536), SHAPE), (dict(kvh=-1), SHAPE),
    (dict(dim=96), SHAPE), (dict(dim=512), SHAPE), (dict(rot=8), SHAPE), (dict(rot=80), SHAPE), (dict(rot=-16), SHAPE), (dict(rows=2 ** 31), SHAPE),
    (dict(qs=255), SHAPE), (dict(ks=64), SHAPE), (dict(qos=128), SHAPE), (dict(kos=127), SHAPE), (dict(qs=2 ** 62), SHAPE), (dict(q=None), ARG),
    (dict(k=None), ARG), (dict(qo=None), ARG), (dict(ko=None), ARG), (dict(pos=None), ARG), (dict(freq=None), ARG), (dict(q=P + 8), ALIGN),
    (dict(qs=257), ALIGN), (dict(k=P + 4), ALIGN), (dict(qo=P + 8), ALIGN), (dict(ko=P + 8), ALIGN), (dict(qw=P + 4), ALIGN), (dict(kw=P + 4), ALIGN),
    (dict(pos=P + 2), ALIGN), (dict(freq=P + 2), ALIGN), (dict(xd=1, qs=260), ALIGN), (dict(rows=0), OK), (dict(rows=0, q=None), OK)])
def test_qk_rope(lib, change, want):
    a = dict(xd=0, rows=2, heads=4, kvh=2, dim=64, q=P, qs=256, k=P, ks=128, qw=P, kw=P, eps=1e-6, pos=P, freq=P, rot=64, pairs=1, factor=1.0, od=0,
             qo=P, qos=256, ko=P, kos=128)
    a.update(change)
    assert lib.qmv_qk_rope(*a.values(), None) == want


LAYER = dict(wt13=2, wt2=2, sd=1, experts=8, dim=128, hidden=64, W1=P, W3=P, W2=P)


@pytest.mark.parametrize("change,want", [
    (dict(wt13=0), FORMAT), (dict(wt2=3), FORMAT), (dict(sd=2), FORMAT), (dict(experts=0), SHAPE), (dict(experts=257, stride=257), SHAPE), (dict(dim=96), SHAPE),
    (dict(dim=0), SHAPE), (dict(dim=2 ** 24), SHAPE), (dict(hidden=32), SHAPE), (dict(hidden=2 ** 24), SHAPE), (dict(W1=None), ARG), (dict(W3=None), ARG),
    (dict(W2=None), ARG), (dict(W1=P + 8), ALIGN), (dict(W2=P + 8), ALIGN), (dict(tokens=-1), ARG), (dict(stride=7), SHAPE), (dict(top=0), SHAPE),
    (dict(top=9), SHAPE), (dict(experts=64, stride=64, top=17), SHAPE), (dict(scale=NAN), ARG), (dict(scale=INF), ARG), (dict(act=2), FORMAT), (dict(xd=2), FORMAT), (dict(od=16), FORMAT),
    (dict(logits=None), ARG), (dict(x=None), ARG), (dict(out=None), ARG), (dict(scratch=None), ARG), (dict(logits=P + 2), ALIGN), (dict(x=P + 8), ALIGN),
    (dict(out=P + 8), ALIGN), (dict(ids=P + 2), ALIGN), (dict(shares=P + 2), ALIGN), (dict(scratch=P + 8), ALIGN), (dict(tokens=2 ** 60), SHAPE),
    (dict(stride=2 ** 62), SHAPE), (dict(tokens=0), OK), (dict(tokens=0, x=None), OK)])
def test_moe(lib, change, want):
    layer = {**LAYER, **{k: v for k, v in change.items() if k in LAYER}}
    a = dict(tokens=2, logits=P, stride=8, top=2, renorm=1, scale=1.0, act=0, xd=1, x=P, od=0, out=P, ids=None, shares=None, scratch=P)
    a.update({k: v for k, v in change.items() if k not in LAYER})
    c = binding._MoeC(*layer.values())
    assert lib.qmv_moe(ctypes.addressof(c), *a.values(), None) == want
    assert lib.qmv_moe(None, *a.values(), None) == ARG


def test_moe_scratch(lib):
    f = lib.qmv_moe_scratch_bytes
    # h's halves and two factors for each 32 of them (twice for float32 outputs) and the routing, for a block of at most 64 tokens
    assert f(1, 2, 64, 0) > 2 * 2 * (64 * 2 + 2 * 8) and f(64, 4, 128, 1) > 64 * 4 * (128 * 2 + 4 * 8) and f(64, 4, 128, 1) == f(1000, 4, 128, 1)
    assert f(-1, 1, 64, 0) == 0 and f(1, 0, 64, 0) == 0 and f(1, 17, 64, 0) == 0 and f(1, 1, 65, 0) == 0 and f(1, 1, 64, 16) == 0
