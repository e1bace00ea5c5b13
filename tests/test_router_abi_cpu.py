"""CPU-only checks of the router's entry points: bad arguments are refused on the host before any launch."""
import ctypes

import pytest

import moe_routed_expert_amd as m

P = ctypes.c_void_p
FAKE = P(0x1000)       # never dereferenced: every call below fails validation or has no work
ODD = P(0x1002)


def router(**kw):
    a = dict(logits=FAKE, dt=1, stride=64, T=100, E=64, topk=8, score=1, bias=FAKE, n_group=8, topk_group=4, group_top=2, renorm=1,
             scale=1.0, ids=FAKE, weights=FAKE, scores=None, d2s=FAKE, rr=FAKE, offsets=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return m.lib().moe_router(*a.values())


INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, d2s=None, rr=None, offsets=None, logits=None, ids=None, weights=None), m.MOE_OK),
    (dict(dt=3), m.MOE_ERR_DTYPE), (dict(T=-1), m.MOE_ERR_SHAPE), (dict(T=(1 << 27) + 1), m.MOE_ERR_SHAPE), (dict(E=0), m.MOE_ERR_SHAPE),
    (dict(E=1025, stride=1025), m.MOE_ERR_SHAPE), (dict(topk=0), m.MOE_ERR_SHAPE), (dict(topk=65, stride=128, E=128), m.MOE_ERR_SHAPE),
    (dict(topk=64, T=1 << 26), m.MOE_ERR_SHAPE), (dict(score=2), m.MOE_ERR_SHAPE), (dict(score=-1), m.MOE_ERR_SHAPE),
    (dict(n_group=0), m.MOE_ERR_SHAPE), (dict(n_group=7), m.MOE_ERR_SHAPE), (dict(E=128, stride=128, n_group=128), m.MOE_ERR_SHAPE),
    (dict(topk_group=0), m.MOE_ERR_SHAPE), (dict(topk_group=9), m.MOE_ERR_SHAPE), (dict(topk=9, topk_group=1), m.MOE_ERR_SHAPE),
    (dict(group_top=0), m.MOE_ERR_SHAPE), (dict(group_top=3), m.MOE_ERR_SHAPE), (dict(renorm=2), m.MOE_ERR_SHAPE),
    (dict(scale=0.0), m.MOE_ERR_SHAPE), (dict(scale=-1.0), m.MOE_ERR_SHAPE), (dict(scale=INF), m.MOE_ERR_SHAPE), (dict(scale=NAN), m.MOE_ERR_SHAPE),
    (dict(logits=None), m.MOE_ERR_NULL), (dict(ids=None), m.MOE_ERR_NULL), (dict(weights=None), m.MOE_ERR_NULL),
    (dict(d2s=None), m.MOE_ERR_NULL), (dict(rr=None), m.MOE_ERR_NULL), (dict(offsets=None), m.MOE_ERR_NULL),
    (dict(T=0, offsets=None), m.MOE_ERR_NULL), (dict(stride=63), m.MOE_ERR_SHAPE), (dict(logits=ODD), m.MOE_ERR_ALIGN),
    (dict(logits=P(0x1001), dt=0), m.MOE_ERR_ALIGN), (dict(ws=None), m.MOE_ERR_NULL), (dict(ws=P(0x1008)), m.MOE_ERR_ALIGN),
    (dict(ws_bytes=64), m.MOE_ERR_WORKSPACE),
])
def test_router_refusals(kw, want):
    assert router(**kw) == want


def test_workspace_size():
    f = m.router_workspace_size
    assert f(0, 64) == 0 and f(64, 64) == 0 and f(100, 0) == 0 and f(100, 1025) == 0 and f((1 << 27) + 1, 8) == 0
    last = 0
    for T in (65, 1000, 8192, 100000, 1000000):
        size = f(T, 256)
        assert size % 256 == 0 and size >= last
        last = size
    assert f(8192, 256) < 1 << 20


def back(**kw):
    a = dict(logits=FAKE, dt=1, stride=64, ids=FAKE, weights=FAKE, dweights=FAKE, dscores=FAKE, ds_stride=64, T=10, E=64, topk=8, score=0,
             renorm=0, scale=1.0, dlogits=FAKE, d_stride=64, stream=None)
    a.update(kw)
    return m.lib().moe_router_backward(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), m.MOE_OK), (dict(T=0, logits=None, ids=None, dlogits=None), m.MOE_OK), (dict(dt=3), m.MOE_ERR_DTYPE),
    (dict(T=-1), m.MOE_ERR_SHAPE), (dict(E=0), m.MOE_ERR_SHAPE), (dict(E=1025, stride=1025), m.MOE_ERR_SHAPE), (dict(topk=65), m.MOE_ERR_SHAPE),
    (dict(topk=0), m.MOE_ERR_SHAPE), (dict(score=2), m.MOE_ERR_SHAPE), (dict(renorm=2), m.MOE_ERR_SHAPE), (dict(scale=0.0), m.MOE_ERR_SHAPE),
    (dict(scale=NAN), m.MOE_ERR_SHAPE), (dict(logits=None), m.MOE_ERR_NULL), (dict(ids=None), m.MOE_ERR_NULL),
    (dict(weights=None), m.MOE_ERR_NULL), (dict(dweights=None), m.MOE_ERR_NULL), (dict(dlogits=None), m.MOE_ERR_NULL),
    (dict(stride=63), m.MOE_ERR_SHAPE), (dict(d_stride=63), m.MOE_ERR_SHAPE), (dict(ds_stride=63), m.MOE_ERR_SHAPE),
    (dict(logits=ODD), m.MOE_ERR_ALIGN), (dict(dlogits=ODD), m.MOE_ERR_ALIGN),
])
def test_backward_refusals(kw, want):
    assert back(**kw) == want
