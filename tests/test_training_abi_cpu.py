"""CPU-only checks of the training entry points: bad arguments are refused on the host before any launch."""
import ctypes

import pytest

import moe_routed_expert_amd as m

P = ctypes.c_void_p
FAKE = P(0x1000)       # never dereferenced: every call below fails validation or has no work
ODD = P(0x1002)


def gemm(**kw):
    a = dict(a=FAKE, a_stride=256, w=FAKE, w_stride_e=128 * 256, w_stride_r=256, n_experts=4, N=128, K=256, dt=0,
             w_trans=0, mode=0, expert_offsets=FAKE, slot_ids=FAKE, m_rows=8, a_row_div=1, out=FAKE, out_dt=1,
             out_stride=128, stream=None)
    a.update(kw)
    return m.lib().moe_b16_grouped_gemm(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(m_rows=0), m.MOE_OK), (dict(m_rows=0, a=None, w=None, out=None), m.MOE_OK),
    (dict(dt=1), m.MOE_ERR_DTYPE), (dict(dt=3), m.MOE_ERR_DTYPE), (dict(out_dt=3), m.MOE_ERR_DTYPE),
    (dict(mode=2), m.MOE_ERR_SHAPE), (dict(w_trans=2), m.MOE_ERR_SHAPE), (dict(w_trans=1, mode=1), m.MOE_ERR_SHAPE),
    (dict(N=0), m.MOE_ERR_SHAPE), (dict(N=124), m.MOE_ERR_SHAPE), (dict(K=252), m.MOE_ERR_SHAPE),
    (dict(K=0), m.MOE_ERR_SHAPE), (dict(N=(1 << 20) + 8), m.MOE_ERR_SHAPE), (dict(m_rows=-1), m.MOE_ERR_SHAPE),
    (dict(m_rows=2 ** 31), m.MOE_ERR_SHAPE), (dict(n_experts=0), m.MOE_ERR_SHAPE), (dict(n_experts=1025), m.MOE_ERR_SHAPE),
    (dict(n_experts=-1), m.MOE_ERR_SHAPE), (dict(out=None), m.MOE_ERR_NULL), (dict(a=None), m.MOE_ERR_NULL),
    (dict(w=None), m.MOE_ERR_NULL), (dict(expert_offsets=None), m.MOE_ERR_NULL),
    (dict(mode=1, m_rows=2 ** 24), m.MOE_ERR_SHAPE), (dict(mode=1, slot_ids=None), m.MOE_ERR_NULL), (dict(mode=1, a_row_div=0), m.MOE_ERR_SHAPE),
    (dict(a_stride=248), m.MOE_ERR_SHAPE), (dict(w_stride_r=248), m.MOE_ERR_SHAPE),
    (dict(w_stride_e=128 * 256 - 8), m.MOE_ERR_SHAPE), (dict(out_stride=120), m.MOE_ERR_SHAPE),
    (dict(w_trans=1, w_stride_r=120), m.MOE_ERR_SHAPE), (dict(w_trans=1, w_stride_r=128, w_stride_e=255 * 128), m.MOE_ERR_SHAPE),
    (dict(a=ODD), m.MOE_ERR_ALIGN), (dict(w=ODD), m.MOE_ERR_ALIGN), (dict(out=ODD), m.MOE_ERR_ALIGN),
    (dict(out=P(0x1001), out_dt=0), m.MOE_ERR_ALIGN), (dict(a_stride=260), m.MOE_ERR_ALIGN),
    (dict(w_stride_r=260, w_stride_e=260 * 128), m.MOE_ERR_ALIGN), (dict(w_stride_e=128 * 256 + 4), m.MOE_ERR_ALIGN),
])
def test_gemm_refusals(kw, want):
    assert gemm(**kw) == want


def test_grouped_tile():
    tiles = {(32, 64), (64, 64), (64, 256), (128, 256), (256, 256)}
    seen = set()
    for R in (1, 8, 100, 1000, 4000, 20000):
        for E in (1, 8, 64, 256):
            for N in (8, 264, 1000, 2048, 8192):
                t = m.b16_grouped_tile(R, E, N, 1024)
                assert t in tiles and t == m.b16_grouped_tile(R, E, N, 1024)
                seen.add(t)
    assert seen == tiles
    out = (ctypes.c_int32 * 2)()
    f = m.lib().moe_b16_grouped_tile
    assert f(8, 4, 64, 64, None) == m.MOE_ERR_NULL
    for bad in ((0, 4, 64, 64), (8, 0, 64, 64), (8, 1025, 64, 64), (8, 4, 60, 64), (8, 4, 64, 0), (2 ** 31, 4, 64, 64)):
        assert f(*bad, out) == m.MOE_ERR_SHAPE


def wgrad(**kw):
    a = dict(dy=FAKE, dy_stride=1024, dt=0, a=FAKE, a_stride=1024, a_dt=0, a_s=FAKE, a_s_stride=8, offsets=FAKE,
             n_experts=8, N=1024, K=1024, m_rows=8, dw=FAKE, dw_dt=1, dw_stride_e=1024 * 1024, dw_stride_n=1024,
             accumulate=0, workspace=None, ws_bytes=0, stream=None)
    a.update(kw)
    return m.lib().moe_b16_grouped_wgrad(*a.values())


LONG = dict(n_experts=1, N=128, K=128, m_rows=1 << 16, dy_stride=128, a_stride=128, dw_stride_n=128)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=1), m.MOE_ERR_DTYPE), (dict(a_dt=2), m.MOE_ERR_DTYPE), (dict(a_dt=1), m.MOE_ERR_DTYPE),
    (dict(dt=3, a_dt=3), m.MOE_ERR_DTYPE), (dict(dw_dt=3), m.MOE_ERR_DTYPE), (dict(N=1020), m.MOE_ERR_SHAPE),
    (dict(K=1020), m.MOE_ERR_SHAPE), (dict(a_dt=3, K=1016), m.MOE_ERR_SHAPE), (dict(n_experts=0), m.MOE_ERR_SHAPE),
    (dict(n_experts=1025), m.MOE_ERR_SHAPE), (dict(m_rows=-1), m.MOE_ERR_SHAPE), (dict(m_rows=2 ** 31), m.MOE_ERR_SHAPE),
    (dict(accumulate=2), m.MOE_ERR_SHAPE), (dict(dw=None), m.MOE_ERR_NULL), (dict(offsets=None), m.MOE_ERR_NULL),
    (dict(dy=None), m.MOE_ERR_NULL), (dict(a=None), m.MOE_ERR_NULL), (dict(a_dt=3, a_s=None), m.MOE_ERR_NULL),
    (dict(dy_stride=1016), m.MOE_ERR_SHAPE), (dict(a_stride=1016), m.MOE_ERR_SHAPE),
    (dict(a_dt=3, a_s_stride=7), m.MOE_ERR_SHAPE), (dict(dw_stride_n=1016), m.MOE_ERR_SHAPE),
    (dict(dw_stride_e=1024 * 1023), m.MOE_ERR_SHAPE), (dict(dy=ODD), m.MOE_ERR_ALIGN), (dict(a=ODD), m.MOE_ERR_ALIGN),
    (dict(dy_stride=1028), m.MOE_ERR_ALIGN), (dict(a_dt=3, a_stride=1032), m.MOE_ERR_ALIGN), (dict(dw=ODD), m.MOE_ERR_ALIGN),
    (dict(LONG), m.MOE_ERR_NULL), (dict(LONG, workspace=FAKE, ws_bytes=64), m.MOE_ERR_WORKSPACE),
    (dict(LONG, workspace=ODD, ws_bytes=1 << 30), m.MOE_ERR_ALIGN),
])
def test_wgrad_refusals(kw, want):
    assert wgrad(**kw) == want


def test_wgrad_workspace_size():
    size = m.b16_grouped_wgrad_workspace_size
    assert size(1 << 16, 1, 128, 128) > 0 and size(1 << 16, 1, 128, 128) % (128 * 128 * 4) == 0
    assert size(64, 1, 128, 128) == 0                 # short rows are not cut
    assert size(16384, 8, 8192, 4096) == 0            # enough tiles
    assert size(-1, 1, 128, 128) == 0 and size(8, 0, 128, 128) == 0 and size(8, 1, 130, 128) == 0


def save(**kw):
    a = dict(x=FAKE, dt=0, in_stride=512, rows=4, n=256, act=1, q=FAKE, q_stride=512, s=FAKE, s_stride=4, h=FAKE,
             h_stride=256, stream=None)
    a.update(kw)
    return m.lib().moe_act_checkpoint(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), m.MOE_OK), (dict(n=0), m.MOE_OK), (dict(dt=3), m.MOE_ERR_DTYPE), (dict(act=6), m.MOE_ERR_SHAPE),
    (dict(act=-1), m.MOE_ERR_SHAPE), (dict(act=0), m.MOE_ERR_SHAPE), (dict(rows=-1), m.MOE_ERR_SHAPE),
    (dict(n=-1), m.MOE_ERR_SHAPE), (dict(x=None), m.MOE_ERR_NULL), (dict(q=None), m.MOE_ERR_NULL),
    (dict(s=None), m.MOE_ERR_NULL), (dict(in_stride=511), m.MOE_ERR_SHAPE), (dict(q_stride=511), m.MOE_ERR_SHAPE),
    (dict(s_stride=3), m.MOE_ERR_SHAPE), (dict(h_stride=255), m.MOE_ERR_SHAPE), (dict(x=P(0x1001)), m.MOE_ERR_ALIGN),
    (dict(s=ODD), m.MOE_ERR_ALIGN), (dict(h=P(0x1001)), m.MOE_ERR_ALIGN),
])
def test_save_refusals(kw, want):
    assert save(**kw) == want


def use(**kw):
    a = dict(dh=FAKE, dt=0, dh_stride=256, q=FAKE, q_stride=512, s=FAKE, s_stride=4, rows=4, n=256, act=1, dx=FAKE,
             dx_stride=512, h=None, h_stride=0, stream=None)
    a.update(kw)
    return m.lib().moe_gated_act_backward(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), m.MOE_OK), (dict(n=0), m.MOE_OK), (dict(dt=3), m.MOE_ERR_DTYPE), (dict(act=0), m.MOE_ERR_SHAPE),
    (dict(act=6), m.MOE_ERR_SHAPE), (dict(dh=None), m.MOE_ERR_NULL), (dict(q=None), m.MOE_ERR_NULL),
    (dict(s=None), m.MOE_ERR_NULL), (dict(dx=None), m.MOE_ERR_NULL), (dict(dh_stride=255), m.MOE_ERR_SHAPE),
    (dict(q_stride=511), m.MOE_ERR_SHAPE), (dict(s_stride=3), m.MOE_ERR_SHAPE), (dict(dx_stride=511), m.MOE_ERR_SHAPE),
    (dict(h=FAKE, h_stride=255), m.MOE_ERR_SHAPE), (dict(dh=P(0x1001)), m.MOE_ERR_ALIGN), (dict(dx=P(0x1001)), m.MOE_ERR_ALIGN),
])
def test_use_refusals(kw, want):
    assert use(**kw) == want


def back(**kw):
    a = dict(dout=FAKE, dout_stride=256, y=FAKE, y_dt=0, y_stride=256, y_rows=32, slots=FAKE, route_rows=None,
             weights=FAKE, T=4, topk=8, H=256, dy=FAKE, dy_stride=256, dweights=FAKE, stream=None)
    a.update(kw)
    return m.lib().moe_topk_reduce_backward(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(T=0), m.MOE_OK), (dict(topk=0), m.MOE_OK), (dict(y_dt=3), m.MOE_ERR_DTYPE), (dict(T=-1), m.MOE_ERR_SHAPE),
    (dict(topk=1025), m.MOE_ERR_SHAPE), (dict(H=-1), m.MOE_ERR_SHAPE), (dict(y_rows=-1), m.MOE_ERR_SHAPE),
    (dict(T=2 ** 31), m.MOE_ERR_SHAPE), (dict(slots=None), m.MOE_ERR_NULL), (dict(weights=None), m.MOE_ERR_NULL),
    (dict(dout=None), m.MOE_ERR_NULL), (dict(dy=None), m.MOE_ERR_NULL), (dict(y=None), m.MOE_ERR_NULL),
    (dict(dout_stride=255), m.MOE_ERR_SHAPE), (dict(dy_stride=255), m.MOE_ERR_SHAPE), (dict(y_stride=255), m.MOE_ERR_SHAPE),
    (dict(dout=P(0x1001)), m.MOE_ERR_ALIGN), (dict(dy=P(0x1001)), m.MOE_ERR_ALIGN), (dict(y=P(0x1001)), m.MOE_ERR_ALIGN),
])
def test_reduce_backward_refusals(kw, want):
    assert back(**kw) == want


def test_router_backward_refusals():
    f = m.lib().moe_route_prep_backward
    assert f(None, None, None, 0, 8, 2, None, 8, None) == m.MOE_OK
    assert f(FAKE, FAKE, FAKE, 4, 1025, 2, FAKE, 1025, None) == m.MOE_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, 4, 0, 2, FAKE, 8, None) == m.MOE_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, 4, 8, 0, FAKE, 8, None) == m.MOE_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, 4, 8, 65, FAKE, 8, None) == m.MOE_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, -1, 8, 2, FAKE, 8, None) == m.MOE_ERR_SHAPE
    assert f(FAKE, FAKE, FAKE, 4, 8, 2, FAKE, 7, None) == m.MOE_ERR_SHAPE
    for i in range(3):
        a = [FAKE, FAKE, FAKE]
        a[i] = None
        assert f(*a, 4, 8, 2, FAKE, 8, None) == m.MOE_ERR_NULL
    assert f(FAKE, FAKE, FAKE, 4, 8, 2, None, 8, None) == m.MOE_ERR_NULL
