"""CPU-only checks of the MXFP4 entry points: bad arguments are refused on the host before any launch."""
import ctypes

import pytest

import moe_routed_expert_amd as m

P = ctypes.c_void_p
FAKE = P(0x1000)       # never dereferenced: every call below fails validation or has no work
ODD = P(0x1002)
BYTE = P(0x1001)


def quant(**kw):
    a = dict(x=FAKE, dt=0, stride=256, rows=4, n=128, act=1, rule=0, q=FAKE, q_stride=64, s=FAKE, s_stride=4, stream=None)
    a.update(kw)
    return m.lib().moe_mx4_quant(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), m.MOE_OK), (dict(rows=0, x=None, q=None, s=None), m.MOE_OK), (dict(n=0), m.MOE_OK),
    (dict(dt=3), m.MOE_ERR_DTYPE), (dict(dt=-1), m.MOE_ERR_DTYPE), (dict(act=6), m.MOE_ERR_SHAPE), (dict(act=-1), m.MOE_ERR_SHAPE),
    (dict(rule=2), m.MOE_ERR_SHAPE), (dict(rule=-1), m.MOE_ERR_SHAPE), (dict(rows=-1), m.MOE_ERR_SHAPE), (dict(n=-2), m.MOE_ERR_SHAPE),
    (dict(n=127), m.MOE_ERR_SHAPE), (dict(n=(1 << 30) + 2), m.MOE_ERR_SHAPE), (dict(x=None), m.MOE_ERR_NULL), (dict(q=None), m.MOE_ERR_NULL),
    (dict(s=None), m.MOE_ERR_NULL), (dict(stride=255), m.MOE_ERR_SHAPE), (dict(act=0, stride=127), m.MOE_ERR_SHAPE),
    (dict(q_stride=63), m.MOE_ERR_SHAPE), (dict(s_stride=3), m.MOE_ERR_SHAPE), (dict(x=BYTE), m.MOE_ERR_ALIGN),
    (dict(x=ODD, dt=1), m.MOE_ERR_ALIGN),
])
def test_quant_refusals(kw, want):
    assert quant(**kw) == want


def dequant(**kw):
    a = dict(q=FAKE, q_stride=64, s=FAKE, s_stride=4, rows=4, n=128, out=FAKE, dt=0, stride=128, stream=None)
    a.update(kw)
    return m.lib().moe_mx4_dequant(*a.values())


@pytest.mark.parametrize("kw,want", [
    (dict(rows=0), m.MOE_OK), (dict(n=0), m.MOE_OK), (dict(dt=3), m.MOE_ERR_DTYPE), (dict(rows=-1), m.MOE_ERR_SHAPE),
    (dict(n=127), m.MOE_ERR_SHAPE), (dict(q=None), m.MOE_ERR_NULL), (dict(s=None), m.MOE_ERR_NULL), (dict(out=None), m.MOE_ERR_NULL),
    (dict(q_stride=63), m.MOE_ERR_SHAPE), (dict(s_stride=3), m.MOE_ERR_SHAPE), (dict(stride=127), m.MOE_ERR_SHAPE),
    (dict(out=BYTE), m.MOE_ERR_ALIGN), (dict(out=ODD, dt=1), m.MOE_ERR_ALIGN),
])
def test_dequant_refusals(kw, want):
    assert dequant(**kw) == want


OPERANDS = dict(a=FAKE, a_stride=128, a_s=FAKE, a_s_stride=8, a_n=8, a_rows=None, w=FAKE, w_stride_e=128 * 128, w_stride_n=128,
                w_s=FAKE, w_s_stride_e=128 * 8, w_s_stride_n=8, n_experts=4)
REFUSED = [
    (dict(m_rows=0), m.MOE_OK), (dict(m_rows=0, a=None, w=None, out=None), m.MOE_OK),
    (dict(mode=2), m.MOE_ERR_SHAPE), (dict(K=240), m.MOE_ERR_SHAPE), (dict(K=0), m.MOE_ERR_SHAPE), (dict(K=(1 << 20) + 32), m.MOE_ERR_SHAPE),
    (dict(m_rows=-1), m.MOE_ERR_SHAPE), (dict(m_rows=2 ** 31), m.MOE_ERR_SHAPE), (dict(n_experts=-1), m.MOE_ERR_SHAPE),
    (dict(n_experts=0), m.MOE_ERR_SHAPE), (dict(n_experts=1025), m.MOE_ERR_SHAPE),
    (dict(a=None), m.MOE_ERR_NULL), (dict(a_s=None), m.MOE_ERR_NULL), (dict(w=None), m.MOE_ERR_NULL), (dict(w_s=None), m.MOE_ERR_NULL),
    (dict(out=None), m.MOE_ERR_NULL), (dict(offsets=None), m.MOE_ERR_NULL), (dict(mode=1, slots=None), m.MOE_ERR_NULL),
    (dict(mode=1, a_row_div=0), m.MOE_ERR_SHAPE), (dict(a_n=0), m.MOE_ERR_SHAPE), (dict(a_n=7), m.MOE_ERR_SHAPE),
    (dict(mode=1, a_row_div=2, a_n=3), m.MOE_ERR_SHAPE), (dict(a_stride=112), m.MOE_ERR_SHAPE), (dict(a_s_stride=4), m.MOE_ERR_SHAPE),
    (dict(w_stride_n=112), m.MOE_ERR_SHAPE), (dict(w_s_stride_n=4), m.MOE_ERR_SHAPE),
    (dict(w_stride_e=128 * 128 - 16), m.MOE_ERR_SHAPE), (dict(w_s_stride_e=128 * 8 - 4), m.MOE_ERR_SHAPE),
    (dict(K=160, a_s_stride=5), m.MOE_ERR_SHAPE),             # a scale row is read to its next multiple of four bytes
    (dict(a=ODD), m.MOE_ERR_ALIGN), (dict(w=ODD), m.MOE_ERR_ALIGN), (dict(a_s=ODD), m.MOE_ERR_ALIGN), (dict(w_s=ODD), m.MOE_ERR_ALIGN),
    (dict(a_stride=136), m.MOE_ERR_ALIGN), (dict(w_stride_n=136, w_stride_e=136 * 256), m.MOE_ERR_ALIGN),
    (dict(w_stride_e=256 * 128 + 8), m.MOE_ERR_ALIGN), (dict(a_s_stride=10), m.MOE_ERR_ALIGN),
    (dict(w_s_stride_n=10, w_s_stride_e=10 * 256), m.MOE_ERR_ALIGN), (dict(w_s_stride_e=256 * 8 + 2), m.MOE_ERR_ALIGN),
]


def gemm(**kw):
    a = dict(OPERANDS, N=128, K=256, mode=0, offsets=FAKE, slots=FAKE, m_rows=8, a_row_div=1, out=FAKE, out_dt=1, out_stride=128,
             stream=None)
    a.update(kw)
    return m.lib().moe_mx4_grouped_gemm(*a.values())


@pytest.mark.parametrize("kw,want", REFUSED + [
    (dict(out_dt=3), m.MOE_ERR_DTYPE), (dict(N=0), m.MOE_ERR_SHAPE), (dict(N=124), m.MOE_ERR_SHAPE), (dict(N=(1 << 20) + 8), m.MOE_ERR_SHAPE),
    (dict(out_stride=120), m.MOE_ERR_SHAPE), (dict(out=ODD), m.MOE_ERR_ALIGN), (dict(out=BYTE, out_dt=0), m.MOE_ERR_ALIGN),
    (dict(mode=1, m_rows=2 ** 24, a_n=2 ** 24), m.MOE_ERR_SHAPE),
])
def test_gemm_refusals(kw, want):
    assert gemm(**kw) == want


def fused(**kw):
    a = dict(OPERANDS, w_stride_e=256 * 128, w_s_stride_e=256 * 8, I=128, K=256, mode=0, offsets=FAKE, slots=FAKE, m_rows=8, a_row_div=1,
             act=1, rule=0, out=FAKE, q_stride=64, s=FAKE, s_stride=4, stream=None)
    a.update(kw)
    return m.lib().moe_mx4_grouped_gemm_act_quant(*a.values())


@pytest.mark.parametrize("kw,want", REFUSED + [
    (dict(act=0), m.MOE_ERR_SHAPE), (dict(act=6), m.MOE_ERR_SHAPE), (dict(rule=2), m.MOE_ERR_SHAPE), (dict(I=0), m.MOE_ERR_SHAPE),
    (dict(I=120), m.MOE_ERR_SHAPE), (dict(s=None), m.MOE_ERR_NULL), (dict(q_stride=63), m.MOE_ERR_SHAPE), (dict(s_stride=3), m.MOE_ERR_SHAPE),
    (dict(out=BYTE), m.MOE_ERR_ALIGN), (dict(q_stride=65), m.MOE_ERR_ALIGN), (dict(w_stride_e=255 * 128), m.MOE_ERR_SHAPE),
    (dict(mode=1, m_rows=2 ** 20, a_n=2 ** 20), m.MOE_ERR_SHAPE),
])
def test_fused_refusals(kw, want):
    assert fused(**kw) == want


def test_grouped_tile():
    seen = set()
    for R in (1, 8, 100, 1000, 4000, 20000):
        for E in (1, 8, 64, 256):
            for N in (8, 264, 1000, 2048, 8192):
                t = m.mx4_grouped_tile(R, E, N, 2048)
                assert t[0] in (32, 64, 128, 256) and t[1] in (64, 128, 256) and t == m.mx4_grouped_tile(R, E, N, 2048)
                seen.add(t)
    assert len(seen) > 2
    out = (ctypes.c_int32 * 2)()
    f = m.lib().moe_mx4_grouped_tile
    assert f(8, 4, 64, 64, None) == m.MOE_ERR_NULL
    for bad in ((0, 4, 64, 64), (8, 0, 64, 64), (8, 1025, 64, 64), (8, 4, 60, 64), (8, 4, 64, 48), (8, 4, 64, 0), (2 ** 31, 4, 64, 64)):
        assert f(*bad, out) == m.MOE_ERR_SHAPE
