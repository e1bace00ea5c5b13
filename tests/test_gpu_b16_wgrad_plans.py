"""Every tile of the weight gradient, with whole and with cut rows, over both operand types, 16- and 8-bit rows, gradients
written and added on, aligned and not.  The plan itself is asserted, so a problem that comes to be taken differently shows."""
import ctypes

import pytest
import torch

import moe_routed_expert_amd as m
from test_gpu_b16_wgrad import BF, FP, F32, wgrad

# tile, rows of a chunk, counts, N, K: N and K end inside a tile, counts inside a step, some experts are empty
PLANS = [((128, 128), 0, [130, 0, 255, 129, 64], 72, 144), ((128, 128), 256, [1500, 0, 600], 72, 80),
         ((256, 128), 0, [70, 0, 130], 1032, 2064), ((256, 128), 256, [9000, 0, 9000], 136, 272),
         ((256, 256), 0, [3, 100, 0, 197], 2056, 1040), ((256, 256), 1024, [15000, 8000, 0, 1000], 136, 2064)]


def plan_of(counts, N, K):
    p = m.b16_grouped_wgrad_plan(sum(counts), len(counts), N, K)
    return p[:2], p[2]


@pytest.mark.parametrize("tile,chunk,counts,N,K", PLANS)
def test_plans(tile, chunk, counts, N, K):
    assert plan_of(counts, N, K) == (tile, chunk)
    size = m.b16_grouped_wgrad_workspace_size(sum(counts), len(counts), N, K)
    assert size == ((sum(counts) // chunk + len(counts)) * N * K * 4 if chunk else 0)


def test_plan_refusals():
    out = (ctypes.c_int32 * 3)()
    f = m.lib().moe_b16_grouped_wgrad_plan
    assert f(8, 4, 64, 64, None) == m.MOE_ERR_NULL
    for bad in ((-1, 4, 64, 64), (8, 0, 64, 64), (8, 1025, 64, 64), (8, 4, 60, 64), (8, 4, 64, 0), (2 ** 31, 4, 64, 64)):
        assert f(*bad, out) == m.MOE_ERR_SHAPE
    assert f(0, 4, 64, 64, out) == m.MOE_OK and out[2] == 0


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("dt,odt", [(BF, F32), (FP, F32), (FP, FP), (BF, BF)])
@pytest.mark.parametrize("tile,chunk,counts,N,K", PLANS)
def test_every_form_of_a_plan(tile, chunk, counts, N, K, dt, odt, saved, accumulate):
    assert plan_of(counts, N, K) == (tile, chunk)
    wgrad(counts, N, K, dt, odt, saved, seed=N + K, accumulate=accumulate)


@pytest.mark.gpu
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("odt,pad", [(BF, 1), (F32, 1), (FP, 4), (F32, 2)])
@pytest.mark.parametrize("tile,chunk,counts,N,K", PLANS[:5])
def test_every_plan_with_unaligned_output(tile, chunk, counts, N, K, odt, pad, accumulate, monkeypatch):
    import test_gpu_b16_wgrad as t
    guarded = t.Guarded
    monkeypatch.setattr(t, "Guarded", lambda shape, dt: guarded(shape, dt, pad=pad))
    wgrad(counts, N, K, BF, odt, False, seed=N + K + 1, accumulate=accumulate)
