"""GPU tests of moe_b16_grouped_wgrad on 8-bit rows at the ends of the operand type's range."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import check, f64, offsets_of, randn, sum_bound

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32

# a matrix of few and one of many tiles, rows that stay whole and rows that are cut
SIZES = [([40, 0, 30], 72, 144), ([300], 2040, 4080), ([6001], 136, 80), ([1500, 1500], 1024, 512)]


@pytest.mark.parametrize("counts,N,K", SIZES)
def test_the_largest_fp16_rows_stay_finite(counts, N, K):
    """Every finite fp16 value has a finite place in the gradient: those from 63488 on (half a step of the 8-bit code
    below 65536 and more) are saved as 65536 and read as 65504."""
    R = sum(counts)
    print("largest fp16 rows R=%d N=%d K=%d" % (R, N, K), flush=True)
    tops = np.array([65504.0, 65472.0, 63520.0, 63488.0, 63456.0, 61440.0, 57344.0, 33000.0])
    x = randn((R, K), FP, 1)
    rng = np.random.default_rng(2)
    at = rng.integers(0, R, 200), rng.integers(0, K, 200)
    x[at] = torch.from_numpy((tops[rng.integers(0, 8, 200)] * rng.choice([-1.0, 1.0], 200))).half()
    x[0, :8] = torch.from_numpy(tops).half()
    q, s = torch.empty((R, K), dtype=torch.uint8, device=dev()), torch.empty((R, -(-K // 128)), device=dev())
    m.act_checkpoint(x.to(dev()), q, s)
    dy = randn((R, N), FP, 3, 0.01)
    dw = torch.empty((len(counts), N, K), dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy.to(dev()), q, to_dev(offsets_of(counts)), dw, a_s=s)
    torch.cuda.synchronize()
    v = f64(q.cpu().view(torch.float8_e4m3fn)) * np.repeat(f64(s), 128, axis=1)[:, :K]
    assert (np.abs(v) == 65536).sum() >= 4 and np.abs(v).max() == 65536
    v = np.clip(v, -65504, 65504)
    # a saved value is off by at most 2^-4 of it, and holding it in range adds nothing to that
    assert np.all(np.abs(v - f64(x)) <= 2.0 ** -4 * np.abs(f64(x)) + 2.0 ** -10 * np.repeat(f64(s), 128, axis=1)[:, :K])
    v16 = v.astype(np.float16).astype(np.float64)           # small values of a group with a large scale: fp16 holds them all
    ref, mag = tr.grouped_wgrad(f64(dy), v16, offsets_of(counts))
    check(dw, ref, sum_bound(max(counts) + 20, mag, F32)(ref), "gradient")


def test_values_past_fp16_are_held_and_nan_stays():
    """Rows saved from fp32 may hold more than fp16 does: held at its largest value; NaN stays NaN."""
    q = torch.full((1, 128), 0x38, dtype=torch.uint8, device=dev())     # 1.0
    q[0, 5], q[0, 7], q[0, 9], q[0, 11] = 0x7E, 0x7F, 0xFF, 0xFE        # 448, NaN, NaN, -448
    dy = torch.ones((1, 8), dtype=FP, device=dev())
    for scale in (128.0, 147.0, 65504.0, 65520.0, 2.0 ** 16, -(2.0 ** 16), 3e38):
        s = torch.full((1, 1), scale, device=dev())
        dw = torch.empty((1, 8, 128), dtype=F32, device=dev())
        m.b16_grouped_wgrad(dy, q, to_dev(np.array([0, 1], np.int32)), dw, a_s=s)
        got = f64(dw)[0, 0]
        assert np.isnan(got[7]) and np.isnan(got[9])
        assert got[0] == np.clip(scale, -65504, 65504)
        assert got[5] == np.clip(448 * scale, -65504, 65504) and got[11] == np.clip(-448 * scale, -65504, 65504)


@pytest.mark.parametrize("e", [-126, -125, -124, -123])
def test_the_least_scales(e):
    """code * scale is a bf16 value from a scale of 2^-124 on; below, it is rounded to bf16's least step, 2^-133."""
    rng = np.random.default_rng(0)
    codes = rng.integers(0, 256, (3, 256)).astype(np.uint8)
    codes[(codes & 0x7F) == 0x7F] = 1
    codes[0, :8] = [1, 2, 3, 0x81, 4, 5, 0x83, 8]                       # the smallest codes: multiples of 2^-9
    q, s = to_dev(codes), torch.full((3, 2), 2.0 ** e, device=dev())
    dy = torch.diag(torch.full((8,), 2.0 ** 100))[:3].to(BF)            # row r of the gradient is 2^100 times row r
    dw = torch.empty((1, 8, 256), dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy.to(dev()), q, to_dev(np.array([0, 3], np.int32)), dw, a_s=s)
    v = torch.from_numpy(codes).view(torch.float8_e4m3fn).double() * 2.0 ** e
    held = v.to(BF).double()
    assert torch.equal(held, v) == (e >= -124)
    assert np.array_equal(f64(dw)[0, :3], (held * 2.0 ** 100).numpy()) and not f64(dw)[0, 3:].any()
