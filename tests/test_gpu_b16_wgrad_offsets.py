"""GPU tests of the weight gradient's offsets: those that decrease leave the gradient untouched, as the products do; those
that are clamped or leave rows out before the first expert do not."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import check, f64, randn, sum_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# rows, N, K: whole rows with each tile, then rows that are cut with each form of the join
SIZES = [(40, 72, 144), (300, 2040, 4080), (6000, 136, 80), (20000, 512, 768)]


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("bad", [(0, 0.8, 0.2, 1), (1, 0, 1, 1), (0.5, 0.5, 0.5, 0.4), (0, 1, -0.1, 1), (0, 1.5, 0.9, 1)])
@pytest.mark.parametrize("R,N,K", SIZES)
def test_decreasing_offsets_leave_the_gradient(R, N, K, bad, accumulate):
    dy, a = randn((R, N), BF, 1).to(dev()), randn((R, K), BF, 2).to(dev())
    offs = to_dev(np.array([int(x * R) for x in bad], np.int32))
    dw = torch.full((3, N, K), 9.0, dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy, a, offs, dw, accumulate=accumulate)
    torch.cuda.synchronize()
    assert bool((dw == 9).all())


def test_decreasing_offsets_of_many_experts():
    """The one decrease is the last of 1024, or in the middle."""
    E, R, N, K = 1024, 5000, 16, 16
    dy, a = randn((R, N), BF, 1).to(dev()), randn((R, K), BF, 2).to(dev())
    for at in (E, 500, 1):
        offs = np.linspace(3, R, E + 1).astype(np.int32)
        offs[at] = offs[at - 1] - 1
        dw = torch.full((E, N, K), 9.0, dtype=F32, device=dev())
        m.b16_grouped_wgrad(dy, a, to_dev(offs), dw)
        torch.cuda.synchronize()
        assert bool((dw == 9).all())


@pytest.mark.parametrize("R,N,K", SIZES)
def test_rows_before_the_first_and_offsets_past_the_rows(R, N, K):
    """Offsets need not start at 0 nor end at m_rows; past m_rows they are clamped, which decreases nothing."""
    dy, a = randn((R, N), BF, 1), randn((R, K), BF, 2)
    offs = np.array([7, R // 3, R // 3, R + 5, 2 * R], np.int32)
    dw = torch.full((4, N, K), 9.0, dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy.to(dev()), a.to(dev()), to_dev(offs), dw)
    torch.cuda.synchronize()
    ref, mag = tr.grouped_wgrad(f64(dy), f64(a), np.minimum(offs, R))
    check(dw, ref, sum_bound(R + 20, mag, F32)(ref), "gradient")
