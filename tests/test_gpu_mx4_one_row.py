"""One row whose stride says nothing about its width, as a transposed column's does: torch calls it contiguous."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from mx4_util import random_mx, to_gpu

pytestmark = pytest.mark.gpu


def odd(t, cols=None):
    """A copy of the single row t as a view of a column's transpose, `cols` elements of memory behind it."""
    n = t.shape[1] if cols is None else cols
    column = torch.zeros((n, 1), dtype=t.dtype, device=dev())
    view = column.t()[:, :t.shape[1]]
    view.copy_(t)
    assert view.stride() == (1, 1)
    return view


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("n", [2, 34, 96, 712, 1024])
def test_quantised_and_read_back(act, n):
    x = torch.randn((1, n * (2 if act else 1)), device=dev()).bfloat16()
    q, s = (torch.zeros((1, c), dtype=torch.uint8, device=dev()) for c in (n // 2, -(-n // 32)))
    m.mx4_quant(x, q, s, act=act)
    oq, os = odd(torch.zeros_like(q)), odd(torch.zeros_like(s))
    m.mx4_quant(odd(x), oq, os, act=act)
    assert torch.equal(oq, q) and torch.equal(os, s)
    out, want = odd(torch.zeros((1, n), device=dev())), torch.zeros((1, n), device=dev())
    m.mx4_dequant(q, s, want)
    m.mx4_dequant(oq, os, out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("mode", [m.MOE_MODE_GROUPED, m.MOE_MODE_SLOT])
@pytest.mark.parametrize("K", [32, 160, 512])
def test_products(mode, K):
    rng = np.random.default_rng(K)
    aq, as_ = to_gpu(*random_mx(rng, (1, K)))
    wq, ws = to_gpu(*random_mx(rng, (2, 128, K)))
    how = dict(mode=mode, expert_offsets=torch.tensor([0, 0, 1], dtype=torch.int32, device=dev()),
               slot_ids=torch.ones(1, dtype=torch.int32, device=dev()))
    want, out = torch.zeros((1, 128), device=dev()), odd(torch.zeros((1, 128), device=dev()))
    m.mx4_grouped_gemm(aq, as_, wq, ws, want, **how)
    oq, os = odd(aq), odd(as_, -(-as_.shape[1] // 4) * 4)     # a scale row is readable to its next multiple of four bytes
    m.mx4_grouped_gemm(oq, os, wq, ws, out, **how)
    assert torch.equal(out, want)
    hq, hs = (torch.zeros((1, c), dtype=torch.uint8, device=dev()) for c in (32, 2))
    gq, gs = odd(torch.zeros_like(hq)), odd(torch.zeros_like(hs))
    m.mx4_grouped_gemm_act_quant(aq, as_, wq, ws, hq, hs, **how)
    m.mx4_grouped_gemm_act_quant(oq, os, wq, ws, gq, gs, **how)
    assert torch.equal(gq, hq) and torch.equal(gs, hs)
