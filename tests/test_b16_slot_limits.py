"""The slot form of the 16-bit products at the most rows that one call takes: both sides of the documented limit."""
import pytest
import torch

import moe_routed_expert_amd as m
from test_training_abi_cpu import gemm

SIDE = 1 << 24


@pytest.mark.parametrize("N,K,cols", [(16, 1024, 16), (24, 1024, 16), (8192, 1024, 16), (8, 1032, 8), (24, 1032, 8), (8192, 1032, 8)])
def test_rows_past_the_limit_are_refused(N, K, cols):
    strides = dict(N=N, K=K, a_stride=K, w_stride_r=K, w_stride_e=N * K, out_stride=N, mode=m.MOE_MODE_SLOT)
    groups = -(-N // cols)
    assert gemm(m_rows=-(-SIDE // groups), **strides) == m.MOE_ERR_SHAPE
    # one row fewer passes the sizes (the missing slots are looked for before the launch is formed, and nothing runs)
    assert gemm(m_rows=-(-SIDE // groups) - 1, slot_ids=None, **strides) == m.MOE_ERR_NULL


@pytest.mark.gpu
@pytest.mark.parametrize("N,K", [(16, 8), (8, 1032)])
def test_the_most_rows(N, K):
    from gpu_util import dev
    print("slot rows=%d N=%d K=%d" % (SIDE - 1, N, K), flush=True)
    a = torch.ones((1, K), dtype=torch.bfloat16, device=dev())
    w = torch.stack([torch.full((N, K), 2.0 ** -e, dtype=torch.bfloat16) for e in range(3)]).to(dev())
    slots = (torch.arange(SIDE - 1, device=dev(), dtype=torch.int32) % 4) - 1
    out = torch.full((SIDE - 1, N), 7.0, dtype=torch.bfloat16, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_SLOT, slot_ids=slots, a_row_div=SIDE)
    torch.cuda.synchronize()
    want = torch.tensor([0.0] + [K * 2.0 ** -e for e in range(3)], device=dev()).bfloat16()[(slots + 1).long()]
    assert bool((out == want[:, None]).all())
