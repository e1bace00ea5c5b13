"""One workspace for every batch of up to the number of tokens that it was sized for."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E", [60, 256])
def test_a_workspace_serves_fewer_tokens(E):
    most, k = 16384, 4
    ws = torch.empty(m.router_workspace_size(most, E), dtype=torch.uint8, device=dev())
    x = torch.from_numpy(np.random.default_rng(E).standard_normal((most, E)).astype(np.float32)).to(dev())
    for T in (most, 8193, 8192, 4100, 65, 7):
        got, want = m.router(x[:T], k, score=m.MOE_SCORE_SIGMOID, workspace=ws), m.router(x[:T], k, score=m.MOE_SCORE_SIGMOID)
        assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5])), T
