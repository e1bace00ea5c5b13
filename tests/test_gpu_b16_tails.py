"""GPU tests of the 16-bit products' last tiles where many experts have one: whole rounds of them."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from test_gpu_b16_gemm import BF, FP, F32, grouped

pytestmark = pytest.mark.gpu

# experts, rows, N: a round and a quarter of short last tiles behind five whole rounds, two rounds behind eight; then
# some of the experts end in long last tiles, in whole ones, or are empty
MANY = [(64, 1100, 0, 1032), (256, 1030, 0, 264), (64, 1150, 60, 1032), (48, 1300, 400, 1032)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("E,rows,spread,N", MANY)
def test_rounds_of_last_tiles(E, rows, spread, N, trans):
    rng = np.random.default_rng(E + spread)
    counts = [rows] * E if not spread else [int(c) for c in rows + rng.integers(-spread, spread + 1, E)]
    if spread:
        counts[3], counts[4], counts[-1] = 1024, 2 * rows, 0
        counts[5] += rows
    K = 72
    assert m.b16_grouped_tile(sum(counts), E, N, K) == (256, 256)
    grouped(counts, N, K, FP if spread else BF, F32 if spread else BF, trans, seed=E, extra=3)
