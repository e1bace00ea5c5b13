"""Weights of a token whose chosen logits lie further apart than fp32 reaches, and the order of its widest logits."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev

from test_gpu_router import SIGMOID, SOFTMAX, check

pytestmark = pytest.mark.gpu
INF, LOW, TOP = np.inf, float(np.finfo(np.float32).min), float(np.finfo(np.float32).max)
BF16_TOP = float(torch.finfo(torch.bfloat16).max)


def widest(E):
    """Every pair of these logits in one token is more than fp32's largest value apart, or masked; the others are small."""
    rows = [[INF, LOW], [LOW, INF], [3e38, -3e38], [2e38, -2e38], [-1e38, INF], [TOP, LOW, -INF, np.nan], [INF, INF, LOW, LOW],
            [-INF, LOW, 3e38, -3e38], [LOW, LOW], [INF, -3e38, 3e38, LOW, 1e30, -1e30]]
    x = np.tile(np.linspace(-2, 2, E, dtype=np.float32), (len(rows), 1))
    x[:, 60:] = -np.inf                                         # at most 64 experts are chosen: these too
    for t, r in enumerate(rows):
        x[t, :len(r)] = r
    return x


# A weight here is 0 (a difference of 1e30 or more under the exponential), or a ratio of numbers of ordinary size, within check's bound.
@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E,topk", [(8, 8), (40, 40), (100, 64)])
def test_weights_of_logits_far_apart(dt, score, renorm, E, topk):
    r = check(widest(E), topk, score, renorm=renorm, scale=1.5, scores=True, dt=dt)
    assert torch.isfinite(r.weights).all() and not torch.signbit(r.weights).any()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_two_routes_far_apart(score):
    """The largest logits only: every weight goes to the larger one (softmax), or by their scores 1 and 0 (sigmoid)."""
    x = torch.tensor([[3e38, -3e38], [LOW, INF], [2e38, -2e38]], device=dev())
    for renorm in (True, False):
        r = m.router(x, 2, score=score, renorm=renorm)
        assert r.weights.tolist() == [[1.0, 0.0]] * 3 and r.expert_ids.tolist() == [[0, 1], [1, 0], [0, 1]]


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("with_groups", [False, True])
@pytest.mark.parametrize("T,E,topk", [(3, 16, 1), (5, 64, 6), (70, 96, 12), (4, 1024, 3)])
def test_infinity_goes_before_the_largest_finite_logit(dt, with_groups, T, E, topk):
    """+inf counts as fp32's largest value, which is above bf16's and fp16's largest finite one (and equal to fp32's)."""
    top = {"bf16": BF16_TOP, "fp16": 65504.0, "fp32": TOP}[dt]
    x = np.zeros((T, E), np.float32)
    x[:, ::2] = top
    x[:, 3::4] = INF
    x[T // 2, E // 2:] = INF
    x[T // 2, :E // 2] = top
    check(x, topk, SOFTMAX, G=4 if with_groups else 1, keep=2 if with_groups and topk > 1 else 1, top=1, dt=dt)
