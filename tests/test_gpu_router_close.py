"""Choices of the router that 32 bits cannot tell apart, or only just: ids against the float64 definition."""
import numpy as np
import pytest
import torch

from test_gpu_router import SIGMOID, SOFTMAX, check

pytestmark = pytest.mark.gpu


def close_logits(T, E, seed, kind):
    """fp32 logits: all the same; steps of one ulp; a few far apart among many close ones; saturated sigmoids."""
    rng = np.random.default_rng(seed)
    if kind == "same":
        return np.full((T, E), 0.37, np.float32)
    if kind == "ulps":
        return (np.float32(0.75) + rng.integers(0, 12, (T, E)) * np.float32(2.0 ** -24)).astype(np.float32)
    if kind == "mixed":
        x = rng.choice(np.array([-2.0, 0.3, 0.30000004, 0.3000001, 1.5], np.float32), (T, E))
        x[::3, : E // 2] = -np.inf                            # and experts that are masked
        return x
    return (30.0 + rng.integers(0, 9, (T, E))).astype(np.float32)   # saturated


@pytest.mark.parametrize("kind", ["same", "ulps", "mixed", "saturated"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,topk", [(3, 40, 33), (20, 64, 8), (70, 100, 7), (33, 300, 64), (5, 1024, 9), (17, 65, 1)])
def test_close(kind, with_bias, T, E, topk):
    # equal choices stay exactly equal in the reference: one bias for pairs of experts, apart by far more than 43 bits
    bias = (np.arange(E) // 2 % 5 * 2.0 ** -22).astype(np.float32) if with_bias else None
    check(close_logits(T, E, T + E, kind), topk, SIGMOID, bias, scale=1.5)


@pytest.mark.parametrize("kind", ["same", "ulps"])
@pytest.mark.parametrize("T,E,topk", [(3, 40, 33), (70, 256, 7), (9, 520, 64)])
def test_close_softmax(kind, T, E, topk):
    check(close_logits(T, E, E, kind), topk, SOFTMAX, None, renorm=False, scores=True)


@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,topk,G,keep", [(20, 64, 8, 8, 3), (70, 256, 6, 8, 4), (5, 512, 64, 64, 9), (66, 90, 4, 9, 2)])
def test_close_groups(top, T, E, topk, G, keep):
    check(close_logits(T, E, G, "mixed"), topk, SIGMOID, None, G, keep, top)
    check(close_logits(T, E, G, "ulps"), topk, SIGMOID, (np.arange(E) // 3 % 2 * 2.0 ** -21).astype(np.float32), G, keep, top)


@pytest.mark.parametrize("spread", [1e-30, 3e-38, 1e30, 3e38])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
def test_widest_and_narrowest_ranges(spread, score):
    """A range of logits that 22 bits cannot step, or whose steps leave fp32."""
    x = np.linspace(-1, 1, 37, dtype=np.float32)[None, :] * np.float32(spread)
    x = np.concatenate([x, -x, np.roll(x, 5, axis=1)])
    check(x, 6, score, None)
    check(torch.from_numpy(x).to(torch.bfloat16), 6, score, None, dt="bf16")


@pytest.mark.parametrize("big", [1e3, 1e20, 3e38])
def test_large_biases(big):
    """A bias that is far larger than every score leaves the others to 64 bits."""
    rng = np.random.default_rng(3)
    bias = np.zeros(130, np.float32)
    bias[::7] = big
    bias[5] = -big
    check(rng.standard_normal((21, 130)).astype(np.float32), 25, SIGMOID, bias)
