"""Choices of the router that 32 bits cannot tell apart, or only just: ids against the float64 definition."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev

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


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("masked", [0.0, 0.6])
@pytest.mark.parametrize("T,E,topk,G,keep", [(30, 64, 8, 8, 3), (90, 256, 6, 8, 4), (20, 512, 8, 16, 5), (9, 1024, 9, 32, 7)])
def test_groups_of_nearly_equal_sums(score, with_bias, masked, T, E, topk, G, keep):
    """Groups in pairs that hold the same logits in another order, one of them off by an ulp or two or none; masked: groups of
    one choosable expert too."""
    rng = np.random.default_rng(E + T)
    size = E // G
    base = rng.standard_normal((T, G // 2, size)).astype(np.float32)
    base[rng.random(base.shape) < masked] = -np.inf
    b = rng.standard_normal((G // 2, size)).astype(np.float32) * 0.1
    x, bias = np.empty((T, G, size), np.float32), np.empty((G, size), np.float32)
    for p in range(G // 2):
        order = rng.permutation(size)
        x[:, 2 * p], bias[2 * p] = base[:, p], b[p]
        x[:, 2 * p + 1], bias[2 * p + 1] = base[:, p][:, order], b[p][order]
    off = rng.integers(-2, 3, T)
    top = x[:, 1].argmax(axis=1)
    for t in range(T):
        v = x[t, 1, top[t]]
        for _ in range(abs(off[t])):
            v = np.nextafter(v, np.float32(np.inf if off[t] > 0 else -np.inf))
        x[t, 1, top[t]] = v if np.isfinite(x[t, 1, top[t]]) else -np.inf
    check(x.reshape(T, E), topk, score, bias.reshape(E) if with_bias else None, G, keep, 2)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace (allocated by the call), many tokens and few."""
    rng = np.random.default_rng(5)
    xs = [torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dev()) for s in ((5000, 200), (9000, 300), (64, 64), (700, 1000))]
    want = [m.router(x, 5) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [m.router(x, 5, stream=s) for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g[:5], w[:5]))
