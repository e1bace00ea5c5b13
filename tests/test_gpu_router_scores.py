"""The router's scores and weights over their whole range: the bounds that its header states."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev

from test_gpu_router import DTS, SIGMOID, SOFTMAX, reference, scores64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("T,E,std", [(40, 64, 1.0), (40, 64, 30.0), (70, 200, 12.0), (20, 1024, 25.0), (33, 513, 300.0)])
def test_bounds(dt, score, T, E, std):
    """In units of 2^-24.  A softmax score: the exponent d log2 e is off by 2.22 of itself (the difference's rounding 1, the constant
    0.22, the product's 1), which is 2.22 d of the exponential, and that 2; the sum of them 2.22 of the mean distance, which is ln E
    < 7 at most, and 2, and 22 additions; its reciprocal and the product 2: 2.22 d + 44.  A sigmoid: 1.22 d + 8.  A weight: 4 of its
    own exponential, that of the renormalised sum 4 and 10 additions or the softmax's sum 40, divisions and products 3 to 6: 64."""
    x = torch.from_numpy((np.random.default_rng(T + E).standard_normal((T, E)) * std).astype(np.float32)).to(DTS[dt])
    x[::7, : E // 2] = -float("inf")
    v, k = x.double().numpy(), 8
    s, shown = scores64(v, score)
    there = shown > -np.inf
    d = np.where(there, np.abs(shown) if score == SIGMOID else shown.max(axis=1, keepdims=True) - shown, 0.0)
    for renorm in (True, False):
        r = m.router(x.to(dev()), k, score=score, renorm=renorm, scale=2.0, want_scores=True)
        got = r.scores.cpu().double().numpy()
        assert (np.abs(got - s) <= (2.5 * d + 48) * U * s + 2.0 ** -126).all()
        ids, w, _ = reference(v, k, score, None, 1, 1, 1, renorm, 2.0)
        got = r.weights.cpu().double().numpy()
        assert np.array_equal(r.expert_ids.cpu().numpy(), ids) and (np.abs(got - w) <= 64 * U * w + 2.0 ** -125).all()
