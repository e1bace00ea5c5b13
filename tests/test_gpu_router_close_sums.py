"""Groups by the sum of their two largest choices, where a third one stands as close to them as the comparison's rounding."""
import numpy as np
import pytest

from test_gpu_router import SIGMOID, SOFTMAX, check

pytestmark = pytest.mark.gpu


def test_the_two_largest_are_summed():
    """Of the second group's choices the second (1 - 8.9e-14) and the third (1 - 1.5e-13) are one value in 43 bits, and the third has
    the lower index.  With the second its sum is 2 in 43 bits, as the first's and the fourth's are; with the third it is not."""
    x = np.full((3, 64), -20.0, np.float32)
    x[:, 16 + 15], x[:, 16 + 12], x[:, 16 + 11] = 68.78687286376953, 30.051692962646484, 29.555986404418945
    x[:, 48 + 7], x[:, 48 + 0], x[:, 48 + 2] = 34.97465515136719, 31.9409236907959, 30.14646339416504
    x[1, :3] = 42.0, 55.0, 47.0
    x[2, 11] = x[2, 12] = x[2, 13] = 40.0
    for keep in (1, 2, 3):
        check(x, 2, SIGMOID, None, 4, keep, 2)


# The choices' own arithmetic is the same here as on the device to their last bit: an exponential of 1e-11 or less is added to
# or divided into 1, where its last bits are lost.
@pytest.mark.parametrize("form", ["saturated", "saturated and biased", "softmax beside a bias of 1"])
@pytest.mark.parametrize("T,E,G,keep", [(60, 64, 4, 2), (90, 64, 8, 3), (20, 96, 3, 1), (40, 256, 8, 4), (12, 1024, 32, 9)])
def test_saturated_groups(form, T, E, G, keep):
    rng = np.random.default_rng(T + E + len(form))
    x = rng.uniform(26, 40, (T, E)).astype(np.float32)
    x[rng.random((T, E)) < 0.5] = -20.0
    bias = None if form == "saturated" else np.ones(E, np.float32)
    if form[1] == "o":
        x[:, E // 2] = 62.0
    check(x, 5, SOFTMAX if form[1] == "o" else SIGMOID, bias, G, keep, 2)
