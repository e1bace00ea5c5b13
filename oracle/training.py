"""Float64 definitions of the 16-bit grouped products and of the routed experts' backward pass (numpy).

Test infrastructure only, like the rest of the oracle: written from the formulas, sharing nothing with the HIP
library.  Functions that the tests bound element-wise also return the sum of the magnitudes of what they add.
"""
import numpy as np
from scipy.special import expit, ndtr


def grouped_gemm(a, w, offsets, trans=False):
    """out[r] = a[r] @ w[e].T (w [E, N, K]) or a[r] @ w[e] (w [E, K, N]), and sum_k |a| |w|."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    rows = int(offsets[-1])
    N = w.shape[2] if trans else w.shape[1]
    out, mag = np.zeros((rows, N)), np.zeros((rows, N))
    for e in range(w.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        m = w[e] if trans else w[e].T
        out[lo:hi] = a[lo:hi] @ m
        mag[lo:hi] = np.abs(a[lo:hi]) @ np.abs(m)
    return out, mag


def slot_gemm(a, w, slots, row_div):
    """Row r uses slot slots[r] and a row r // row_div; a slot outside the bank gives zeros."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    out, mag = np.zeros((len(slots), w.shape[1])), np.zeros((len(slots), w.shape[1]))
    for r, e in enumerate(slots):
        if 0 <= e < w.shape[0]:
            out[r] = w[e] @ a[r // row_div]
            mag[r] = np.abs(w[e]) @ np.abs(a[r // row_div])
    return out, mag


def grouped_wgrad(dy, a, offsets):
    """dW[e] = dy[rows].T @ a[rows], and sum_r |dy| |a|."""
    dy, a = np.asarray(dy, np.float64), np.asarray(a, np.float64)
    E = len(offsets) - 1
    out, mag = np.zeros((E, dy.shape[1], a.shape[1])), np.zeros((E, dy.shape[1], a.shape[1]))
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        out[e] = dy[lo:hi].T @ a[lo:hi]
        mag[e] = np.abs(dy[lo:hi]).T @ np.abs(a[lo:hi])
    return out, mag


def e4m3_round(t):
    """The e4m3 value nearest to t (|t| <= 448), ties to the even mantissa: step 2^(e - 3), least exponent -6."""
    t = np.asarray(t, np.float64)
    e = np.maximum(np.frexp(t)[1] - 1, -6)
    step = np.exp2(e - 3.0)
    return np.rint(t / step) * step


def save8(v):
    """(values of the codes, scales) of rows v: per 128 columns the smallest power of two s with max|v| / s <= 448,
    at least 2^-126 (0 for zeros); a non-finite value's code is NaN and its group's scale is the largest."""
    v = np.asarray(v, np.float64)
    rows, n = v.shape
    groups = (n + 127) // 128
    q, s = np.zeros((rows, n)), np.zeros((rows, groups))
    for j in range(groups):
        x = v[:, 128 * j:128 * (j + 1)]
        top = np.abs(x).max(axis=1)
        for r in range(rows):
            if top[r] == 0:
                continue
            k = -126
            while 2.0 ** k * 448 < top[r]:
                k += 1
            s[r, j] = 2.0 ** k
            q[r, 128 * j:128 * (j + 1)] = e4m3_round(x[r] / s[r, j])
    return q, s


def gate(act, g):
    """act(g) and its derivative, moe_act values 1..5."""
    g = np.asarray(g, np.float64)
    if act == 1:
        r = expit(g)
        return g * r, r * (1 + g * expit(-g))
    if act == 2:
        p = ndtr(g)
        return g * p, p + g * np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
    if act == 3:
        return np.maximum(g, 0), (g > 0).astype(np.float64)
    if act == 4:
        return expit(g), expit(g) * expit(-g)
    return g, np.ones_like(g)


def gated_act(act, x):
    n = x.shape[1] // 2
    return gate(act, x[:, :n])[0] * x[:, n:]


def gated_act_backward(act, x, dh):
    """[d gate | d up] of h = act(gate) * up."""
    n = x.shape[1] // 2
    f, d = gate(act, x[:, :n])
    return np.concatenate([dh * x[:, n:] * d, dh * f], axis=1)


def reduce(y, slots, weights, route_rows=None):
    T, k = slots.shape
    out = np.zeros((T, y.shape[1]))
    for t in range(T):
        for j in range(k):
            if slots[t, j] >= 0:
                out[t] += weights[t, j] * y[t * k + j if route_rows is None else route_rows[t * k + j]]
    return out


def reduce_backward(dout, y, slots, weights, route_rows=None):
    """dy (NaN where no route writes), dweights, and sum_h |dout| |y| per route."""
    T, k = slots.shape
    dy = np.full(y.shape, np.nan)
    dw, mag = np.zeros((T, k)), np.zeros((T, k))
    for t in range(T):
        for j in range(k):
            row = t * k + j if route_rows is None else route_rows[t * k + j]
            if slots[t, j] < 0 or not 0 <= row < y.shape[0]:
                if route_rows is None:
                    dy[row] = 0
                continue
            dy[row] = weights[t, j] * dout[t]
            dw[t, j] = dout[t] @ y[row]
            mag[t, j] = np.abs(dout[t]) @ np.abs(y[row])
    return dy, dw, mag


def route_weights(logits, ids):
    """The softmax over each token's selected logits."""
    l = np.take_along_axis(logits, ids, axis=1)
    p = np.exp(l - l.max(axis=1, keepdims=True))
    return p / p.sum(axis=1, keepdims=True)


def route_backward(ids, weights, dweights, E):
    T, k = ids.shape
    out = np.zeros((T, E))
    for t in range(T):
        mean = weights[t] @ dweights[t]
        for j in range(k):
            if 0 <= ids[t, j] < E:
                out[t, ids[t, j]] += weights[t, j] * (dweights[t, j] - mean)
    return out
