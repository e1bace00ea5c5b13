"""MXFP4 in numpy and float64: the format's values, its quantisation, and the bounds of products over it."""
import numpy as np
import torch

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
TIES = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])      # between neighbours; a tie goes to the even code
ACTS = {"silu": 1, "gelu": 2, "relu": 3, "sigmoid": 4, "mul": 5}


def decode(q, s):
    """Codes [..., k/2] and scale bytes [..., ceil(k/32)] (numpy uint8) as float64 values [..., k]."""
    code = np.stack([q & 15, q >> 4], axis=-1).reshape(*q.shape[:-1], -1)
    v = np.where(code >= 8, -1.0, 1.0) * GRID[code & 7]
    scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return v * np.repeat(scale, 32, axis=-1)[..., :v.shape[-1]]


def scale_bytes(amax, ceil):
    """Scale bytes of groups of largest magnitude amax (float64 of fp32 values)."""
    m, e = np.frexp(amax)                                     # amax = m 2^e, m in [0.5, 1)
    e = np.where(m <= 0.75, e - 3, e - 2) if ceil else e - 3
    b = np.clip(e + 127, 0, None)
    return np.where(np.isfinite(amax), np.where(amax == 0, 0, b), 255).astype(np.uint8)


def quantise(v, ceil=False):
    """(codes, scale bytes) of float64 rows of fp32 values [rows, n], n even."""
    rows, n = v.shape
    groups = -(-n // 32)
    p = np.zeros((rows, groups * 32))
    p[:, :n] = v
    p = p.reshape(rows, groups, 32)
    with np.errstate(invalid="ignore"):
        amax = np.where(np.isfinite(p).all(axis=2), np.abs(p).max(axis=2), np.nan)
    s = scale_bytes(amax, ceil)
    bad = (s == 255)[:, :, None]
    t = np.abs(np.where(bad, 0.0, p)) / np.exp2(np.where(s == 255, 127, s).astype(np.float64) - 127)[:, :, None]
    code = np.zeros(t.shape, np.uint8)
    for i, tie in enumerate(TIES):
        code += (t >= tie) if i % 2 else (t > tie)
    code = np.where(bad, 0, code + 8 * np.signbit(p)).astype(np.uint8).reshape(rows, -1)[:, :n]
    return code[:, 0::2] | (code[:, 1::2] << 4), s


def gate(act, g, u):
    """act(g) * u in float64."""
    from math import erfc
    g, u = np.asarray(g, np.float64), np.asarray(u, np.float64)
    if act == "silu":
        return g / (1 + np.exp(-g)) * u
    if act == "gelu":
        return g * 0.5 * np.vectorize(erfc)(-g / np.sqrt(2.0)) * u
    if act == "relu":
        return np.maximum(g, 0) * u
    if act == "sigmoid":
        return u / (1 + np.exp(-g))
    return g * u


def random_mx(rng, shape, lo=120, hi=126):
    """Random codes and scale bytes for elements [..., k]; scale rows padded to a multiple of 4 bytes with 255."""
    *lead, k = shape
    q = rng.integers(0, 256, (*lead, k // 2)).astype(np.uint8)
    s = rng.integers(lo, hi + 1, (*lead, k // 32)).astype(np.uint8)
    return q, s


def to_gpu(q, s):
    """Device tensors of codes and scales; a scale row's padding to four bytes holds 255, the NaN scale."""
    pad = -s.shape[-1] % 4
    wide = np.concatenate([s, np.full((*s.shape[:-1], pad), 255, np.uint8)], axis=-1)
    return torch.from_numpy(q).cuda(), torch.from_numpy(wide).cuda()[..., :s.shape[-1]]


def product_bound(K, mag):
    """|device - exact| of a sum over K: each MFMA of 128 products is within 2^-23 of the magnitudes it adds, its own and
    the accumulator's, which is at most mag; slot mode adds three sums more."""
    return (-(-K // 128) + 4) * 2.0 ** -23 * mag
