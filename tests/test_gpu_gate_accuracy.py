"""GPU tests of the gated activations and their slopes far from zero, where their values are small: the error is bounded
relative to each value, as a gradient that is scaled up afterwards sees it."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from oracle import training as tr
from train_util import HALF, NAMES, TINY, check, f64

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def far_gates():
    """Both signs of every e4m3 mantissa from 2^-6 to 120: exact in 8 bits, so forward and backward see the same gate."""
    g = np.array([(1 + k / 8) * 2.0 ** e for e in range(-6, 7) for k in range(8)])
    return np.concatenate([-g[g <= 120][::-1], [0.0], g[g <= 120]])


def gate_errors(act, g, dt):
    """Bounds on the error of act(g) and act'(g) in fp32: relative to each value, or to the terms of a slope that is a sum,
    plus what may be flushed to 0.

    sigmoid: with t = e^-|g| and q = 1 / (1 + t), act is q or t q and the slope t q^2.  t: to 16 bits the exponent
    |g| log2 e carries a relative 2^-23 (the constant's rounding and the product's), so |g| 2^-23 in t, and the hardware
    exp2 an ulp: (|g| + 1) 2^-23; to fp32 expf 2 ulp, 2^-22.  q: the sum 2^-24, the reciprocal 2^-23 (fp32: the division
    2^-24), and t / (1 + t) of t's error, which takes away from that of the products.  Each product 2^-24.
    gelu: act is g Phi(g), the slope Phi(g) + g phi(g).  Phi's lower tail, to 16 bits e R: the exponent's three roundings
    are 1.5 z^2 / 2 2^-23, exp2 2^-23, R 10 2^-24 (3.5e-7 measured over all z, and the reciprocal's ulp), two products; to
    fp32 erfcf 16 ulp and its argument's 2^-23, which z^2 + 1 multiplies.  1 - tail: 2^-24 more.  phi: the exponential
    (fp32: 2 ulp and z^2 / 2 2^-24 from the exponent), the constant and a product."""
    a, (f, d) = np.abs(g), tr.gate(act, g)
    if act == 2:
        dens = np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
        et = (0.75 * a * a + 7) * 2 * U if dt != F32 else (a * a + 18) * 2 * U
        ed = (0.75 * a * a + 2) * 2 * U if dt != F32 else a * a * U / 2 + 6 * U
        ep = et * tr.gate(2, -a)[0] / np.where(a > 0, -a, 1) + np.where(a > 0, 0, et / 2)     # Phi(-|g|)
        ep = ep + np.where(g >= 0, 2 * U, 0) + 2.0 ** -126
        return a * ep + U * np.abs(f), ep + a * (ed * dens + 2.0 ** -126) + U * (a * dens + np.abs(d))
    if act == 4:
        et, eq = ((a + 1) * 2 * U, 3 * U) if dt != F32 else (4 * U, 2 * U)
        return (et + eq + U) * f + 2.0 ** -126, (et + 2 * eq + 2 * U) * d + 2.0 ** -126
    raise ValueError(act)


@pytest.mark.parametrize("act", [2, 4])
@pytest.mark.parametrize("dt", [BF, FP, F32])
def test_gates_far_from_zero(dt, act):
    print("gates act=%d %s" % (act, NAMES[dt]), flush=True)
    gates, n = far_gates(), 8
    rows = len(gates)
    up = 2.0 ** np.array([0, 4, 6, 8, -3, 5, 3, 1])                     # powers of two: exact in every type
    x = np.concatenate([np.repeat(gates[:, None], n, 1), np.repeat(up[None], rows, 0)], 1)
    xd = torch.from_numpy(x).to(dt).to(dev())
    q, s = torch.empty((rows, 2 * n), dtype=torch.uint8, device=dev()), torch.empty((rows, 2), device=dev())
    h, h2 = (torch.empty((rows, n), dtype=dt, device=dev()) for _ in range(2))
    m.act_checkpoint(xd, q, s, act=act, h=h)
    dh = 2.0 ** np.array([0, 3, 5, 4, 6, 1, 2, 0])
    dx = torch.empty((rows, 2 * n), dtype=dt, device=dev())
    m.gated_act_backward(torch.from_numpy(np.repeat(dh[None], rows, 0)).to(dt).to(dev()), q, s, dx, act=act, h=h2)
    torch.cuda.synchronize()
    g, u = x[:, :n], x[:, n:]
    f, d = tr.gate(act, g)
    ef, ed = gate_errors(act, g, dt)

    def bound(ref, err):
        # the products with up and dh are with powers of two: exact
        return err + HALF[dt] * (np.abs(ref) + err) + TINY[dt] + 2.0 ** -148

    for got in (h, h2):
        check(got, f * u, bound(f * u, ef * u), "h")
    check(dx, np.concatenate([dh * u * d, dh * f], 1),
          np.concatenate([bound(dh * u * d, ed * dh * u), bound(dh * f, ef * dh)], 1), "dx")


@pytest.mark.parametrize("act", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("n", [8, 5])
def test_a_nan_gate_is_not_lost(n, dt, act):
    """An overflow upstream has to stay visible behind every activation, in the forward pass and in the gradients."""
    x = torch.full((3, 2 * n), 2.0, dtype=dt)
    x[1, 3], x[2, :n] = float("nan"), -1.0
    q, s = torch.empty((3, 2 * n), dtype=torch.uint8, device=dev()), torch.empty((3, 2), device=dev())
    h, h2, dx = (torch.empty((3, w), dtype=dt, device=dev()) for w in (n, n, 2 * n))
    m.act_checkpoint(x.to(dev()), q, s, act=act, h=h)
    m.gated_act_backward(torch.ones((3, n), dtype=dt, device=dev()), q, s, dx, act=act, h=h2)
    torch.cuda.synchronize()
    want = np.zeros((3, n), bool)
    want[1, 3] = True
    for got in (h, h2, dx[:, n:]):
        assert np.array_equal(~np.isfinite(f64(got)), want)
    assert np.array_equal(~np.isfinite(f64(dx[:, :n])), want & (act != 5))
