"""MXFP4 of gated activations whose gates lie far below zero, against float64."""
import numpy as np
import pytest
import torch
from scipy.special import expit, log_ndtr

import moe_routed_expert_amd as m
from gpu_util import dev
from mx4_util import ACTS, GRID, decode, quantise

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# The gates whose value is at least 2^-126.
LOWEST = {"silu": -91.5, "sigmoid": -87.0, "gelu": -13.0}


def gate64(act, g):
    """Relative accuracy over the whole range."""
    g = np.asarray(g, np.float64)
    return {"silu": lambda: g * expit(g), "sigmoid": lambda: expit(g), "gelu": lambda: g * np.exp(log_ndtr(g))}[act]()


def gate_eps(act, g):
    """Relative error of act(g) * up.  In units of 2^-24: SiLU and sigmoid: the exponent |g| log2 e is off by 1.22 of itself (its
    constant and its rounding), which is 1.22 |g| of the exponential; that is a square, two hardware exponentials of 2 each; 1 + t
    and its reciprocal 6 together, three products 3, up 1: 1.22 |g| + 14.  GELU: the exponent g^2 / 2 log2 e is off by 2.22 of
    itself, 1.11 g^2; the exponentials 4, the fitted factor 6, three products 3, up 1: 1.11 g^2 + 14."""
    g = np.abs(np.asarray(g, np.float64))
    return ((1.25 * g * g + 32) if act == "gelu" else (1.25 * g + 16)) * U


def check_codes(act, rule, q, s, g, u):
    """Codes and scales of act(g) * u: a scale is that of a maximum as near as the bound, a code half a step from the value.  A
    subnormal gate is the rounded product of two normal numbers: half a step of 2^-149 more."""
    f, u = gate64(act, g), np.asarray(u, np.float64)
    h = f * u
    off = gate_eps(act, g) * np.abs(h) + np.where(np.abs(f) < 2.0 ** -126, 2.0 ** -150, 0.0) * np.abs(u)
    n = h.shape[1]
    lo, hi = quantise(np.maximum(np.abs(h) - off, 0.0), rule == 1)[1], quantise(np.abs(h) + off, rule == 1)[1]
    assert ((s >= lo) & (s <= hi)).all(), np.argwhere((s < lo) | (s > hi))[:4]
    v = decode(q, s)
    scale = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1)[:, :n]
    t = np.minimum(np.abs(h) / scale, 6.0)
    i = np.clip(np.searchsorted(GRID, t, side="right") - 1, 0, 6)
    step = (GRID[i + 1] - GRID[i]) * scale
    err = np.abs(np.minimum(np.abs(h), 6.0 * scale) * np.sign(h) - v)
    bad = err > step / 2 + off * 1.001
    assert not bad.any(), (np.argwhere(bad)[:4], np.asarray(g)[bad][:4], h[bad][:4], v[bad][:4])


def run(x, act, rule):
    rows, n = x.shape[0], x.shape[1] // 2
    q, s = (torch.empty(shape, dtype=torch.uint8, device=dev()) for shape in ((rows, n // 2), (rows, -(-n // 32))))
    m.mx4_quant(x.to(dev()), q, s, act=ACTS[act], rule=rule)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("act", sorted(LOWEST))
@pytest.mark.parametrize("large_up", [False, True])
def test_tails(dt, rule, act, large_up):
    """Groups of gates next to each other, from -1 to the lowest whose value is normal; ups of ordinary size, or as large as the type
    takes them (the product is then of any size)."""
    rng = np.random.default_rng(5)
    rows, groups = 12, 16
    ends = np.linspace(-1.0, LOWEST[act] + 1.0, rows * groups).reshape(rows, groups)
    g = np.clip(np.repeat(ends, 32, axis=1) + rng.uniform(-0.9, 0.9, (rows, groups * 32)), LOWEST[act], None)
    u = rng.standard_normal(g.shape) * (1.0 if not large_up else 1e3 if dt is torch.float16 else 1e30)
    x = torch.from_numpy(np.concatenate([g, u], axis=1)).to(dt)
    q, s = run(x, act, rule)
    n = groups * 32
    x = x.double().numpy()
    check_codes(act, rule, q, s, np.clip(x[:, :n], LOWEST[act] - 1, None), x[:, n:])
    assert (np.abs(decode(q, s)).reshape(rows, groups, 32).max(axis=2) > 0).all()


@pytest.mark.parametrize("act", sorted(LOWEST))
def test_gates_above_zero(act):
    rng = np.random.default_rng(6)
    x = torch.from_numpy(np.concatenate([rng.uniform(0, 100, (7, 320)), rng.standard_normal((7, 320))], axis=1)).float()
    q, s = run(x, act, 0)
    x = x.double().numpy()
    check_codes(act, 0, q, s, x[:, :320], x[:, 320:])


@pytest.mark.parametrize("act", sorted(LOWEST))
def test_below_the_normal_range(act):
    """Gates whose values go through fp32's subnormals to zero, with ups of 1e30."""
    g = np.linspace(LOWEST[act], 4 * LOWEST[act], 2048).reshape(8, 256)
    x = torch.from_numpy(np.concatenate([g, np.full_like(g, 1e30)], axis=1)).float()
    for rule in (0, 1):
        q, s = run(x, act, rule)
        check_codes(act, rule, q, s, x[:, :256].double().numpy(), x[:, 256:].double().numpy())


@pytest.mark.parametrize("mode", [m.MOE_MODE_GROUPED, m.MOE_MODE_SLOT])
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_the_fused_product_keeps_them(mode, act):
    """Gates of exactly -16 .. -88 out of the product, ups of 2^90 times a code: the requant in the epilogue is that of the stored rows, and both
    within the bound."""
    code = {0.0: 0, 0.5: 1, 1.0: 2, 1.5: 3, 2.0: 4, 3.0: 5, 4.0: 6, 6.0: 7}
    pairs = [(1.0, 0.0), (1.5, 0.0), (2.0, 0.0), (1.0, 1.5), (3.0, 0.0), (2.0, 1.5), (4.0, 0.0), (3.0, 1.5), (4.0, 1.0), (4.0, 1.5)]
    I, K, rows = 32 * len(pairs), 64, 3
    aq, as_ = np.zeros((rows, K // 2), np.uint8), np.full((rows, K // 32), 127, np.uint8)
    aq[:, 0] = aq[:, 16] = code[1.0]                            # k = 0 and k = 32, a scale group each
    wq, ws = np.zeros((1, 2 * I, K // 2), np.uint8), np.full((1, 2 * I, K // 32), 127, np.uint8)
    g, u = np.zeros(I), np.zeros(I)
    for c in range(I):
        (a, b), up = pairs[c // 32], list(code)[1 + c % 7]
        wq[0, c, 0], wq[0, c, 16] = code[a] + 8, code[b] + 8
        wq[0, I + c, 0] = code[up]
        g[c], u[c] = -16 * (a + b), up * 2.0 ** 90
    ws[0, :I], ws[0, I:] = 127 + 4, 127 + 90
    gpu = [torch.from_numpy(t).to(dev()) for t in (aq, np.pad(as_, ((0, 0), (0, 2))), wq, np.pad(ws, ((0, 0), (0, 0), (0, 2))))]
    gpu[1], gpu[3] = gpu[1][:, :K // 32], gpu[3][:, :, :K // 32]
    how = dict(mode=mode, expert_offsets=torch.tensor([0, rows], dtype=torch.int32, device=dev()),
               slot_ids=torch.zeros(rows, dtype=torch.int32, device=dev()))
    c1 = torch.empty((rows, 2 * I), device=dev())
    m.mx4_grouped_gemm(*gpu, c1, **how)
    assert np.array_equal(c1[:, :I].cpu().numpy(), np.tile(g, (rows, 1)))
    assert np.array_equal(c1[:, I:].cpu().numpy(), np.tile(u, (rows, 1)))
    for rule in (0, 1):
        q, s = run(c1.cpu(), act, rule)
        check_codes(act, rule, q, s, np.tile(g, (rows, 1)), np.tile(u, (rows, 1)))
        gq, gs = torch.empty((rows, I // 2), dtype=torch.uint8, device=dev()), torch.empty((rows, I // 32), dtype=torch.uint8, device=dev())
        m.mx4_grouped_gemm_act_quant(*gpu, gq, gs, act=ACTS[act], rule=rule, **how)
        torch.cuda.synchronize()
        assert np.array_equal(gq.cpu().numpy(), q) and np.array_equal(gs.cpu().numpy(), s)
