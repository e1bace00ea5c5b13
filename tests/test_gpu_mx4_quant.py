"""Rows to MXFP4 and back: codes and scales bit for bit against the format's definition in float64."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from mx4_util import ACTS, GRID, decode, gate, quantise
from train_util import Guarded, randn, replayed

pytestmark = pytest.mark.gpu
DTS = [torch.bfloat16, torch.float16, torch.float32]


def run(x, act=0, rule=0, q=None, s=None):
    rows, n = x.shape[0], x.shape[1] // (1 if act == 0 else 2)
    q = torch.full((rows, n // 2), 0x77, dtype=torch.uint8, device=dev()) if q is None else q
    s = torch.full((rows, -(-n // 32)), 0x77, dtype=torch.uint8, device=dev()) if s is None else s
    m.mx4_quant(x, q, s, act=act, rule=rule)
    torch.cuda.synchronize()
    return q.cpu().numpy(), s.cpu().numpy()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("rows,n", [(1, 32), (3, 2), (5, 30), (7, 34), (37, 712), (4, 1000), (9, 4160), (300, 128), (2, 8200)])
def test_rows(dt, rule, rows, n):
    x = randn((rows, n), dt, rows * 1000 + n, 1.7)
    q, s = run(x.to(dev()), rule=rule)
    rq, rs = quantise(x.double().numpy(), rule == 1)
    assert np.array_equal(s, rs) and np.array_equal(q, rq)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rule", [0, 1])
def test_special_values(dt, rule):
    """Groups of zeros, ties, borders of the scale, the smallest and largest magnitudes, infinities and NaN."""
    big, tiny = torch.finfo(dt).max, torch.finfo(dt).smallest_normal
    sub = tiny * torch.finfo(dt).eps
    rows = [torch.zeros(32), -torch.zeros(32), torch.full((32,), -6.0), torch.full((32,), 7.0), torch.full((32,), 8.0)]
    for top in (4.0, 6.0, 6.25, 7.5, 8.0):
        ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.5, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, top])
        for e in (-8, 0, 8):
            rows.append(torch.cat([ties * 2.0 ** e, torch.zeros(17)]))
    for x in (big, -big, tiny, sub, -sub, 4 * sub, 64 * tiny):
        rows.append(torch.cat([torch.full((16,), float(x)), torch.full((16,), float(x) / 8)]))
    for x in (float("inf"), -float("inf"), float("nan")):
        rows.append(torch.cat([torch.ones(31), torch.tensor([x])]))
        rows.append(torch.cat([torch.tensor([x]), torch.zeros(31)]))
    x = torch.stack(rows).to(dt)
    q, s = run(x.to(dev()), rule=rule)
    rq, rs = quantise(x.double().numpy(), rule == 1)
    assert np.array_equal(s, rs) and np.array_equal(q, rq)
    assert (s[-6:] == 255).all() and (q[-6:] == 0).all()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,n,pad", [(5, 64, 0), (6, 96, 1), (4, 712, 8), (33, 1024, 24)])
def test_strided_views_and_what_lies_around(dt, rows, n, pad):
    x = randn((rows + 2, n + 2 * pad + 3), dt, n)
    view = x.to(dev())[1:1 + rows, pad:pad + n]
    gq, gs = Guarded((rows, n // 2), torch.uint8, pad=pad), Guarded((rows, -(-n // 32)), torch.uint8, pad=3)
    q, s = run(view, q=gq.view, s=gs.view)
    rq, rs = quantise(x[1:1 + rows, pad:pad + n].double().numpy())
    assert np.array_equal(s, rs) and np.array_equal(q, rq) and gq.intact() and gs.intact()


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("rows,n", [(1, 32), (5, 44), (37, 712)])
def test_gated(dt, act, rule, rows, n):
    """ReLU and the product are exact.  A transcendental gate is within 2^-19 of its value (the sigmoid's exponent -g log2 e
    rounds to 2^-24 of at most 2^4 and the hardware exp2 and reciprocal add an ulp each; the fitted Phi is within 3.5e-7),
    so its scale is that of a maximum as near, and a code is half a step from the value, more by 2^-19 of it."""
    x = randn((rows, 2 * n), dt, rows + n, 1.3)
    q, s = run(x.to(dev()), act=ACTS[act], rule=rule)
    h = gate(act, x[:, :n].double().numpy(), x[:, n:].double().numpy())
    if act in ("relu", "mul"):
        rq, rs = quantise(h.astype(np.float32).astype(np.float64), rule == 1)
        assert np.array_equal(s, rs)
        if act == "mul":
            assert np.array_equal(q, rq)
        assert np.array_equal(decode(q, s), decode(rq, rs))       # ReLU: zeros of either sign
        return
    eps = 2.0 ** -19
    lo, hi = quantise(h * (1 - eps), rule == 1)[1], quantise(h * (1 + eps), rule == 1)[1]
    assert ((s == lo) | (s == hi)).all()
    v = decode(q, s)
    scale = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, axis=1)[:, :n]
    t = np.minimum(np.abs(h) / scale, 6.0)
    i = np.clip(np.searchsorted(GRID, t, side="right") - 1, 0, 6)
    step = (GRID[i + 1] - GRID[i]) * scale
    err = np.abs(np.minimum(np.abs(h), 6.0 * scale) * np.sign(h) - v)
    assert (err <= step / 2 + eps * np.abs(h) * 1.001).all()


def test_gate_of_nan_and_infinity():
    x = torch.ones(3, 128)
    x[0, 5], x[1, 70], x[2, 33] = float("nan"), float("inf"), -float("inf")
    for act in range(1, 6):
        q, s = run(x.to(dev()), act=act)
        assert s[0].tolist()[0] == 255 and s[0, 1] != 255 and (q[0, :16] == 0).all()
        assert s[1, 0] == 255 and s[1, 1] != 255               # up = inf at column 6 of the first group
        assert (s[2, 1] == 255) == (act in (1, 2, 5))          # 0 * -inf of SiLU and GELU, -inf of the product; ReLU and sigmoid give 0
        assert s[2, 0] != 255


@pytest.mark.parametrize("dt", DTS)
def test_every_code_and_scale_read_back(dt):
    q = torch.arange(256, dtype=torch.uint8).repeat(256, 1)
    s = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    out = torch.empty((256, 512), dtype=dt, device=dev())
    m.mx4_dequant(q.to(dev()), s.to(dev()), out)
    ref = decode(q.numpy(), s.numpy())
    got = out.cpu()
    assert torch.isnan(got[255]).all()
    want = torch.from_numpy(ref[:255]).to(dt)                  # one rounding from float64
    assert torch.equal(got[:255], want)


@pytest.mark.parametrize("dt", DTS)
@pytest.mark.parametrize("rows,n,pad", [(1, 2, 0), (3, 30, 1), (5, 712, 4), (64, 1024, 8)])
def test_read_back_strided(dt, rows, n, pad):
    x = randn((rows, n), dt, n)
    q, s = quantise(x.double().numpy())
    wide = torch.full((rows, n // 2 + pad), 0xFF, dtype=torch.uint8)
    wide[:, :n // 2] = torch.from_numpy(q)
    g = Guarded((rows, n), dt, pad=pad)
    m.mx4_dequant(wide.to(dev())[:, :n // 2], torch.from_numpy(s).to(dev()), g.view)
    torch.cuda.synchronize()
    assert torch.equal(g.view.cpu(), torch.from_numpy(decode(q, s)).to(dt)) and g.intact()


def test_rows_past_32_bits():
    """Row offsets of more than 2^32 elements on every operand."""
    rows, stride = 3, (1 << 31) + 64
    x = torch.empty(2 * stride + 64, dtype=torch.bfloat16, device=dev())
    xs = x.as_strided((rows, 64), (stride, 1))
    v = randn((rows, 64), torch.bfloat16, 1)
    xs.copy_(v)
    qb = torch.empty(2 * stride + 32, dtype=torch.uint8, device=dev())
    q, s = run(xs, q=qb.as_strided((rows, 32), (stride, 1)))
    rq, rs = quantise(v.double().numpy())
    assert np.array_equal(q, rq) and np.array_equal(s, rs)
    xs.zero_()
    m.mx4_dequant(qb.as_strided((rows, 32), (stride, 1)), torch.from_numpy(rs).to(dev()), xs)
    assert torch.equal(xs.cpu(), torch.from_numpy(decode(rq, rs)).to(torch.bfloat16))


def test_no_rows_and_refusals():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=dev())
    m.mx4_quant(e, torch.empty((0, 32), dtype=torch.uint8, device=dev()), torch.empty((0, 2), dtype=torch.uint8, device=dev()))
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device=dev())
    u = lambda *shape: torch.empty(shape, dtype=torch.uint8, device=dev())  # noqa: E731
    for bad in (lambda: m.mx4_quant(x, u(2, 31), u(2, 2)), lambda: m.mx4_quant(x, u(2, 32), u(2, 1)), lambda: m.mx4_quant(x[:, :63], u(2, 31), u(2, 2)),
                lambda: m.mx4_quant(x, u(2, 32).float(), u(2, 2)), lambda: m.mx4_quant(x.t(), u(64, 1), u(64, 1)),
                lambda: m.mx4_dequant(u(2, 32), u(2, 3), x), lambda: m.mx4_dequant(u(3, 32), u(3, 2), x)):
        with pytest.raises(AssertionError):
            bad()


def test_captured():
    x = torch.empty((19, 1024), dtype=torch.bfloat16, device=dev())
    q, s = torch.empty((19, 256), dtype=torch.uint8, device=dev()), torch.empty((19, 16), dtype=torch.uint8, device=dev())
    v = torch.empty((19, 512), dtype=torch.float32, device=dev())

    def call():
        m.mx4_quant(x, q, s, act=1, rule=1)
        m.mx4_dequant(q, s, v)
    for got, want in replayed(call, None, [q, s, v], lambda i: x.copy_(randn((19, 1024), torch.bfloat16, i))):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
