"""GPU tests of moe_act_checkpoint and moe_gated_act_backward against the float64 definitions."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from oracle import training as tr
from train_util import HALF, NAMES, TINY, Guarded, check, f64, randn, replayed

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def rows_of(rows, width, dt, seed):
    x = randn((rows, width), F32, seed)
    return (x * torch.exp(torch.linspace(-4, 2, max(rows, 1)))[:rows, None]).to(dt)


def gate_errors(act, g, dt):
    """Bounds on the device's absolute error of act(g) and act'(g), in fp32 before any rounding to dt.

    r, the sigmoid, has relative error er.  fp32: expf within 2 ulp (2^-22) of a value whose share of 1 + e^-g is
    1 - r, the sum and the division half an ulp each: er <= 2^-22 + 2^-23.  16 bits: the exponent -g log2 e carries a
    relative 2^-23 (the constant's and the product's rounding), i.e. |g| 2^-23 in e^-g, exp2 and rcp an ulp each,
    the sum half: er <= (|g| + 5) 2^-23.  Below -87 the fast form may flush a sigmoid below 2^-125 to 0.
    silu: f = g r;  d = r + f (1 - r): 1 - r is off by er r + U, so d by er r (1 + |g| (1 + r)) + 4 U (r + |f|).
    gelu: erff within 4 ulp of at most 1 (2^-21), so p = (1 + erf) / 2 is off by at most 2^-21; f = g p; the density's
    exponent carries g^2 2^-23, expf 2^-22.
    sigmoid: d = r (1 - r) is off by er r + r (er r + U) + U r."""
    f, d = tr.gate(act, g)
    a = np.abs(g)
    er = 2.0 ** -22 + 2.0 ** -23 if dt == F32 else (a + 5) * 2.0 ** -23
    r = tr.gate(4, g)[0]
    flush = 2.0 ** -125 if dt != F32 else 0.0
    if act == 1:
        return a * (er * r + flush) + 2 * U * np.abs(f), er * r * (1 + a * (1 + r)) + 4 * U * (r + np.abs(f)) + flush * (1 + a)
    if act == 2:
        dens = np.exp(-g * g / 2) / np.sqrt(2 * np.pi)
        return a * 2.0 ** -21 + 2 * U * np.abs(f), 2.0 ** -21 + a * dens * (a * a * 2.0 ** -23 + 2.0 ** -21) + 2 * U * np.abs(d)
    if act == 4:
        return er * r + flush, 2 * er * r + 3 * U * r + flush
    return np.zeros_like(g), np.zeros_like(g)


def bound(dt, ref, err):
    return err + HALF[dt] * (np.abs(ref) + err) + TINY[dt] + 2.0 ** -148


def values(q, s, n):
    return f64(q.cpu().view(torch.float8_e4m3fn)) * np.repeat(f64(s), 128, axis=1)[:, :n]


@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("rows,n", [(1, 1), (1, 8), (3, 100), (5, 128), (2, 129), (7, 512), (4, 520), (130, 1000), (9, 2048), (2, 4099)])
def test_save_rows(rows, n, dt):
    print("save rows=%d n=%d %s" % (rows, n, NAMES[dt]), flush=True)
    x = rows_of(rows, n, dt, n)
    groups = -(-n // 128)
    q, s = Guarded((rows, n), torch.uint8, fill=9), Guarded((rows, groups), F32)
    m.act_checkpoint(x.to(dev()), q.view, s.view)
    torch.cuda.synchronize()
    assert q.intact() and s.intact()
    rq, rs = tr.save8(f64(x))
    assert np.array_equal(f64(s.view), rs)
    assert np.array_equal(f64(q.view.cpu().contiguous().view(torch.float8_e4m3fn)), rq)


@pytest.mark.parametrize("act", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("rows,n", [(1, 8), (3, 100), (6, 712), (33, 1024)])
def test_save_gated(rows, n, dt, act):
    x = rows_of(rows, 2 * n, dt, n + act)
    groups = -(-n // 128)
    q = torch.full((rows, 2 * n), 9, dtype=torch.uint8, device=dev())
    s = torch.full((rows, 2 * groups), float("nan"), dtype=F32, device=dev())
    h = Guarded((rows, n), dt)
    m.act_checkpoint(x.to(dev()), q, s, act=act, h=h.view)
    torch.cuda.synchronize()
    assert h.intact()
    for half in (0, 1):
        rq, rs = tr.save8(f64(x[:, half * n:(half + 1) * n]))
        assert np.array_equal(f64(s[:, half * groups:(half + 1) * groups]), rs)
        assert np.array_equal(f64(q[:, half * n:(half + 1) * n].cpu().contiguous().view(torch.float8_e4m3fn)), rq)
    g, u = f64(x[:, :n]), f64(x[:, n:])
    ref = tr.gate(act, g)[0] * u
    ef, _ = gate_errors(act, g, dt)
    check(h.view, ref, bound(dt, ref, ef * np.abs(u) + 2 * U * np.abs(ref)), "h")
    m.act_checkpoint(x.to(dev()), q.fill_(1), s, act=act)              # without h: the same codes
    torch.cuda.synchronize()
    assert np.array_equal(f64(q[:, n:].cpu().contiguous().view(torch.float8_e4m3fn)), rq)


@pytest.mark.parametrize("act", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("rows,n", [(1, 1), (2, 8), (3, 100), (37, 712), (5, 2048), (70, 1032)])
@pytest.mark.parametrize("with_h", [True, False])
def test_backward(rows, n, dt, act, with_h):
    x, dh = rows_of(rows, 2 * n, F32, n + act) * 3, randn((rows, n), dt, n, 0.1)
    groups = -(-n // 128)
    q = torch.empty((rows, 2 * n), dtype=torch.uint8, device=dev())
    s = torch.empty((rows, 2 * groups), dtype=F32, device=dev())
    m.act_checkpoint(x.to(dev()), q, s, act=act)
    dx, h = Guarded((rows, 2 * n), dt), Guarded((rows, n), dt)
    m.gated_act_backward(dh.to(dev()), q, s, dx.view, act=act, h=h.view if with_h else None)
    torch.cuda.synchronize()
    assert dx.intact() and h.intact() and (with_h or bool((h.view == h.fill).all()))
    g, u = values(q[:, :n].contiguous(), s[:, :groups], n), values(q[:, n:].contiguous(), s[:, groups:], n)
    f, d = tr.gate(act, g)
    ef, ed = gate_errors(act, g, dt)
    dhv = f64(dh)
    ref = tr.gated_act_backward(act, np.concatenate([g, u], 1), dhv)
    eg = np.abs(dhv * u) * ed + 2 * U * np.abs(ref[:, :n])
    eu = np.abs(dhv) * ef + U * np.abs(ref[:, n:])
    check(dx.view, ref, bound(dt, ref, np.concatenate([eg, eu], 1)), "dx")
    if with_h:
        check(h.view, f * u, bound(dt, f * u, ef * np.abs(u) + U * np.abs(f * u)), "h")


def test_backward_of_scales_that_are_no_powers_of_two():
    rows, n = 5, 256
    x, dh = rows_of(rows, 2 * n, BF, 1), randn((rows, n), F32, 2)
    q = torch.empty((rows, 2 * n), dtype=torch.uint8, device=dev())
    s = torch.empty((rows, 4), dtype=F32, device=dev())
    m.act_quant(x.to(dev()), q, s)
    dx = torch.empty((rows, 2 * n), dtype=F32, device=dev())
    m.gated_act_backward(dh.to(dev()), q, s, dx, act=5)
    v = values(q, s, 2 * n)
    ref = tr.gated_act_backward(5, v, f64(dh))
    check(dx, ref, bound(F32, ref, 4 * U * np.abs(ref)), "dx")


@pytest.mark.parametrize("dt", [BF, FP, F32])
def test_non_finite_and_extreme_values(dt):
    """A NaN or infinity becomes the NaN code; its neighbours in the group stay finite, other groups unchanged."""
    x = randn((4, 384), F32, 3).to(dt)
    x[0, 5], x[1, 130], x[2, 383] = float("nan"), float("inf"), float("-inf")
    x[3, :128] = float("nan")
    q = torch.empty((4, 384), dtype=torch.uint8, device=dev())
    s = torch.empty((4, 3), dtype=F32, device=dev())
    m.act_checkpoint(x.to(dev()), q, s)
    torch.cuda.synchronize()
    got = q.cpu().view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(np.isnan(got), ~np.isfinite(x.float().numpy()))
    assert bool(torch.isfinite(s).all())
    clean = np.ones((4, 3), bool)
    clean[0, 0] = clean[1, 1] = clean[2, 2] = clean[3, 0] = False
    rq, rs = tr.save8(np.nan_to_num(f64(x), posinf=0, neginf=0))
    for r, j in np.argwhere(clean):
        assert f64(s)[r, j] == rs[r, j]
        assert np.array_equal(got[r, 128 * j:128 * (j + 1)], rq[r, 128 * j:128 * (j + 1)])


def test_borders_of_the_scale():
    """Group maxima at and next to 448 * 2^k, at the ends of fp32's range and among its subnormals."""
    tops = [448.0, np.nextafter(np.float32(448), np.float32(0)), np.nextafter(np.float32(448), np.float32(1e9)), 1.0, 1.75,
            np.nextafter(np.float32(1.75), np.float32(2)), 3.4028235e38, 2.0 ** -118, 2.0 ** -119, 2.0 ** -126, 2.0 ** -130,
            2.0 ** -149, 0.0, -0.0]
    x = np.zeros((len(tops), 128), np.float32)
    x[:, 64] = tops
    x[:, 3] = -np.asarray(tops, np.float32) * np.float32(0.3)
    q = torch.empty((len(tops), 128), dtype=torch.uint8, device=dev())
    s = torch.empty((len(tops), 1), dtype=F32, device=dev())
    m.act_checkpoint(torch.from_numpy(x).to(dev()), q, s)
    torch.cuda.synchronize()
    rq, rs = tr.save8(x)
    assert np.array_equal(f64(s), rs)
    assert np.array_equal(f64(q.cpu().view(torch.float8_e4m3fn)), rq)


def test_gradient_that_overflowed_stays_visible():
    """fp16 training with loss scaling looks for non-finite gradients: they must not be clamped away."""
    q = torch.full((2, 256), 0x38, dtype=torch.uint8, device=dev())
    s = torch.ones((2, 2), dtype=F32, device=dev())
    dh = torch.ones((2, 128), dtype=FP, device=dev())
    dh[0, 3], dh[1, 4] = float("inf"), float("nan")
    dx = torch.zeros((2, 256), dtype=FP, device=dev())
    m.gated_act_backward(dh, q, s, dx, act=1)
    bad = ~torch.isfinite(dx).cpu().numpy()
    assert bad.sum() == 4 and bad[0, 3] and bad[0, 131] and bad[1, 4] and bad[1, 132]


def test_strided_and_unaligned_rows():
    for off, pad in ((8, 16), (1, 3), (4, 4)):
        n = 200
        buf = torch.full((6, 2 * n + 32), float("nan"), dtype=BF)
        buf[:, off:off + 2 * n] = randn((6, 2 * n), BF, off)
        x = buf.to(dev())[:, off:off + 2 * n]
        q, s, h = Guarded((6, 2 * n), torch.uint8, pad=pad, fill=9), Guarded((6, 4), F32, pad=1), Guarded((6, n), BF, pad=pad)
        m.act_checkpoint(x, q.view, s.view, act=3, h=h.view)
        dx = Guarded((6, 2 * n), BF, pad=pad)
        m.gated_act_backward(h.view, q.view, s.view, dx.view, act=5)
        torch.cuda.synchronize()
        assert q.intact() and s.intact() and h.intact() and dx.intact()
        rq, rs = tr.save8(f64(x[:, :n]))
        assert np.array_equal(f64(q.view[:, :n].cpu().contiguous().view(torch.float8_e4m3fn)), rq)
        v = np.concatenate([values(q.view[:, k * n:(k + 1) * n].contiguous(), s.view[:, 2 * k:2 * k + 2].contiguous(), n) for k in (0, 1)], 1)
        ref = tr.gated_act_backward(5, v, f64(h.view))
        check(dx.view, ref, bound(BF, ref, 4 * U * np.abs(ref)), "dx")


def test_many_rows():
    """More rows than the grid's second dimension holds blocks of."""
    rows = 4 * 65535 + 9
    x = torch.zeros((rows, 8), dtype=BF, device=dev())
    x[:, 0] = 1
    x[-1, 1] = 448
    q = torch.full((rows, 8), 9, dtype=torch.uint8, device=dev())
    s = torch.zeros((rows, 1), dtype=F32, device=dev())
    m.act_checkpoint(x, q, s)
    torch.cuda.synchronize()
    assert bool((s[:-1] == 2.0 ** -8).all()) and float(s[-1]) == 1.0
    assert bool((q[:-1, 0] == 0x78).all()) and bool((q[:-1, 1:] == 0).all()) and int(q[-1, 1]) == 0x7E


@pytest.mark.parametrize("n", [200, 1024])
def test_graph_replay_and_other_stream(n):
    x, dh = randn((20, 2 * n), BF, 1).to(dev()), randn((20, n), BF, 2).to(dev())
    q = torch.empty((20, 2 * n), dtype=torch.uint8, device=dev())
    s = torch.empty((20, 2 * -(-n // 128)), dtype=F32, device=dev())
    h, dx = torch.empty((20, n), dtype=BF, device=dev()), torch.empty((20, 2 * n), dtype=BF, device=dev())

    def call(stream=None):
        m.act_checkpoint(x, q, s, act=1, h=h, stream=stream)
        m.gated_act_backward(dh, q, s, dx, act=1, stream=stream)

    for got, want in replayed(call, None, [q, s, h, dx], lambda i: x.copy_(randn((20, 2 * n), BF, 30 + i))):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    keep = dx.clone()
    dx.fill_(0)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    call(st)
    st.synchronize()
    assert torch.equal(dx, keep)


def test_binding_checks():
    x, q = torch.zeros((4, 64), dtype=BF, device=dev()), torch.zeros((4, 64), dtype=torch.uint8, device=dev())
    s1, s2, h = torch.zeros((4, 1), device=dev()), torch.zeros((4, 2), device=dev()), torch.zeros((4, 32), dtype=BF, device=dev())
    for bad in (lambda: m.act_checkpoint(x, q[:, :32], s1), lambda: m.act_checkpoint(x, q, s2), lambda: m.act_checkpoint(x, q, s1, act=1),
                lambda: m.act_checkpoint(x[:, :63], q[:, :63], s2, act=1), lambda: m.act_checkpoint(x, q, s2, act=1, h=h.half()),
                lambda: m.act_checkpoint(x.cpu(), q, s1), lambda: m.gated_act_backward(h, q[:, :32], s2, x),
                lambda: m.gated_act_backward(h, q, s1, x), lambda: m.gated_act_backward(h, q, s2, x.half()),
                lambda: m.gated_act_backward(h, q, s2, h)):
        with pytest.raises(AssertionError):
            bad()
    with pytest.raises(m.MoeError):
        m.act_checkpoint(x, q, s1, h=x)
