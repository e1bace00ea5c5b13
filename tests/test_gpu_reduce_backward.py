"""GPU tests of moe_topk_reduce_backward and moe_route_prep_backward, and of a whole training step."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import HALF, NAMES, TINY, Guarded, check, f64, offsets_of, randn, replayed, sum_bound

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24


def reduce_case(T, k, H, dt, seed, drop=0.3, mapped=False):
    rng = np.random.default_rng(seed)
    dout, y = randn((T, H), BF, seed, 0.3), randn((T * k, H), dt, seed + 1)
    slots = np.where(rng.random((T, k)) < drop, -1, rng.integers(0, 9, (T, k))).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    w[slots < 0] = np.nan                                  # never read
    rows = rng.permutation(T * k).astype(np.int32) if mapped else None
    return dout, y, slots, w, rows


def run_reduce(T, k, H, dt, seed, drop=0.3, mapped=False, need_dw=True):
    print("reduce backward T=%d k=%d H=%d %s mapped=%d" % (T, k, H, NAMES[dt], mapped), flush=True)
    dout, y, slots, w, rows = reduce_case(T, k, H, dt, seed, drop, mapped)
    dy = Guarded((T * k, H), dt)
    dw = torch.full((T, k), float("nan"), device=dev()) if need_dw else None
    m.topk_reduce_backward(dout.to(dev()), y.to(dev()) if need_dw else None, to_dev(slots), to_dev(w), dy.view, dw,
                           route_rows=None if rows is None else to_dev(rows))
    torch.cuda.synchronize()
    assert dy.intact()
    rdy, rdw, mag = tr.reduce_backward(f64(dout), f64(y), slots, np.nan_to_num(w).astype(np.float64), rows)
    got = f64(dy.view)
    left = np.isnan(rdy)
    assert np.all(got[left] == dy.fill), "a row that no route names changed"
    ref = np.where(left, got, rdy)
    check(got, ref, HALF[dt] * np.abs(ref) * (1 + 2 * U) + 2 * U * np.abs(ref) + TINY[dt], "dy")
    if need_dw:
        check(dw, rdw, (H + 8) * 2 * U * mag + 2.0 ** -140, "dweights")
        assert np.all(f64(dw)[slots < 0] == 0)


@pytest.mark.parametrize("mapped", [False, True])
@pytest.mark.parametrize("dt", [BF, FP, F32])
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (1, 8, 64), (3, 2, 100), (9, 6, 2056), (5, 9, 2048), (2, 17, 4100), (1030, 6, 72), (1025, 9, 33)])
def test_reduce_backward(T, k, H, dt, mapped):
    run_reduce(T, k, H, dt, T + H, mapped=mapped)


@pytest.mark.parametrize("drop", [0.0, 1.0])
def test_all_and_none_active(drop):
    for T in (4, 1030):
        run_reduce(T, 4, 264, BF, T, drop=drop)
        run_reduce(T, 4, 264, BF, T, drop=drop, mapped=True)


def test_without_the_weights_gradient():
    run_reduce(6, 3, 264, BF, 1, need_dw=False)
    run_reduce(1100, 3, 40, F32, 2, need_dw=False, mapped=True)


def test_rows_out_of_range_are_skipped():
    T, k, H = 4, 2, 64
    dout, y, slots, w, _ = reduce_case(T, k, H, BF, 5, drop=0.0)
    rows = np.array([0, 99, -3, 5, 2 ** 31 - 1, 1, 7, 8], np.int32)      # rows 8 and up are not there
    dy = Guarded((8, H), BF)
    dw = torch.full((T, k), float("nan"), device=dev())
    m.topk_reduce_backward(dout.to(dev()), y.to(dev()), to_dev(slots), to_dev(w), dy.view, dw, route_rows=to_dev(rows))
    torch.cuda.synchronize()
    assert dy.intact()
    rdy, rdw, mag = tr.reduce_backward(f64(dout), f64(y), slots, w.astype(np.float64), rows)
    left = np.isnan(rdy)
    assert np.all(f64(dy.view)[left] == dy.fill) and np.all(f64(dw).reshape(-1)[[1, 2, 4, 7]] == 0)
    check(dw, rdw, (H + 8) * 2 * U * mag + 2.0 ** -140, "dweights")


def test_unaligned_and_strided_rows():
    for off in (1, 4, 8):
        T, k, H = 5, 3, 136
        dout, y, slots, w, _ = reduce_case(T, k, H, FP, off)
        db = torch.full((T, H + 16), float("nan"), dtype=BF)
        db[:, off:off + H] = dout
        yb = torch.full((T * k, H + 16), float("nan"), dtype=FP)
        yb[:, off:off + H] = y
        dy, dw = Guarded((T * k, H), FP, pad=off), torch.empty((T, k), device=dev())
        m.topk_reduce_backward(db.to(dev())[:, off:off + H], yb.to(dev())[:, off:off + H], to_dev(slots), to_dev(w), dy.view, dw)
        torch.cuda.synchronize()
        assert dy.intact()
        rdy, rdw, mag = tr.reduce_backward(f64(dout), f64(y), slots, np.nan_to_num(w).astype(np.float64))
        check(dy.view, rdy, HALF[FP] * np.abs(rdy) * (1 + 2 * U) + 2 * U * np.abs(rdy) + TINY[FP], "dy")
        check(dw, rdw, (H + 8) * 2 * U * mag + 2.0 ** -140, "dweights")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 8, 2), (5, 64, 8), (9, 100, 6), (4, 1024, 64), (1001, 256, 6)])
def test_route_backward(T, E, k):
    rng = np.random.default_rng(E)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.dirichlet(np.ones(k), T).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    out = Guarded((T, E), F32, pad=3)
    m.route_prep_backward(to_dev(ids), to_dev(w), to_dev(dw), out.view)
    torch.cuda.synchronize()
    assert out.intact()
    w64, dw64 = w.astype(np.float64), dw.astype(np.float64)
    ref = tr.route_backward(ids, w64, dw64, E)
    # the mean's k products and sums lose 2^-23 of sum |w dw| each at most, then a difference and a product
    s = (k + 2) * 2.0 ** -23 * np.abs(w64 * dw64).sum(1, keepdims=True)
    err = np.zeros((T, E))
    np.put_along_axis(err, ids.astype(np.int64), w64 * (s + 2.0 ** -22 * np.abs(dw64)), axis=1)
    check(out.view, ref, err, "dlogits")
    named = np.zeros((T, E), bool)
    np.put_along_axis(named, ids.astype(np.int64), True, axis=1)
    assert np.all(f64(out.view)[~named] == 0)


def test_route_backward_odd_ids():
    """An id out of range is skipped, one named twice gets the sum."""
    ids = np.array([[3, 3, -1], [0, 7, 2 ** 31 - 1]], np.int32)
    w = np.array([[0.5, 0.25, 0.25], [0.5, 0.25, 0.25]], np.float32)
    dw = np.array([[1.0, 2.0, 4.0], [1.0, 2.0, 4.0]], np.float32)
    out = torch.full((2, 8), float("nan"), device=dev())
    m.route_prep_backward(to_dev(ids), to_dev(w), to_dev(dw), out)
    ref = tr.route_backward(ids, w.astype(np.float64), dw.astype(np.float64), 8)
    assert np.array_equal(f64(out), ref)                   # sums of powers of two: exact


def test_more_items_than_a_grid_holds():
    """More tokens than workgroups of one launch: they are taken in turn."""
    T, H = (1 << 23) + 5, 8
    dout = torch.ones((T, H), dtype=BF, device=dev())
    y = torch.full((T, H), 0.5, dtype=BF, device=dev())
    slots = torch.zeros((T, 1), dtype=torch.int32, device=dev())
    w = (torch.arange(T, device=dev()) % 7).float()[:, None].contiguous()
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    m.topk_reduce_backward(dout, y, slots, w, dy, dw)
    assert bool((dw == 4).all()) and bool((dy.float() == w).all())
    del dout, y, dy
    T = (1 << 25) + 3
    ids = torch.zeros((T, 1), dtype=torch.int32, device=dev())
    w, dw = torch.full((T, 1), 0.5, device=dev()), (torch.arange(T, device=dev()) % 9).float()[:, None].contiguous()
    out = torch.full((T, 1), float("nan"), device=dev())
    m.route_prep_backward(ids, w, dw, out)
    assert bool((out == 0.25 * dw).all())


def test_graph_replay():
    T, k, H, E = 12, 4, 264, 16
    dout, y, slots, w, rows = reduce_case(T, k, H, BF, 3, mapped=True)
    w = np.nan_to_num(w)
    t = dict(dout=dout.to(dev()), y=y.to(dev()), slots=to_dev(slots), w=to_dev(w), rows=to_dev(rows))
    ids = to_dev(np.stack([np.random.default_rng(i).permutation(E)[:k] for i in range(T)]).astype(np.int32))
    dy, dw, dl = torch.zeros((T * k, H), dtype=BF, device=dev()), torch.zeros((T, k), device=dev()), torch.zeros((T, E), device=dev())

    def call():
        dy.zero_()
        m.topk_reduce_backward(t["dout"], t["y"], t["slots"], t["w"], dy, dw, route_rows=t["rows"])
        m.route_prep_backward(ids, t["w"], dw, dl)

    def fresh(i):
        a, b, c, d, e = reduce_case(T, k, H, BF, 50 + i, mapped=True)
        t["dout"].copy_(a), t["y"].copy_(b), t["slots"].copy_(torch.from_numpy(c))
        t["w"].copy_(torch.from_numpy(np.nan_to_num(d))), t["rows"].copy_(torch.from_numpy(e))

    for got, want in replayed(call, None, [dy, dw, dl], fresh):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_binding_checks():
    T, k, H = 4, 2, 64
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt, device=dev())
    i = z(T, k, dt=torch.int32)
    w = z(T, k, dt=F32)
    for bad in (lambda: m.topk_reduce_backward(z(T, H, dt=FP), z(8, H), i, w, z(8, H), w), lambda: m.topk_reduce_backward(z(T, H), z(7, H), i, w, z(7, H), w),
                lambda: m.topk_reduce_backward(z(T, H), z(8, H, dt=FP), i, w, z(8, H), w), lambda: m.topk_reduce_backward(z(T, H), z(8, H), i.long(), w, z(8, H), w),
                lambda: m.topk_reduce_backward(z(T, H), z(8, H), i, w.double(), z(8, H), w), lambda: m.topk_reduce_backward(z(3, H), z(8, H), i, w, z(8, H), w),
                lambda: m.topk_reduce_backward(z(T, H), z(8, H), i, w, z(8, H), w, route_rows=i.view(-1)[:7]),
                lambda: m.route_prep_backward(i, w, w, z(T, 8)), lambda: m.route_prep_backward(i, w, w, z(3, 8, dt=F32)),
                lambda: m.route_prep_backward(i.cpu(), w, w, z(T, 8, dt=F32))):
        with pytest.raises(AssertionError):
            bad()
    with pytest.raises(m.MoeError):                         # y is needed for dweights
        m.topk_reduce_backward(z(T, H), None, i, w, z(8, H), w)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("T,E,k,H,I", [(1, 4, 2, 256, 128), (50, 8, 2, 264, 144), (300, 4, 2, 512, 256)])
def test_training_step(T, E, k, H, I, saved):
    """Routing, forward and backward as a training program runs them, each operator on what the one before it
    wrote; every result against the float64 definition on that step's own inputs."""
    print("training step T=%d E=%d k=%d H=%d I=%d saved=%d" % (T, E, k, H, I, saved), flush=True)
    d = dev()
    new = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=d)
    logits, x = randn((T, E), F32, 1).to(d), randn((T, H), BF, 2).to(d)
    w13, w2 = randn((E, 2 * I, H), BF, 3, H ** -0.5).to(d), randn((E, H, I), BF, 4, I ** -0.5).to(d)
    dout = randn((T, H), BF, 5, 0.1).to(d)
    R, G = T * k, -(-H // 128)
    ids, w, d2s, rows, offs = m.route_prep(logits, k)
    # the layer's input, replicated per route: 16-bit rows as bytes, or the 8-bit rows with their scales
    xr = new(R, H)
    none = torch.empty((T, 0), dtype=F32, device=d)
    m.gather_rows_scales(x.view(torch.uint8), none, d2s, xr.view(torch.uint8), torch.empty((R, 0), dtype=F32, device=d), g=0)
    xq, xs, xrq, xrs = new(T, H, dt=torch.uint8), new(T, G, dt=F32), new(R, H, dt=torch.uint8), new(R, G, dt=F32)
    if saved:
        m.act_checkpoint(x, xq, xs)
        m.gather_rows_scales(xq, xs, d2s, xrq, xrs)
    # forward
    g2 = 2 * -(-I // 128)
    c1, h, cq, cs = new(R, 2 * I), new(R, I), new(R, 2 * I, dt=torch.uint8), new(R, g2, dt=F32)
    m.b16_grouped_gemm(xr, w13, c1, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    m.act_checkpoint(c1, cq, cs, act=1, h=h)
    y, out = new(R, H), new(T, H)
    m.b16_grouped_gemm(h, w2, y, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    m.topk_reduce(y, ids, w, out, route_rows=rows)
    # backward
    dy, dw, dl = new(R, H), new(T, k, dt=F32), new(T, E, dt=F32)
    m.topk_reduce_backward(dout, y, ids, w, dy, dw, route_rows=rows)
    m.route_prep_backward(ids, w, dw, dl)
    dh, dc1, h2 = new(R, I), new(R, 2 * I), new(R, I)
    m.b16_grouped_gemm(dy, w2, dh, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, w_trans=True)
    m.gated_act_backward(dh, cq, cs, dc1, act=1, h=h2)
    dw2, dw13 = new(E, H, I, dt=F32), new(E, 2 * I, H, dt=F32)
    m.b16_grouped_wgrad(dy, h2, offs, dw2)
    if saved and H % 16:                                    # saved rows need a width of whole 16-byte pieces
        with pytest.raises(m.MoeError):
            m.b16_grouped_wgrad(dc1, xrq, offs, dw13, a_s=xrs)
        return
    m.b16_grouped_wgrad(dc1, xrq if saved else xr, offs, dw13, a_s=xrs if saved else None)
    dxr, dx = new(R, H), new(T, H)
    m.b16_grouped_gemm(dc1, w13, dxr, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, w_trans=True)
    m.topk_reduce(dxr, ids, torch.ones_like(w), dx, route_rows=rows)
    torch.cuda.synchronize()

    o, idn, wn, rn = offs.cpu().numpy(), ids.cpu().numpy(), f64(w), rows.cpu().numpy()
    assert torch.equal(xr, x[d2s.long()])
    for got, a, bank, trans, n in ((c1, xr, w13, False, H), (y, h, w2, False, I), (dh, dy, w2, True, H), (dxr, dc1, w13, True, 2 * I)):
        ref, mag = tr.grouped_gemm(f64(a), f64(bank), o, trans)
        check(got, ref, sum_bound(n, mag, BF)(ref), "product")
    rdy, rdw, mag = tr.reduce_backward(f64(dout), f64(y), idn, wn, rn)
    check(dy, rdy, HALF[BF] * np.abs(rdy) * (1 + 2 * U) + 2 * U * np.abs(rdy) + TINY[BF], "dy")
    check(dw, rdw, (H + 8) * 2 * U * mag + 2.0 ** -140, "dweights")
    longest = int(np.diff(o).max())
    ref, mag = tr.grouped_wgrad(f64(dy), f64(h2), o)
    check(dw2, ref, sum_bound(longest + 20, mag, F32)(ref), "dW2")
    if saved:
        xv = f64(xrq.cpu().view(torch.float8_e4m3fn)) * np.repeat(f64(xrs), 128, axis=1)[:, :H]
        assert np.all(np.abs(xv - f64(xr)) <= 2.0 ** -4 * np.abs(f64(xr)) + 2.0 ** -10 * np.repeat(f64(xrs), 128, axis=1)[:, :H])
    else:
        xv = f64(xr)
    ref, mag = tr.grouped_wgrad(f64(dc1), xv, o)
    check(dw13, ref, sum_bound(longest + 20, mag, F32)(ref), "dW13")

    # the whole step in float64 from its inputs: what separates the two is the 16-bit rounding of each result (2^-8
    # relative a step, about six steps deep) and, in the gradients through the activation, the 8-bit rounding of the
    # saved values (2^-4 of each at most, and errors of different elements are independent)
    c164, _ = tr.grouped_gemm(f64(xr), f64(w13), o)
    h64 = tr.gated_act(1, c164)
    y64, _ = tr.grouped_gemm(h64, f64(w2), o)
    rel = lambda a, b: np.linalg.norm(a - b) / np.linalg.norm(b)
    assert rel(f64(out), tr.reduce(y64, idn, wn, rn)) < 6 * 2.0 ** -8
    dy64, dw64, _ = tr.reduce_backward(f64(dout), y64, idn, wn, rn)
    dh64, _ = tr.grouped_gemm(dy64, f64(w2), o, trans=True)
    dc164 = tr.gated_act_backward(1, c164, dh64)
    for got, want in ((dw2, tr.grouped_wgrad(dy64, h64, o)[0]), (dw13, tr.grouped_wgrad(dc164, f64(xr), o)[0])):
        assert rel(f64(got), want) < 2 * 2.0 ** -4
    dx64 = tr.reduce(tr.grouped_gemm(dc164, f64(w13), o, trans=True)[0], idn, np.ones_like(wn), rn)
    assert rel(f64(dx), dx64) < 2 * 2.0 ** -4
