"""GPU test of a training step whose router drops routes after the rows were laid out: their rows stay in the experts'
ranges, and must add nothing to any gradient."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from oracle import training as tr
from train_util import check, f64, randn, replayed, sum_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("T,E,k,H,I", [(5, 4, 2, 256, 128), (300, 8, 3, 264, 144)])
def test_step_with_dropped_routes(T, E, k, H, I):
    """As documented: dy is cleared before the reduce's backward.  In a graph that is replayed with other routes dropped
    each time, so what a step leaves in dy is another step's."""
    print("dropped routes T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I), flush=True)
    new = lambda *s, dt=BF: torch.empty(s, dtype=dt, device=dev())  # noqa: E731
    R = T * k
    x, dout = randn((T, H), BF, 2).to(dev()), randn((T, H), BF, 5, 0.1).to(dev())
    w13, w2 = randn((E, 2 * I, H), BF, 3, H ** -0.5).to(dev()), randn((E, H, I), BF, 4, I ** -0.5).to(dev())
    ids, w, d2s, rows, offs = m.route_prep(randn((T, E), F32, 1).to(dev()), k)
    slots = ids.clone()
    xr = x[d2s.long()].contiguous()
    c1, h, y, out, dy, dh, dc1, h2, dxr, dx = new(R, 2 * I), new(R, I), new(R, H), new(T, H), new(R, H), new(R, I), new(R, 2 * I), new(R, I), new(R, H), new(T, H)
    cq, cs = new(R, 2 * I, dt=torch.uint8), new(R, 2 * -(-I // 128), dt=F32)
    dw, dl, dw2, dw13 = new(T, k, dt=F32), new(T, E, dt=F32), new(E, H, I, dt=F32), new(E, 2 * I, H, dt=F32)
    ones = torch.ones_like(w)
    product = lambda *a, **kw: m.b16_grouped_gemm(*a, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, **kw)  # noqa: E731

    def step():
        product(xr, w13, c1)
        m.act_checkpoint(c1, cq, cs, act=1, h=h)
        product(h, w2, y)
        m.topk_reduce(y, slots, w, out, route_rows=rows)
        dy.zero_()
        m.topk_reduce_backward(dout, y, slots, w, dy, dw, route_rows=rows)
        m.route_prep_backward(ids, w, dw, dl)
        product(dy, w2, dh, w_trans=True)
        m.gated_act_backward(dh, cq, cs, dc1, act=1, h=h2)
        m.b16_grouped_wgrad(dy, h2, offs, dw2)
        m.b16_grouped_wgrad(dc1, xr, offs, dw13)
        product(dc1, w13, dxr, w_trans=True)
        m.topk_reduce(dxr, slots, ones, dx, route_rows=rows)

    def drop(i):
        gone = torch.from_numpy(np.random.default_rng(i).random((T, k)) < [0.3, 0.6, 1.0][i]).to(dev())
        slots.copy_(torch.where(gone, torch.full_like(ids, -1), ids))

    outputs = [dw, dl, dw2, dw13, dx]
    dy.fill_(float("nan"))
    for i, (got, want) in enumerate(replayed(step, None, outputs, drop)):
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        if i == 2:                                          # every route dropped: no gradient at all
            assert not any(bool(a.any()) for a in got)

    drop(0)
    dy.fill_(float("nan"))
    step()
    torch.cuda.synchronize()
    o, sn, wn, rn = offs.cpu().numpy(), slots.cpu().numpy(), f64(w), rows.cpu().numpy()
    rdy, rdw, _ = tr.reduce_backward(f64(dout), f64(y), sn, wn, rn)
    rdy = np.nan_to_num(rdy)                                # dropped routes' rows
    assert (sn < 0).any() and np.all(f64(dy)[rn[sn.reshape(-1) < 0]] == 0)
    # what the step's own 16-bit dy gives: a dropped route's row takes no part, so leaving it out changes nothing
    active = np.zeros(R, bool)
    active[rn[sn.reshape(-1) >= 0]] = True
    for got, a, b in ((dw2, dy, h2), (dw13, dc1, xr)):
        ref, mag = tr.grouped_wgrad(f64(a) * active[:, None], f64(b), o)
        check(got, ref, sum_bound(int(np.diff(o).max()) + 20, mag, F32)(ref), "weight gradient")
    assert np.abs(f64(dy) - rdy).max() <= 2.0 ** -8 * np.abs(rdy).max()
    ref, mag = tr.grouped_gemm(f64(dc1) * active[:, None], f64(w13), o, trans=True)
    check(dxr, ref, sum_bound(2 * I, mag, BF)(ref), "dx rows")
    assert np.all(f64(dw)[sn < 0] == 0)
    rdl = tr.route_backward(ids.cpu().numpy(), wn, f64(dw), E)
    assert np.allclose(f64(dl), rdl, rtol=0, atol=(k + 4) * 2.0 ** -22 * np.abs(f64(dw)).max())
