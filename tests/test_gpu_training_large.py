"""GPU tests of the training operators at element offsets past 32 bits: the rows and matrices at the far end."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import HALF, TINY, check, f64, offsets_of, randn, sum_bound

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def test_product_output_and_input():
    """More than 2^31 output elements (K = 8), then more than 2^31 input elements (N = 8)."""
    R, W = 270000, 8192
    counts = [1000, R - 1000 - 77, 77]
    offs = offsets_of(counts)
    for N, K in ((W, 8), (8, W)):
        print("product R=%d N=%d K=%d" % (R, N, K), flush=True)
        g = torch.Generator(device="cuda")
        g.manual_seed(1)
        a = torch.empty((R, K), dtype=BF, device=dev()).normal_(generator=g)
        w = randn((3, N, K), BF, 2).to(dev())
        out = torch.empty((R, N), dtype=BF, device=dev())
        m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offs))
        torch.cuda.synchronize()
        for lo, hi, e in ((990, 1000, 0), (1000, 1010, 1), (R - 90, R - 77, 1), (R - 77, R, 2)):
            ref, mag = tr.grouped_gemm(f64(a[lo:hi]), f64(w[e:e + 1]), [0, hi - lo])
            check(out[lo:hi], ref, sum_bound(K, mag, BF)(ref), "rows %d" % lo)
        del a, out


def test_bank_and_gradient():
    """A bank and a gradient of more than 2^31 elements: the last experts."""
    E, N, K = 40, 8192, 8192
    counts = [0] * E
    counts[0], counts[37], counts[39] = 5, 3, 70
    R = sum(counts)
    w = torch.zeros((E, N, K), dtype=BF, device=dev())
    for e in (0, 37, 39):
        w[e] = randn((N, K), BF, e, 0.02).to(dev())
    a, dy, offs = randn((R, K), BF, 1).to(dev()), randn((R, N), BF, 2).to(dev()), to_dev(offsets_of(counts))
    out = torch.empty((R, N), dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    slot = torch.empty((1, N), dtype=F32, device=dev())
    m.b16_grouped_gemm(a[R - 1:], w, slot, mode=m.MOE_MODE_SLOT, slot_ids=torch.tensor([39], dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    for lo, hi, e in ((0, 5, 0), (5, 8, 37), (8, R, 39)):
        ref, mag = tr.grouped_gemm(f64(a[lo:hi]), f64(w[e:e + 1]), [0, hi - lo])
        check(out[lo:hi], ref, sum_bound(K, mag, F32)(ref), "expert %d" % e)
    check(slot, ref[-1:], sum_bound(K, mag[-1:], F32)(ref[-1:]), "slot")
    dw = w.fill_(7)
    m.b16_grouped_wgrad(dy, a, offs, dw)
    torch.cuda.synchronize()
    for lo, hi, e in ((0, 5, 0), (5, 8, 37), (8, R, 39)):
        ref, mag = tr.grouped_wgrad(f64(dy[lo:hi]), f64(a[lo:hi]), [0, hi - lo])
        check(dw[e], ref[0], sum_bound(hi - lo + 20, mag, BF)(ref)[0], "gradient of expert %d" % e)
    assert bool((dw[38] == 0).all()) and bool((dw[1:37:9] == 0).all())


def test_most_rows():
    """2^31 - 1 rows, the most there are, nearly all of one expert: counts rounded up to tiles and chunks pass an int."""
    R, W = 2 ** 31 - 1, 8
    at = [0, 3, 4, 5, 2 ** 30, R - 2, R - 1]
    a = torch.zeros((R, W), dtype=BF, device=dev())
    some = randn((len(at), W), BF, 1)
    for i, r in enumerate(at):
        a[r] = some[i].to(dev())
    w, offs = randn((2, W, W), BF, 2), to_dev(np.array([0, 4, R], np.int32))
    out = torch.full((R, W), 3.0, dtype=BF, device=dev())
    m.b16_grouped_gemm(a, w.to(dev()), out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    torch.cuda.synchronize()
    print("product of %d rows done" % R, flush=True)
    ref, mag = tr.grouped_gemm(f64(some), f64(w), [0, 2, len(at)])
    check(torch.stack([out[r] for r in at]), ref, sum_bound(W, mag, BF)(ref), "rows")
    for r in at:
        out[r] = 0
    for lo in range(0, R, 2 ** 28):
        assert bool((out[lo:lo + 2 ** 28] == 0).all()), "rows from %d" % lo
    dy = out
    other = randn((len(at), W), BF, 3)
    for i, r in enumerate(at):
        dy[r] = other[i].to(dev())
    dw = torch.empty((2, W, W), dtype=F32, device=dev())
    assert m.b16_grouped_wgrad_workspace_size(R, 2, W, W) > 0
    m.b16_grouped_wgrad(dy, a, offs, dw)
    torch.cuda.synchronize()
    ref, mag = tr.grouped_wgrad(f64(other), f64(some), [0, 2, len(at)])
    check(dw, ref, sum_bound(len(at) + 600, mag, F32)(ref), "gradient")     # zeros add without an error


def test_elementwise_rows():
    R, n = 1100000, 1024
    x = torch.zeros((R, 2 * n), dtype=BF, device=dev())
    tail = randn((3, 2 * n), BF, 3)
    x[-3:] = tail.to(dev())
    q = torch.empty((R, 2 * n), dtype=torch.uint8, device=dev())
    s = torch.empty((R, 16), dtype=F32, device=dev())
    m.act_checkpoint(x, q, s, act=5)
    dh, dx = torch.ones((R, n), dtype=BF, device=dev()), x
    m.gated_act_backward(dh, q, s, dx, act=5)
    torch.cuda.synchronize()
    for half in (0, 1):
        rq, rs = tr.save8(f64(tail[:, half * n:(half + 1) * n]))
        assert np.array_equal(f64(s[-3:, 8 * half:8 * half + 8]), rs)
        v = rq * np.repeat(rs, 128, axis=1)
        assert np.array_equal(f64(dx[-3:, (1 - half) * n:(2 - half) * n]), v)     # d up = gate, d gate = up: exact bf16 values
    assert bool((q[R // 2] == 0).all()) and bool((dx[R // 2] == 0).all())


def test_reduce_rows():
    T, k, H = 140000, 2, 8192
    dout = torch.ones((T, H), dtype=BF, device=dev())
    y = torch.full((T * k, H), 0.25, dtype=BF, device=dev())
    slots, w = torch.zeros((T, k), dtype=torch.int32, device=dev()), torch.full((T, k), 0.5, device=dev())
    w[-1, 1] = 3.0
    dw = torch.empty((T, k), device=dev())
    dy = torch.empty_like(y)
    m.topk_reduce_backward(dout, y, slots, w, dy, dw)
    torch.cuda.synchronize()
    assert bool((dw == 2048).all())
    assert bool((dy[-1] == 3).all()) and bool((dy[-2] == 0.5).all()) and bool((dy[0] == 0.5).all())
