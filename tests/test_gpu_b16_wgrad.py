"""GPU tests of moe_b16_grouped_wgrad against the float64 definition."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import HALF, NAMES, TINY, Guarded, check, f64, offsets_of, randn, replayed, sum_bound

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def saved_rows(R, K, seed, pow2=True):
    """Codes, scales and values: through the library's own quantizers (they have tests of their own)."""
    x = randn((R, K), F32, seed)
    if R:
        x *= torch.exp(torch.linspace(-3, 3, R))[:, None]
    x = x.to(dev())
    q = torch.empty((R, K), dtype=torch.uint8, device=dev())
    s = torch.empty((R, -(-K // 128)), dtype=F32, device=dev())
    if R:
        (m.act_checkpoint if pow2 else m.act_quant)(x, q, s)
    v = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128, 1)[:, :K]
    return q, s, v.cpu().numpy()


def wgrad(counts, N, K, dt, odt, saved, seed, extra=0, accumulate=False, pow2=True):
    E, R = len(counts), int(sum(counts))
    print("wgrad E=%d R=%d N=%d K=%d %s->%s saved=%d acc=%d" % (E, R, N, K, NAMES[dt], NAMES[odt], saved, accumulate), flush=True)
    dy = randn((R + extra, N), dt, seed, 0.3)
    offs = offsets_of(counts)
    if saved:
        a, a_s, av = saved_rows(R + extra, K, seed + 1, pow2)
    else:
        a, a_s = randn((R + extra, K), dt, seed + 1).to(dev()), None
        av = f64(a)
    dyd = dy.to(dev())
    if extra:                                               # rows behind the last expert are not read
        dyd[R:] = float("nan")
        if saved:
            a_s[R:] = float("nan")
    out = Guarded((E, N, K), odt)
    old = randn((E, N, K), odt, seed + 2)
    if accumulate:
        out.view.copy_(old)
    m.b16_grouped_wgrad(dyd, a, to_dev(offs), out.view, a_s=a_s, accumulate=accumulate)
    torch.cuda.synchronize()
    assert out.intact()
    ref, mag = tr.grouped_wgrad(f64(dy[:R]), av[:R], offs)
    lost = HALF[dt] * mag if saved and not pow2 else 0.0     # a scale that is no power of two: one rounding to dt
    if accumulate:
        ref, mag = ref + f64(old), mag + np.abs(f64(old))
    longest = max(counts) if counts else 0
    bound = sum_bound(longest + 20, mag, odt)(ref) + lost * (1 + HALF[odt])
    check(out.view, ref, bound, "wgrad")
    return out


COUNTS = {"one": [1], "few": [3, 0, 16, 1, 0, 65], "many": [130, 0, 255, 129, 64], "long": [1500, 0, 700]}


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_rows_per_expert(counts, dt, saved):
    wgrad(COUNTS[counts], 136, 208, dt, F32, saved, seed=len(counts))


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("N,K", [(8, 16), (16, 8), (72, 112), (128, 128), (264, 272), (520, 1008), (1000, 528)])
def test_widths(N, K, saved):
    if saved and K % 16:
        K += 8
    wgrad(COUNTS["few"], N, K, BF, BF, saved, seed=N + K)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("counts,E,N,K", [("few", 128, 520, 272), ("one", 130, 512, 512)])
def test_large_tiles(counts, E, N, K, saved):
    """Enough tiles for the 256 x 256 form, most experts empty or short."""
    rng = np.random.default_rng(E)
    c = rng.integers(0, 90, E) * (rng.random(E) < 0.7)
    wgrad(list(c), N, K, BF, F32, saved, seed=E)


# rows an expert, matrix, and whether the rows are cut: each tile whole and cut, both forms of the join
PLANS = [([6001], 136, 80, True), ([0, 9000, 5], 72, 80, True), ([12000, 7000, 0, 1001], 512, 768, True), ([20000], 520, 528, True),
         ([65536], 1024, 1024, True), ([300], 2040, 4080, False), ([200, 0, 3, 64], 1032, 2064, False), ([1500, 1500], 1024, 512, None)]


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("counts,N,K,cut", PLANS)
def test_every_plan(counts, N, K, cut, saved):
    if cut is not None:
        assert (m.b16_grouped_wgrad_workspace_size(sum(counts), len(counts), N, K) > 0) == cut
    wgrad(counts, N, K, BF, F32, saved, seed=N)


@pytest.mark.parametrize("odt", [BF, FP, F32])
@pytest.mark.parametrize("counts,N,K", [([3, 9000, 0], 72, 80), ([12000, 8001], 512, 768)])
def test_cut_rows_added_on(counts, N, K, odt):
    assert m.b16_grouped_wgrad_workspace_size(sum(counts), len(counts), N, K) > 0
    one = wgrad(counts, N, K, FP, odt, False, seed=5, accumulate=True)
    two = wgrad(counts, N, K, FP, odt, False, seed=5, accumulate=True)
    assert torch.equal(one.view, two.view)


@pytest.mark.parametrize("saved", [False, True])
@pytest.mark.parametrize("odt", [BF, FP, F32])
@pytest.mark.parametrize("accumulate", [False, True])
def test_output_types(odt, accumulate, saved):
    wgrad(COUNTS["many"], 72, 144, BF, odt, saved, seed=5, accumulate=accumulate)
    wgrad(COUNTS["long"], 72, 144, FP, odt, saved, seed=6, accumulate=accumulate)


def test_saved_rows_with_other_scales():
    wgrad(COUNTS["many"], 136, 272, BF, F32, True, seed=7, pow2=False)
    wgrad(COUNTS["many"], 136, 272, FP, F32, True, seed=8, pow2=False)


def test_rows_behind_the_last_are_not_read():
    for saved in (False, True):
        wgrad([40, 0, 30], 72, 80, BF, F32, saved, seed=9, extra=50)


def test_cut_rows():
    """A long range over few tiles is cut and joined; the result holds the same bound and repeats bit for bit."""
    assert m.b16_grouped_wgrad_workspace_size(6001, 1, 136, 72) > 0
    for odt in (F32, BF):
        one = wgrad([6001], 136, 72, BF, odt, False, seed=10)
        two = wgrad([6001], 136, 72, BF, odt, False, seed=10)
        assert torch.equal(one.view, two.view)
    wgrad([0, 5000, 3], 40, 48, FP, F32, True, seed=11, accumulate=True)


def test_no_rows():
    for accumulate in (False, True):
        dw = torch.full((2, 16, 32), 4.0, dtype=BF, device=dev())
        z = torch.empty((0, 16), dtype=BF, device=dev())
        m.b16_grouped_wgrad(z, torch.empty((0, 32), dtype=BF, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev()),
                            dw, accumulate=accumulate)
        torch.cuda.synchronize()
        assert bool((dw == (4.0 if accumulate else 0.0)).all())


def test_strided_operands():
    R, N, K, c = 100, 72, 80, [60, 40]
    dy = torch.full((R, N + 16), float("nan"), dtype=BF)
    dy[:, 8:8 + N] = randn((R, N), BF, 1)
    a = torch.full((R, K + 16), float("nan"), dtype=BF)
    a[:, 8:8 + K] = randn((R, K), BF, 2)
    dyd, ad = dy.to(dev()), a.to(dev())
    dw = torch.empty((2, N, K), dtype=F32, device=dev())
    m.b16_grouped_wgrad(dyd[:, 8:8 + N], ad[:, 8:8 + K], to_dev(offsets_of(c)), dw)
    torch.cuda.synchronize()
    ref, mag = tr.grouped_wgrad(f64(dy[:, 8:8 + N]), f64(a[:, 8:8 + K]), offsets_of(c))
    check(dw, ref, sum_bound(60, mag, F32)(ref), "strided")


def test_unaligned_output():
    for odt, pad in ((BF, 1), (F32, 1), (FP, 4)):
        out = Guarded((2, 24, 40), odt, pad=pad)
        dy, a = randn((50, 24), BF, 1), randn((50, 40), BF, 2)
        m.b16_grouped_wgrad(dy.to(dev()), a.to(dev()), to_dev(offsets_of([20, 30])), out.view)
        torch.cuda.synchronize()
        assert out.intact()
        ref, mag = tr.grouped_wgrad(f64(dy), f64(a), offsets_of([20, 30]))
        check(out.view, ref, sum_bound(30, mag, odt)(ref), "unaligned")


@pytest.mark.parametrize("saved", [False, True])
def test_non_finite_values_stay_in_their_expert(saved):
    c, N, K = [10, 7, 70], 72, 144
    offs = offsets_of(c)
    dy = randn((87, N), BF, 1)
    dy[10, 5] = float("inf")                               # first row of expert 1
    if saved:
        q, s, _ = saved_rows(87, K, 2)
        q[16, 130] = 0x7F                                  # NaN code in its last row
        a, a_s = q, s
    else:
        a, a_s = randn((87, K), BF, 2).to(dev()), None
        a[16, 130] = float("nan")
    dw = torch.empty((3, N, K), dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy.to(dev()), a, to_dev(offs), dw, a_s=a_s)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(dw).cpu().numpy()
    want = np.zeros((3, N, K), bool)
    want[1, 5], want[1, :, 130] = True, True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("saved,counts", [(False, [40, 30]), (True, [40, 30]), (False, [3000, 1000])])
def test_graph_replay(saved, counts):
    R, N, K = int(sum(counts)), 72, 80
    dy = randn((R, N), BF, 1).to(dev())
    a, a_s, _ = saved_rows(R, K, 2) if saved else (randn((R, K), BF, 2).to(dev()), None, None)
    offs = to_dev(offsets_of(counts))
    dw = torch.empty((2, N, K), dtype=F32, device=dev())
    ws = torch.empty(m.b16_grouped_wgrad_workspace_size(R, 2, N, K) or 16, dtype=torch.uint8, device=dev())
    call = lambda: m.b16_grouped_wgrad(dy, a, offs, dw, a_s=a_s, workspace=ws)

    def fresh(i):
        dy.copy_(randn((R, N), BF, 20 + i))
        offs.copy_(torch.tensor([0, [R, 0, R // 3][i], R], dtype=torch.int32))

    for got, want in replayed(call, None, [dw], fresh):
        assert torch.equal(got[0], want[0])


def test_other_stream_with_a_workspace():
    dy, a = randn((6001, 72), BF, 1).to(dev()), randn((6001, 80), BF, 2).to(dev())
    offs = to_dev(offsets_of([6001]))
    one, two = torch.empty((1, 72, 80), dtype=F32, device=dev()), torch.empty((1, 72, 80), dtype=F32, device=dev())
    m.b16_grouped_wgrad(dy, a, offs, one)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.b16_grouped_wgrad(dy, a, offs, two, stream=s)
    s.synchronize()
    assert torch.equal(one, two)


def test_binding_checks():
    dy, a = torch.zeros((4, 16), dtype=BF, device=dev()), torch.zeros((4, 32), dtype=BF, device=dev())
    offs, dw = torch.zeros(3, dtype=torch.int32, device=dev()), torch.zeros((2, 16, 32), dtype=BF, device=dev())
    s = torch.zeros((4, 1), device=dev())
    for bad in (lambda: m.b16_grouped_wgrad(dy, a, offs, dw, a_s=s), lambda: m.b16_grouped_wgrad(dy, a.byte(), offs, dw),
                lambda: m.b16_grouped_wgrad(dy[:, :8], a, offs, dw), lambda: m.b16_grouped_wgrad(dy, a[:, :16], offs, dw),
                lambda: m.b16_grouped_wgrad(dy, a, offs[:2], dw), lambda: m.b16_grouped_wgrad(dy, a, offs, dw, m_rows=5),
                lambda: m.b16_grouped_wgrad(dy, a, offs.cpu(), dw)):
        with pytest.raises(AssertionError):
            bad()
    with pytest.raises(m.MoeError):
        m.b16_grouped_wgrad(dy, a.half(), offs, dw)
