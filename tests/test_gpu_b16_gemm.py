"""GPU tests of moe_b16_grouped_gemm against the float64 definition."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev, to_dev
from oracle import training as tr
from train_util import NAMES, Guarded, check, f64, offsets_of, randn, replayed, sum_bound

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def grouped(counts, N, K, dt, odt, trans, seed, extra=0, w=None, a=None):
    E, R = len(counts), int(sum(counts))
    print("b16 gemm E=%d R=%d N=%d K=%d %s->%s trans=%d" % (E, R, N, K, NAMES[dt], NAMES[odt], trans), flush=True)
    a = randn((R + extra, K), dt, seed) if a is None else a
    w = randn((E, K, N) if trans else (E, N, K), dt, seed + 1, 0.05) if w is None else w
    offs = offsets_of(counts)
    out = Guarded((R + extra, N), odt)
    m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out.view, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offs),
                       w_trans=trans)
    torch.cuda.synchronize()
    assert out.intact(), "wrote outside its rows and columns"
    if extra:
        assert bool((out.view[R:] == out.fill).all()), "rows behind the last expert changed"
    ref, mag = tr.grouped_gemm(f64(a[:R]), f64(w), offs, trans)
    if R:
        check(out.view[:R], ref, sum_bound(K, mag, odt)(ref), "grouped gemm")
    return out


# up to 16, 64, 256 and more rows an expert, tiles that end inside an expert, empty experts
COUNTS = {"one": [1], "few": [3, 0, 16, 1, 0, 17], "mid": [0, 33, 64, 65], "many": [130, 0, 255, 129, 1],
          "large": [300, 513], "last_empty": [5, 9, 0, 0]}


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("counts", sorted(COUNTS))
def test_rows_per_expert(counts, dt, trans):
    grouped(COUNTS[counts], 264, 200, dt, F32, trans, seed=len(counts))


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("N,K", [(8, 8), (8, 520), (16, 64), (72, 72), (128, 128), (256, 64), (264, 136), (520, 1000), (1000, 520)])
@pytest.mark.parametrize("counts", ["few", "large"])
def test_widths(counts, N, K, trans):
    grouped(COUNTS[counts], N, K, BF, BF, trans, seed=N + K)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("odt", [BF, FP, F32])
@pytest.mark.parametrize("counts", ["few", "mid", "many", "large"])
def test_output_types(counts, dt, odt):
    grouped(COUNTS[counts], 136, 328, dt, odt, False, seed=7)
    grouped(COUNTS[counts], 136, 328, dt, odt, True, seed=8)


# problems of each output tile: ragged rows, empty experts, last tiles of few and of many rows, whole tiles only, N and
# K that end inside a tile and a step
TILES = [((32, 64), [0, 33, 5, 64, 1], 264, 200), ((64, 64), [21, 0, 33, 18, 64, 40, 1, 23, 8, 15, 30, 20, 17, 29, 12, 2], 1000, 520),
         ((64, 256), [63, 64, 65, 0] * 8 + [50] * 8, 2056, 72), ((64, 256), [130, 7, 64, 0, 100, 128, 1] * 2, 2056, 136),
         ((128, 256), [129, 0, 127, 128, 1, 300] * 4, 1032, 136), ((128, 256), [2001, 1999], 1000, 72),
         ((256, 256), [2660, 3300, 1029, 2011], 1032, 72), ((256, 256), [2660, 3300, 0, 3040], 1032, 328),
         ((256, 256), [4096, 4096], 1032, 200), ((256, 256), [0, 0, 8000, 200, 1, 255, 257, 100], 1288, 136)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt,odt", [(BF, F32), (FP, FP), (BF, BF)])
@pytest.mark.parametrize("tile,counts,N,K", TILES)
def test_every_tile(tile, counts, N, K, dt, odt, trans):
    assert m.b16_grouped_tile(int(sum(counts)), len(counts), N, K) == tile
    grouped(counts, N, K, dt, odt, trans, seed=N + K + len(counts), extra=2)


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("tile,counts,N,K", [TILES[i] for i in (0, 1, 3, 4, 7)])
def test_every_tile_keeps_non_finite_values_apart(tile, counts, N, K, trans):
    c, R, E = counts, int(sum(counts)), len(counts)
    a, w = randn((R, K), BF, 1), randn((E, K, N) if trans else (E, N, K), BF, 2)
    offs = offsets_of(c)
    busy = [e for e in range(E) if c[e] > 0]
    r, e = int(offs[busy[-1]]), busy[0]
    a[r, K - 1] = float("nan")
    if trans:
        w[e, 3, N - 1] = float("inf")
    else:
        w[e, N - 1, 3] = float("inf")
    out = torch.empty((R, N), dtype=F32, device=dev())
    m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offs), w_trans=trans)
    torch.cuda.synchronize()
    want = np.zeros((R, N), bool)
    want[r] = True
    want[offs[e]:offs[e + 1], N - 1] = True
    assert np.array_equal(~torch.isfinite(out).cpu().numpy(), want)


@pytest.mark.parametrize("odt,pad", [(BF, 1), (F32, 1), (FP, 4), (F32, 2)])
def test_every_tile_with_unaligned_output(odt, pad):
    for tile, c, N, K in TILES[::2]:
        R = int(sum(c))
        a, w = randn((R, K), BF, 1), randn((len(c), N, K), BF, 2)
        out = Guarded((R, N), odt, pad=pad)
        m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out.view, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offsets_of(c)))
        torch.cuda.synchronize()
        assert out.intact()
        ref, mag = tr.grouped_gemm(f64(a), f64(w), offsets_of(c))
        check(out.view, ref, sum_bound(K, mag, odt)(ref), "unaligned output")


# large tiles whose last tiles of at most 128 rows would open one more round (they go to a launch of their own), rows and N
# of experts; then the same where a longer last tile opens it anyway
TAILS = [([2137, 2100, 2062, 1650], 4104), ([4200], 8192), ([0, 1920, 2048, 2100, 2049, 0, 1921, 1600], 4104),
         ([2137, 2100, 2062, 1737], 4104)]


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("dt,odt", [(BF, BF), (FP, F32)])
@pytest.mark.parametrize("counts,N", TAILS)
def test_last_tiles_of_a_full_round(counts, N, dt, odt, trans):
    K = 200
    assert m.b16_grouped_tile(sum(counts), len(counts), N, K) == (256, 256)
    grouped(counts, N, K, dt, odt, trans, seed=N, extra=5)


def test_last_tiles_keep_non_finite_values_apart_and_replay():
    counts, N, K = TAILS[0][0], TAILS[0][1], 72
    R = sum(counts)
    a, w = randn((R, K), BF, 1).to(dev()), randn((4, N, K), BF, 2, 0.05).to(dev())
    offs, out = to_dev(offsets_of(counts)), torch.empty((R, N), dtype=BF, device=dev())
    call = lambda: m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)  # noqa: E731

    def fresh(i):
        a.copy_(randn((R, K), BF, 10 + i))
        offs.copy_(to_dev(offsets_of([counts, [R - 6000, 3000, 2900, 100], counts[::-1]][i])))
        a[R - 1 - i, 3] = float("inf")
        a[2136 - i, 71] = float("nan")

    for got, eager in replayed(call, None, [out], fresh):
        assert torch.equal(got[0].nan_to_num(nan=7e4), eager[0].nan_to_num(nan=7e4))
        assert int((~torch.isfinite(got[0])).any(dim=1).sum()) == 2


def test_large_tiles_replayed():
    """The 256 x 256 and 128 x 256 tiles in a graph whose offsets change, some experts empty, then all rows in one."""
    for (R, E, N, K), cuts in (((9000, 4, 1032, 200), [(0, 9000, 9000), (2000, 2100, 6000), (9000, 9000, 9000)]),
                               ((4000, 4, 1000, 72), [(0, 0, 0), (1000, 1001, 3500), (128, 256, 384)])):
        a, w = randn((R, K), BF, 1).to(dev()), randn((E, K, N), BF, 2).to(dev())
        offs, out = to_dev(offsets_of([R, 0, 0, 0])), torch.empty((R, N), dtype=BF, device=dev())
        call = lambda: m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, w_trans=True)

        def fresh(i):
            offs.copy_(torch.tensor([0, *cuts[i], R], dtype=torch.int32))

        for got, want in replayed(call, None, [out], fresh):
            assert torch.equal(got[0], want[0])


def test_rows_behind_the_last_are_left():
    grouped([5, 0, 20], 64, 96, BF, BF, False, seed=3, extra=30)
    grouped([300, 290], 64, 96, FP, F32, True, seed=4, extra=3)


def test_many_experts():
    rng = np.random.default_rng(0)
    grouped(list(rng.integers(0, 4, 1024)), 40, 72, BF, F32, False, seed=5)
    grouped(list(rng.multinomial(3000, np.ones(256) / 256)), 264, 136, FP, FP, True, seed=6)


@pytest.mark.parametrize("counts,N,K", [("few", 2048, 2048), ("mid", 1536, 4096), ("large", 768, 2048)])
def test_long_reduction(counts, N, K):
    grouped(COUNTS[counts], N, K, BF, F32, False, seed=11)


def test_no_rows_at_all():
    out = torch.full((4, 64), 2.0, device=dev(), dtype=BF)
    a, w = torch.zeros((4, 64), device=dev(), dtype=BF), torch.zeros((3, 64, 64), device=dev(), dtype=BF)
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=torch.zeros(4, dtype=torch.int32, device=dev()))
    torch.cuda.synchronize()
    assert bool((out == 2).all())


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", ["few", "many", "large"])
def test_strided_operands(counts, trans):
    c = COUNTS[counts]
    R, N, K = int(sum(c)), 136, 200
    a = torch.full((R, K + 24), float("nan"), dtype=BF)
    a[:, 8:8 + K] = randn((R, K), BF, 1)
    rows, width = (K, N) if trans else (N, K)
    w = torch.full((len(c), rows + 2, width + 16), float("nan"), dtype=BF)
    w[:, 1:1 + rows, 8:8 + width] = randn((len(c), rows, width), BF, 2, 0.05)
    ad, wd = a.to(dev()), w.to(dev())
    out = torch.empty((R, N), dtype=F32, device=dev())
    m.b16_grouped_gemm(ad[:, 8:8 + K], wd[:, 1:1 + rows, 8:8 + width], out, mode=m.MOE_MODE_GROUPED,
                       expert_offsets=to_dev(offsets_of(c)), w_trans=trans)
    torch.cuda.synchronize()
    ref, mag = tr.grouped_gemm(f64(a[:, 8:8 + K]), f64(w[:, 1:1 + rows, 8:8 + width]), offsets_of(c), trans)
    check(out, ref, sum_bound(K, mag, F32)(ref), "strided")


@pytest.mark.parametrize("counts", ["few", "many", "large"])
@pytest.mark.parametrize("odt,pad", [(BF, 1), (F32, 1), (FP, 4), (F32, 2)])
def test_unaligned_output(counts, odt, pad):
    c = COUNTS[counts]
    R, N, K = int(sum(c)), 72, 64
    a, w = randn((R, K), BF, 1), randn((len(c), N, K), BF, 2)
    out = Guarded((R, N), odt, pad=pad)
    m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out.view, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offsets_of(c)))
    torch.cuda.synchronize()
    assert out.intact()
    ref, mag = tr.grouped_gemm(f64(a), f64(w), offsets_of(c))
    check(out.view, ref, sum_bound(K, mag, odt)(ref), "unaligned output")


@pytest.mark.parametrize("trans", [False, True])
@pytest.mark.parametrize("counts", ["few", "many", "large"])
def test_non_finite_values_stay_where_they_belong(counts, trans):
    """An infinity or NaN in one row of A or one expert's bank reaches that row's or column's outputs only, also
    next to the ends of experts, of K (no multiple of 64) and of N."""
    c = COUNTS[counts]
    R, N, K, E = int(sum(c)), 136, 200, len(c)
    a, w = randn((R, K), BF, 1), randn((E, K, N) if trans else (E, N, K), BF, 2)
    offs = offsets_of(c)
    busy = [e for e in range(E) if c[e] > 0]
    r, e = int(offs[busy[-1]]), busy[0]
    a[r, K - 1] = float("nan")
    if trans:
        w[e, 3, N - 1] = float("inf")
    else:
        w[e, N - 1, 3] = float("inf")
    out = torch.empty((R, N), dtype=F32, device=dev())
    m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offs), w_trans=trans)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(out).cpu().numpy()
    want = np.zeros((R, N), bool)
    want[r] = True
    want[offs[e]:offs[e + 1], N - 1] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("odt", [BF, FP, F32])
@pytest.mark.parametrize("N,K,rows,div", [(8, 8, 1, 1), (24, 520, 5, 2), (1536, 2048, 8, 8), (1000, 712, 17, 1), (264, 4104, 6, 3)])
def test_slot_mode(N, K, rows, div, dt, odt):
    print("slot N=%d K=%d rows=%d div=%d" % (N, K, rows, div), flush=True)
    E = 5
    a, w = randn((-(-rows // div), K), dt, N), randn((E, N, K), dt, K, 0.05)
    slots = np.random.default_rng(rows).integers(-1, E, rows).astype(np.int32)
    slots[rows // 2] = E                                    # beyond the bank: a zero row
    out = Guarded((rows, N), odt)
    m.b16_grouped_gemm(a.to(dev()), w.to(dev()), out.view, mode=m.MOE_MODE_SLOT, slot_ids=to_dev(slots), a_row_div=div)
    torch.cuda.synchronize()
    assert out.intact()
    ref, mag = tr.slot_gemm(f64(a), f64(w), slots, div)
    check(out.view, ref, sum_bound(K, mag, odt)(ref), "slot")
    off = (slots < 0) | (slots >= E)
    assert not np.any(np.signbit(f64(out.view)[off]))


def test_slot_mode_reads_nothing_of_inactive_rows():
    a = torch.full((2, 64), float("nan"), dtype=BF, device=dev())
    w = torch.full((1, 16, 64), float("nan"), dtype=BF, device=dev())
    out = torch.full((4, 16), float("nan"), dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_SLOT, slot_ids=torch.full((4,), -1, dtype=torch.int32, device=dev()), a_row_div=2)
    assert bool((out == 0).all())
    rc = m.lib().moe_b16_grouped_gemm(None, 64, None, 0, 64, 0, 16, 64, m.MOE_BF16, 0, m.MOE_MODE_SLOT, None,
                                      torch.full((4,), -1, dtype=torch.int32, device=dev()).data_ptr(), 4, 1,
                                      out.fill_(1).data_ptr(), m.MOE_F32, 16, m._stream())
    assert rc == m.MOE_OK
    torch.cuda.synchronize()
    assert bool((out == 0).all())


@pytest.mark.parametrize("mode,rows", [("grouped", 40), ("grouped", 900), ("trans", 300), ("slot", 6)])
def test_graph_replay(mode, rows):
    """One captured graph serves other row counts per expert: offsets, slots and values change in place."""
    E, N, K = 3, 136, 200
    a = randn((rows, K), BF, 1).to(dev())
    w = randn((E, K, N) if mode == "trans" else (E, N, K), BF, 2).to(dev())
    offs = to_dev(offsets_of([rows, 0, 0]))
    slots = torch.zeros(rows, dtype=torch.int32, device=dev())
    out = torch.empty((rows, N), dtype=BF, device=dev())

    def call():
        if mode == "slot":
            m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_SLOT, slot_ids=slots)
        else:
            m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, w_trans=mode == "trans")

    def fresh(i):
        a.copy_(randn((rows, K), BF, 10 + i))
        cut = sorted(np.random.default_rng(i).integers(0, rows + 1, 2))
        offs.copy_(torch.tensor([0, cut[0], cut[1], rows], dtype=torch.int32))
        slots.copy_(torch.from_numpy(np.random.default_rng(i).integers(-1, E, rows).astype(np.int32)))

    for got, want in replayed(call, None, [out], fresh):
        assert torch.equal(got[0], want[0])


def test_other_stream():
    a, w = randn((70, 200), BF, 1).to(dev()), randn((2, 136, 200), BF, 2).to(dev())
    offs = to_dev(offsets_of([33, 37]))
    one, two = torch.empty((70, 136), dtype=F32, device=dev()), torch.empty((70, 136), dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, one, mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    m.b16_grouped_gemm(a, w, two, mode=m.MOE_MODE_GROUPED, expert_offsets=offs, stream=s)
    s.synchronize()
    assert torch.equal(one, two)


def test_offsets_beyond_m_rows_are_clamped():
    a, w = randn((40, 64), BF, 1).to(dev()), randn((2, 32, 64), BF, 2).to(dev())
    out = torch.full((40, 32), 9.0, dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(np.array([0, 10, 40], np.int32)), m_rows=25)
    torch.cuda.synchronize()
    ref, mag = tr.grouped_gemm(f64(a[:25]), f64(w), [0, 10, 25])
    check(out[:25], ref, sum_bound(64, mag, F32)(ref), "clamped")
    assert bool((out[25:] == 9).all())


@pytest.mark.parametrize("offs", [[0, 30, 10, 40], [40, 0, 40, 40], [5, 5, 5, 4], [0, 40, -3, 40]])
@pytest.mark.parametrize("N,K", [(32, 64), (4096, 2048)])
def test_decreasing_offsets_leave_the_output(offs, N, K):
    a, w = randn((40, K), BF, 1).to(dev()), randn((3, N, K), BF, 2).to(dev())
    out = torch.full((40, N), 9.0, dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(np.array(offs, np.int32)))
    torch.cuda.synchronize()
    assert bool((out == 9).all())


def test_decreasing_offsets_of_every_expert():
    E = 1024
    a, w = randn((E, 8), BF, 1).to(dev()), randn((E, 8, 8), BF, 2).to(dev())
    out = torch.full((E, 8), 9.0, dtype=F32, device=dev())
    m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(np.arange(E, -1, -1, dtype=np.int32)))
    torch.cuda.synchronize()
    assert bool((out == 9).all())


@pytest.mark.parametrize("dt", [BF, FP])
@pytest.mark.parametrize("mode", ["forward", "trans", "slot"])
def test_subnormal_operands_count(dt, mode):
    """Values below a type's normal range (common among fp16 gradients) are not flushed."""
    tiny = {FP: 2.0 ** -20, BF: 2.0 ** -130}[dt]
    K, N = 200, 72
    a = torch.full((40, K), tiny, dtype=dt)
    w = randn((2, K, N) if mode == "trans" else (2, N, K), dt, 1).sign() * {FP: 1.0, BF: 2.0 ** 20}[dt]
    out = torch.empty((40, N), dtype=F32, device=dev())
    if mode == "slot":
        slots = np.arange(40, dtype=np.int32) % 2
        m.b16_grouped_gemm(a.to(dev()), w.to(dt).to(dev()), out, mode=m.MOE_MODE_SLOT, slot_ids=to_dev(slots))
        ref, _ = tr.slot_gemm(f64(a), f64(w), slots, 1)
    else:
        m.b16_grouped_gemm(a.to(dev()), w.to(dt).to(dev()), out, mode=m.MOE_MODE_GROUPED, expert_offsets=to_dev(offsets_of([25, 15])),
                           w_trans=mode == "trans")
        ref, _ = tr.grouped_gemm(f64(a), f64(w), [0, 25, 40], mode == "trans")
    assert np.array_equal(f64(out), ref)                   # sums of a few equal powers of two: exact


def test_binding_checks():
    a, w = torch.zeros((4, 64), dtype=BF, device=dev()), torch.zeros((2, 32, 64), dtype=BF, device=dev())
    out, offs = torch.zeros((4, 32), dtype=BF, device=dev()), torch.zeros(3, dtype=torch.int32, device=dev())
    kw = dict(mode=m.MOE_MODE_GROUPED, expert_offsets=offs)
    for bad in (lambda: m.b16_grouped_gemm(a.half(), w, out, **kw), lambda: m.b16_grouped_gemm(a[:, :56], w, out, **kw),
                lambda: m.b16_grouped_gemm(a, w, out[:, :24], **kw), lambda: m.b16_grouped_gemm(a[:3], w, out, **kw),
                lambda: m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_GROUPED, expert_offsets=offs.long()),
                lambda: m.b16_grouped_gemm(a.cpu(), w, out, **kw), lambda: m.b16_grouped_gemm(a, w, out, m_rows=5, **kw),
                lambda: m.b16_grouped_gemm(a, w, out, mode=m.MOE_MODE_SLOT, slot_ids=offs)):
        with pytest.raises(AssertionError):
            bad()
