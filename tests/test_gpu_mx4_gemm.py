"""The MXFP4 products against float64: every tile, ragged and odd sizes, maps, masks, the slot form, the fused requant."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from mx4_util import ACTS, decode, product_bound, random_mx, to_gpu
from train_util import HALF, TINY, Guarded, f64, offsets_of, replayed

pytestmark = pytest.mark.gpu
G, S = m.MOE_MODE_GROUPED, m.MOE_MODE_SLOT


class Problem:
    """Random operands of E experts: `rows` rows of A, banks [E, N, K]."""

    def __init__(self, E, rows, N, K, seed=0, lo=120, hi=126):
        rng = np.random.default_rng(seed + E * 7 + rows * 3 + N + K)
        self.E, self.N, self.K = E, N, K
        (self.aq, self.as_), (self.wq, self.ws) = random_mx(rng, (rows, K), lo, hi), random_mx(rng, (E, N, K), lo, hi)
        self.a, self.w = decode(self.aq, self.as_), decode(self.wq, self.ws)
        self.gpu = to_gpu(self.aq, self.as_) + to_gpu(self.wq, self.ws)

    def exact(self, ar, experts):
        """(products, magnitudes) of rows ar (-1: zeros) with their experts (-1: zeros)."""
        out, mag = np.zeros((len(ar), self.N)), np.zeros((len(ar), self.N))
        for r, (i, e) in enumerate(zip(ar, experts)):
            if i >= 0 and e >= 0:
                out[r], mag[r] = self.w[e] @ self.a[i], np.abs(self.w[e]) @ np.abs(self.a[i])
        return out, mag


def close(got, ref, mag, K, dt):
    got, b = f64(got), product_bound(K, mag)
    bad = np.abs(got - ref) > b + HALF[dt] * (np.abs(ref) + b) + TINY[dt]
    assert np.isfinite(got).all() and not bad.any(), (bad.sum(), np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4])


def experts_of(counts):
    return np.repeat(np.arange(len(counts)), counts)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("counts,N,K", [
    ([1], 8, 32), ([5], 64, 64), ([0, 3, 0, 1], 72, 96), ([17, 0, 40, 1], 136, 288), ([300], 520, 544), ([33, 31], 264, 1024),
    ([70, 0, 130, 65], 320, 800), ([257, 255, 1], 264, 320), ([513, 700], 520, 512), ([64] * 9, 1000, 2048), ([1] * 40, 48, 160),
])
def test_grouped(dt, counts, N, K):
    R = sum(counts)
    p = Problem(len(counts), R, N, K)
    g = Guarded((R + 2, N), dt, pad=8)
    offs = torch.from_numpy(offsets_of(counts)).to(dev())
    print("mx4 grouped", counts, N, K, dt, m.mx4_grouped_tile(R + 2, len(counts), N, K), flush=True)
    aq = torch.cat([p.gpu[0], p.gpu[0][:1], p.gpu[0][:1]])
    as_ = torch.nn.functional.pad(torch.cat([p.gpu[1], p.gpu[1][:1], p.gpu[1][:1]]), (0, -(K // 32) % 4), value=255)[:, :K // 32]
    m.mx4_grouped_gemm(aq, as_, *p.gpu[2:], g.view, mode=G, expert_offsets=offs)
    torch.cuda.synchronize()
    close(g.view[:R], *p.exact(range(R), experts_of(counts)), K, dt)
    assert (g.view[R:] == g.fill).all() and g.intact()         # rows behind the last expert's stay


def tile_cases():
    """Of every tile that some problem takes, the one of least work; odd sizes."""
    found = {}
    for R in (24, 40, 333, 900, 1500, 2600, 5001):
        for E in (1, 2, 4, 16, 30):
            for N in (64, 200, 1000, 2000, 5000):
                for K in (160, 544, 1056, 2048):
                    t, work = m.mx4_grouped_tile(R, E, N, K), R * N * K
                    if t not in found or work < found[t][0]:
                        found[t] = (work, (R, E, N, K))
    every = {m.mx4_grouped_tile(R, E, N, K) for R in (1, 30, 300, 3000, 30000) for E in (1, 8, 64, 256) for N in (64, 512, 4096) for K in (256, 2048)}
    assert every <= set(found), every - set(found)
    return [case for _, case in found.values()]


def test_every_tile():
    """Ragged rows; expected products on the GPU in float64 from the decoded operands."""
    for case in tile_cases():
        every_tile(*case)


def last_round_cases():
    """Of the large tiles: launches whose last round leaves less and more than half of the card idle, or is their only one."""
    slots = torch.cuda.get_device_properties(0).multi_processor_count // 8 * 8
    found = {}
    for counts in [(700,), (2348, 1900), (3000,), (5000,), (1500, 1400, 700, 900), (6000, 2000), (4096, 300), (1290, 0, 130)]:
        for N in (520, 1032, 2056, 4360, 6152, 8200):
            for K in (544, 640):
                bp, bq = m.mx4_grouped_tile(sum(counts), len(counts), N, K)
                tiles = sum(-(-c // bp) for c in counts) * -(-N // bq)
                what, work = (bp, K % 128, tiles > slots, 0 < tiles % slots * 2 <= slots), sum(counts) * N * K
                if bp >= 128 and (what not in found or work < found[what][0]):
                    found[what] = (work, (counts, N, K))
    assert {(256, 0, True, True), (256, 0, True, False), (128, 0, True, True), (256, 32, True, True)} <= set(found) or slots != 256
    return [case for _, case in found.values()]


def test_last_rounds():
    for counts, N, K in last_round_cases():
        every_tile(sum(counts), len(counts), N, K, counts)
        if N % 64 == 8:
            fused_in_every_tile(sum(counts), len(counts), N, K, counts)


def every_tile(R, E, N, K, counts=None):
    rng = np.random.default_rng(R)
    counts = rng.multinomial(R, rng.dirichlet(np.ones(E))) if counts is None else counts
    p = Problem(E, R, N, K)
    out = torch.empty((R, N), dtype=torch.float32, device=dev())
    print("mx4 tile", R, E, N, K, m.mx4_grouped_tile(R, E, N, K), flush=True)
    m.mx4_grouped_gemm(*p.gpu, out, mode=G, expert_offsets=torch.from_numpy(offsets_of(counts)).to(dev()))
    at = 0
    for e, n in enumerate(counts):
        a, w = torch.from_numpy(p.a[at:at + n]).cuda(), torch.from_numpy(p.w[e]).cuda()
        close(out[at:at + n], (a @ w.t()).cpu().numpy(), (a.abs() @ w.abs().t()).cpu().numpy(), K, torch.float32)
        at += n


@pytest.mark.parametrize("mode", [G, S])
def test_row_map(mode):
    """Rows by a map: repeated, in any order, outside of A (zeros)."""
    counts, N, K, rows = [20, 0, 45, 3], 72, 352, 19
    R = sum(counts)
    p = Problem(4, rows, N, K)
    rng = np.random.default_rng(1)
    amap = rng.integers(-3, rows + 3, R).astype(np.int32)
    amap[:3] = [2 ** 31 - 1, -2 ** 31, rows]
    ar = np.where((amap >= 0) & (amap < rows), amap, -1)
    out = torch.full((R, N), 9.0, device=dev())
    how = dict(expert_offsets=torch.from_numpy(offsets_of(counts)).to(dev())) if mode == G else dict(
        slot_ids=torch.from_numpy(experts_of(counts).astype(np.int32)).to(dev()))
    m.mx4_grouped_gemm(*p.gpu, out, mode=mode, a_rows=torch.from_numpy(amap).to(dev()), **how)
    close(out, *p.exact(ar, experts_of(counts)), K, torch.float32)
    assert (out[torch.from_numpy(ar < 0).to(dev())] == 0).all()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("rows,div,E,N,K", [(1, 1, 1, 8, 32), (8, 8, 64, 192, 2048), (6, 3, 5, 1000, 544), (16, 1, 3, 72, 512), (7, 2, 4, 24, 7168), (5, 5, 2, 40, 96)])
def test_slot(dt, rows, div, E, N, K):
    p = Problem(E, -(-rows // div), N, K)
    slots = np.random.default_rng(rows).integers(0, E, rows).astype(np.int32)
    slots[rows // 2:rows // 2 + 1] = -1 if rows > 1 else 0
    if rows > 4:
        slots[1], slots[3] = E, -5
    g = Guarded((rows, N), dt)
    m.mx4_grouped_gemm(*p.gpu, g.view, mode=S, slot_ids=torch.from_numpy(slots).to(dev()), a_row_div=div)
    torch.cuda.synchronize()
    live = (slots >= 0) & (slots < E)
    close(g.view, *p.exact(np.arange(rows) // div, np.where(live, slots, -1)), K, dt)
    got = f64(g.view)
    assert (got[~live] == 0).all() and not np.signbit(got[~live]).any() and g.intact()


def test_slot_reads_nothing_of_an_inactive_route():
    p = Problem(2, 4, 64, 256)
    aq, as_, wq, ws = p.gpu
    as_[1] = 255                                               # NaN scales of the row and the expert that no route names
    ws[1] = 255
    out = torch.empty((4, 64), device=dev())
    m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=S, slot_ids=torch.tensor([0, -1, 0, 0], dtype=torch.int32, device=dev()))
    assert (out[1] == 0).all() and torch.isfinite(out).all()


def test_empty_bank():
    out = torch.full((3, 16), 5.0, device=dev())
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev())  # noqa: E731
    m.mx4_grouped_gemm(u(3, 64), u(3, 4), u(0, 16, 64), u(0, 16, 4), out, mode=S, slot_ids=torch.tensor([0, -1, 3], dtype=torch.int32, device=dev()))
    assert (out == 0).all()


@pytest.mark.parametrize("mode", [G, S])
@pytest.mark.parametrize("K", [256, 288, 1056])
def test_nan_scales_reach_their_sums_alone(mode, K):
    counts, N = [9, 8], 40
    p = Problem(2, 17, N, K)
    aq, as_, wq, ws = p.gpu
    as_[4, K // 32 - 1] = 255
    ws[1, 7, 0] = 255
    out = torch.empty((17, N), device=dev())
    how = dict(expert_offsets=torch.tensor([0, 9, 17], dtype=torch.int32, device=dev())) if mode == G else dict(
        slot_ids=torch.from_numpy(experts_of(counts).astype(np.int32)).to(dev()))
    m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=mode, **how)
    want = torch.zeros((17, N), dtype=torch.bool)
    want[4], want[9:, 7] = True, True
    assert torch.equal(torch.isnan(out).cpu(), want) and torch.isfinite(out).cpu().logical_or(want).all()


@pytest.mark.parametrize("mode", [G, S])
def test_rows_outside_are_zeros_that_a_nan_of_the_bank_reaches(mode):
    """0 * NaN: what a row of zeros in A itself gives."""
    N, K = 40, 1056
    p = Problem(2, 5, N, K)
    aq, as_, wq, ws = p.gpu
    aq[2], as_[2], ws[1, 7, 3] = 0, 0, 255
    amap = torch.tensor([-1, 2, 5, 1], dtype=torch.int32, device=dev())
    how = dict(expert_offsets=torch.tensor([0, 0, 4], dtype=torch.int32, device=dev())) if mode == G else dict(
        slot_ids=torch.ones(4, dtype=torch.int32, device=dev()))
    out = torch.empty((4, N), device=dev())
    m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=mode, a_rows=amap, **how)
    zeros = torch.zeros(N, device=dev())
    zeros[7] = float("nan")
    for r in range(3):
        assert torch.equal(torch.isnan(out[r]), torch.isnan(zeros)) and (torch.nan_to_num(out[r]) == 0).all()
    assert torch.isnan(out[3, 7]) and torch.isfinite(out[3]).sum() == N - 1


def test_decreasing_offsets_leave_out_untouched():
    p = Problem(3, 20, 64, 256)
    for offs in ([0, 12, 5, 20], [0, 20, 20, 19]):
        out = torch.full((20, 64), 3.0, device=dev())
        m.mx4_grouped_gemm(*p.gpu, out, mode=G, expert_offsets=torch.tensor(offs, dtype=torch.int32, device=dev()))
        assert (out == 3.0).all()


def test_offsets_are_clamped():
    p = Problem(3, 20, 64, 256)
    out, want = (torch.full((20, 64), 3.0, device=dev()) for _ in range(2))
    m.mx4_grouped_gemm(*p.gpu, out, mode=G, expert_offsets=torch.tensor([-4, 8, 30, 40], dtype=torch.int32, device=dev()))
    m.mx4_grouped_gemm(*p.gpu, want, mode=G, expert_offsets=torch.tensor([0, 8, 20, 20], dtype=torch.int32, device=dev()))
    assert torch.equal(out, want)


def test_extreme_scales():
    """Scales whose products leave fp32's range on the way to a result within it, and subnormal results."""
    p = Problem(1, 4, 16, 128, lo=127, hi=127)
    aq, as_, wq, ws = p.gpu
    out = torch.empty((4, 16), device=dev())
    offs = torch.tensor([0, 4], dtype=torch.int32, device=dev())
    for sa, sw in ((254, 0), (0, 254), (60, 60), (64, 62)):
        as_.fill_(sa)
        ws.fill_(sw)
        m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=G, expert_offsets=offs)
        f = 2.0 ** (sa + sw - 254)
        ref, mag = p.exact(range(4), [0] * 4)
        assert (np.abs(f64(out) - ref * f) <= product_bound(128, mag * f) + 2.0 ** -149).all()


def test_strided_operands_and_offsets_past_32_bits():
    """Experts 2.2 GB apart, rows of A 1.1 GB apart, output rows 4.3 GB apart."""
    N, K, rows = 24, 288, 4
    p = Problem(3, rows, N, K)
    aq, as_, wq, ws = p.gpu

    def spread(t, stride):
        buf = torch.empty((t.shape[0] - 1) * stride + t[0].numel() * 2 + 4096, dtype=t.dtype, device=dev())
        view = buf.as_strided(t.shape, (stride,) + tuple(st for st in (t.stride() if t.dim() == 2 else t.stride())[1:]))
        view.copy_(t)
        return view
    big_w = spread(wq.contiguous(), (1 << 31) + (1 << 27))
    big_a = spread(aq.contiguous(), 1 << 30)
    out = torch.empty(3 * ((1 << 30) + 8) + 64, device=dev()).as_strided((rows, N), ((1 << 30) + 8, 1))
    m.mx4_grouped_gemm(big_a, as_, big_w, ws, out, mode=G, expert_offsets=torch.tensor([0, 1, 1, 4], dtype=torch.int32, device=dev()))
    close(out, *p.exact(range(rows), [0, 2, 2, 2]), K, torch.float32)
    out.zero_()
    m.mx4_grouped_gemm(big_a, as_, big_w, ws, out, mode=S, slot_ids=torch.tensor([0, 2, 1, 2], dtype=torch.int32, device=dev()))
    close(out, *p.exact(range(rows), [0, 2, 1, 2]), K, torch.float32)


@pytest.mark.parametrize("mode", [G, S])
@pytest.mark.parametrize("act", sorted(ACTS))
@pytest.mark.parametrize("rule", [0, 1])
@pytest.mark.parametrize("counts,I,K", [([5], 32, 32), ([40, 0, 7], 96, 288), ([130, 64, 1], 160, 1056), ([3, 300], 768, 512)])
def test_fused_is_the_two_calls(mode, act, rule, counts, I, K):
    """Bit for bit the product in fp32 and the quantisation of it."""
    R, E = sum(counts), len(counts)
    p = Problem(E, R, 2 * I, K)
    print("mx4 fused", mode, act, rule, counts, I, K, flush=True)
    slots = experts_of(counts).astype(np.int32)
    if mode == S:
        slots[::3] = -1
    how = dict(mode=mode, expert_offsets=torch.from_numpy(offsets_of(counts)).to(dev())) if mode == G else dict(
        mode=mode, slot_ids=torch.from_numpy(slots).to(dev()))
    c1 = torch.empty((R, 2 * I), device=dev())
    m.mx4_grouped_gemm(*p.gpu, c1, **how)
    wq, ws = (torch.empty(s, dtype=torch.uint8, device=dev()) for s in ((R, I // 2), (R, I // 32)))
    m.mx4_quant(c1, wq, ws, act=ACTS[act], rule=rule)
    gq, gs = Guarded((R, I // 2), torch.uint8, pad=6), Guarded((R, I // 32), torch.uint8, pad=3)
    m.mx4_grouped_gemm_act_quant(*p.gpu, gq.view, gs.view, act=ACTS[act], rule=rule, **how)
    torch.cuda.synchronize()
    assert torch.equal(gs.view, ws) and torch.equal(gq.view, wq) and gq.intact() and gs.intact()


def test_fused_in_every_tile():
    for case in tile_cases():
        fused_in_every_tile(*case)


def fused_in_every_tile(R, E, N, K, counts=None):
    I = -(-N // 64) * 32
    counts = np.random.default_rng(R).multinomial(R, np.ones(E) / E) if counts is None else counts
    p = Problem(E, R, 2 * I, K)
    offs = torch.from_numpy(offsets_of(counts)).to(dev())
    c1 = torch.empty((R, 2 * I), device=dev())
    m.mx4_grouped_gemm(*p.gpu, c1, mode=G, expert_offsets=offs)
    want, got = ([torch.empty(s, dtype=torch.uint8, device=dev()) for s in ((R, I // 2), (R, I // 32))] for _ in range(2))
    m.mx4_quant(c1, *want, act=1)
    m.mx4_grouped_gemm_act_quant(*p.gpu, *got, mode=G, expert_offsets=offs)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("mode", [G, S])
def test_captured(mode):
    counts, I, K = [9, 0, 20], 64, 512
    R = sum(counts)
    p, other = Problem(3, R, 2 * I, K), [Problem(3, R, 2 * I, K, seed=s) for s in (1, 2, 3)]
    offs = torch.from_numpy(offsets_of(counts)).to(dev())
    slots = torch.from_numpy(experts_of(counts).astype(np.int32)).to(dev())
    out = torch.empty((R, 2 * I), dtype=torch.bfloat16, device=dev())
    q, s = torch.empty((R, I // 2), dtype=torch.uint8, device=dev()), torch.empty((R, I // 32), dtype=torch.uint8, device=dev())
    how = dict(mode=mode, expert_offsets=offs, slot_ids=slots)

    def call():
        m.mx4_grouped_gemm(*p.gpu, out, **how)
        m.mx4_grouped_gemm_act_quant(*p.gpu, q, s, **how)

    def fresh(i):
        for t, o in zip(p.gpu, other[i].gpu):
            t.copy_(o)
        offs[1] = 9 - i
    for got, want in replayed(call, None, [out, q, s], fresh):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once():
    p, q = Problem(4, 400, 256, 512), Problem(4, 300, 512, 1024, seed=5)
    outs, want = [], []
    for x in (p, q):
        R = len(x.a)
        offs = torch.from_numpy(offsets_of([R // 4] * 4)).to(dev())
        out, ref = torch.empty((R, x.N), device=dev()), torch.empty((R, x.N), device=dev())
        m.mx4_grouped_gemm(*x.gpu, ref, mode=G, expert_offsets=offs)
        outs.append((x, out, offs))
        want.append(ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in outs]
    for _ in range(5):
        for st, (x, out, offs) in zip(streams, outs):
            m.mx4_grouped_gemm(*x.gpu, out, mode=G, expert_offsets=offs, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(o[1], w) for o, w in zip(outs, want))


def test_refusals():
    p = Problem(2, 8, 32, 288)
    aq, as_, wq, ws = p.gpu
    out = torch.empty((8, 32), device=dev())
    offs = torch.tensor([0, 4, 8], dtype=torch.int32, device=dev())
    how = dict(mode=G, expert_offsets=offs)
    for bad in (lambda: m.mx4_grouped_gemm(aq[:, :128], as_, wq, ws, out, **how), lambda: m.mx4_grouped_gemm(aq, as_[:, :8], wq, ws, out, **how),
                lambda: m.mx4_grouped_gemm(aq, as_.contiguous(), wq, ws, out, **how),      # 9 scale bytes a row, not padded
                lambda: m.mx4_grouped_gemm(aq, as_, wq, ws, out[:, :24], **how), lambda: m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=G, expert_offsets=offs[:2]),
                lambda: m.mx4_grouped_gemm(aq, as_, wq, ws, out, mode=S, slot_ids=offs), lambda: m.mx4_grouped_gemm(aq, as_, wq, ws, out, a_rows=offs, **how),
                lambda: m.mx4_grouped_gemm(aq.float(), as_, wq, ws, out, **how), lambda: m.mx4_grouped_gemm(aq, as_, wq, ws, out, m_rows=9, **how)):
        with pytest.raises((AssertionError, m.MoeError)):
            bad()
    with pytest.raises(m.MoeError):
        m.mx4_grouped_gemm(aq[:7], as_[:7], wq, ws, out, **how)                            # fewer rows than the call's
