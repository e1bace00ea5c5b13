"""The router against its definition in float64: ids and maps exactly, weights and scores within derived bounds."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from train_util import replayed

pytestmark = pytest.mark.gpu
SOFTMAX, SIGMOID = 0, 1
DTS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def scores64(x, score):
    """Scores of float64 logits; -inf masks."""
    x = np.where(np.isnan(x), -np.inf, np.minimum(x, 3.4028234663852886e38))
    if score == SIGMOID:
        t = np.exp(-np.abs(x))
        return np.where(x >= 0, 1 / (1 + t), t / (1 + t)), x
    top = x.max(axis=1, keepdims=True)
    with np.errstate(invalid="ignore"):
        e = np.where(x > -np.inf, np.exp(x - np.where(top > -np.inf, top, 0)), 0.0)
    z = e.sum(axis=1, keepdims=True)
    return np.divide(e, z, out=np.zeros_like(e), where=z > 0), x


def rounded(v):
    """Values as the router compares them: 43 significant bits."""
    mant, e = np.frexp(v)
    return np.where(np.isfinite(v), np.ldexp(np.round(mant * 2.0 ** 43), e - 43), v)


def reference(x, topk, score, bias, G, keep, top, renorm, scale):
    s, x = scores64(x.astype(np.float64), score)
    T, E = x.shape
    c = s + bias.astype(np.float64) if bias is not None else s
    rank = rounded(c) if bias is not None else x
    there = (x > -np.inf) & (c > -np.inf)                      # a NaN choice is none either
    ids = np.full((T, topk), -1, np.int32)
    w = np.zeros((T, topk))
    for t in range(T):
        ok = there[t].copy()
        if G > 1 and keep < G:
            size = E // G
            value = np.full(G, -np.inf)
            for g in range(G):
                members = [e for e in range(g * size, (g + 1) * size) if ok[e]]
                if members:
                    by = c[t] if top == 2 else rank[t]
                    value[g] = rounded(sum(sorted((by[e] for e in members), reverse=True)[:top]))
            best = [g for g in sorted(range(G), key=lambda g: (-value[g], g)) if value[g] > -np.inf][:keep]
            ok &= np.isin(np.arange(E) // size, best)
        order = [e for e in np.argsort(-np.where(ok, rank[t], -np.inf), kind="stable") if ok[e]][:topk]
        ids[t, :len(order)] = order
        if order:
            v = s[t, order]
            if renorm:
                low = x[t, order].max()
                low = min(low, 0.0) if score == SIGMOID else low
                l = x[t, order]
                v = np.exp(np.where((l >= 0) & (score == SIGMOID), 0.0, l - low)) / (1 + np.exp(-np.abs(l)) if score == SIGMOID else 1)
                v = v / v.sum()
            w[t, :len(order)] = scale * v
    return ids, w, s


def reference_maps(ids, E):
    T, k = ids.shape
    flat = ids.reshape(-1)
    order = sorted((i for i in range(T * k) if flat[i] >= 0), key=lambda i: (flat[i], i))
    d2s, rr = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
    d2s[:len(order)] = np.array(order, np.int64) // k
    rr[order] = np.arange(len(order))
    offs = np.concatenate([[0], np.cumsum(np.bincount(flat[flat >= 0], minlength=E))]).astype(np.int32)
    return d2s, rr, offs


# A weight is formed in 64 bits from fp32 logits (the softmax's sum over all experts in fp32 when nothing asks for more: each
# of its terms is within (4 + |d|) 2^-24, d e^-d weighted, and at most 6 + 16 additions round), then rounded once.
W_REL = 2.0 ** -19


def check(x, topk, score, bias=None, G=1, keep=1, top=2, renorm=True, scale=1.0, scores=False, dt="fp32", rows=None):
    x = torch.as_tensor(x).to(DTS[dt])
    T, E = x.shape
    b = None if bias is None else torch.as_tensor(bias, dtype=torch.float32)
    print("router T=%d E=%d topk=%d" % (T, E, topk), score, G, keep, top, renorm, dt, flush=True)
    r = m.router(x.to(dev()) if rows is None else rows, topk, score=score, bias=None if b is None else b.to(dev()), n_group=G, topk_group=keep,
                 group_top=top, renorm=renorm, scale=scale, want_scores=scores)
    torch.cuda.synchronize()
    ids, w, s = reference(x.double().numpy(), topk, score, None if b is None else b.numpy(), G, keep, top, renorm, scale)
    assert np.array_equal(r.expert_ids.cpu().numpy(), ids)
    d2s, rr, offs = reference_maps(ids, E)
    assert np.array_equal(r.expert_offsets.cpu().numpy(), offs)
    assert np.array_equal(r.route_rows.cpu().numpy(), rr)
    assert np.array_equal(r.dst2src.cpu().numpy(), d2s)
    got = r.weights.cpu().double().numpy()
    assert (np.abs(got - w) <= W_REL * np.abs(w) + scale * 2.0 ** -126).all(), np.abs(got - w).max()
    assert (got[ids < 0] == 0).all()
    if scores:
        d = np.abs(np.where(np.isfinite(x.double().numpy()), x.double().numpy(), 0))
        d = d + d.max(axis=1, keepdims=True)                   # |l - max| at most
        got = r.scores.cpu().double().numpy()
        assert (np.abs(got - s) <= (W_REL + d * 2.0 ** -24) * s + 2.0 ** -125).all()
    return r


def logits(T, E, seed, std=1.5):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((T, E)) * std + 0.5 * rng.standard_normal(E)).astype(np.float32)


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,topk", [(1, 8, 1), (3, 7, 7), (16, 64, 8), (17, 65, 6), (64, 256, 8), (65, 33, 4), (200, 300, 5), (129, 1024, 64), (70, 1, 1)])
def test_ranges(dt, score, with_bias, T, E, topk):
    bias = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.05 if with_bias else None
    check(logits(T, E, T + E), topk, score, bias, renorm=T % 2 == 0, scale=2.5 if E % 2 else 1.0, scores=E % 2 == 0, dt=dt)


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("top", [1, 2])
@pytest.mark.parametrize("T,E,topk,G,keep", [(5, 16, 2, 4, 1), (40, 64, 8, 8, 4), (100, 256, 8, 8, 4), (33, 160, 6, 8, 3), (20, 64, 4, 64, 5), (20, 512, 8, 64, 7),
                                             (9, 40, 8, 2, 2), (66, 1000, 9, 50, 10), (7, 12, 6, 2, 1)])
def test_groups(score, with_bias, top, T, E, topk, G, keep):
    bias = np.random.default_rng(E).standard_normal(E).astype(np.float32) * 0.1 if with_bias else None
    check(logits(T, E, T * E), topk, score, bias, G, keep, top, dt="fp32" if T % 2 else "bf16")


@pytest.mark.parametrize("T", [8192, 8193, 32768, 40001])
def test_many_tokens(T):
    """A chunk of 16 tokens, of 64, and the scan between."""
    E, topk = 32, 4
    x = torch.from_numpy(logits(T, E, T))
    x[::7] = -float("inf")
    r = m.router(x.to(dev()), topk, score=SIGMOID)
    top, ids = torch.sort(x, dim=1, descending=True, stable=True)
    ids = torch.where(top[:, :topk] > -float("inf"), ids[:, :topk], -1).int().numpy()
    assert np.array_equal(r.expert_ids.cpu().numpy(), ids)
    for got, want in zip((r.dst2src, r.route_rows, r.expert_offsets), reference_maps(ids, E)):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("T", [6, 100])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("with_bias,G,keep,top", [(False, 1, 1, 1), (True, 1, 1, 1), (False, 4, 2, 1), (False, 4, 2, 2), (True, 4, 2, 2)])
def test_masks_and_ties(T, score, with_bias, G, keep, top):
    """Rows without an expert, with fewer than topk, NaN and infinities, the type's lowest value, equal logits; experts that the
    bias takes away."""
    E = 32
    rng = np.random.default_rng(7)
    x = rng.integers(-2, 3, (T, E)).astype(np.float32)         # many ties
    x[0] = -np.inf
    x[1, 3:] = -np.inf
    x[2, :] = np.nan
    x[2, 9] = 0.5
    x[3] = np.finfo(np.float32).min
    x[3, 5] = 1.0
    x[4, 7] = np.inf
    x[4, 20:] = np.nan
    x[5] = 0.25
    bias = None
    if with_bias:
        bias = (rng.integers(-1, 2, E) * 0.125).astype(np.float32)
        bias[4], bias[11] = -np.inf, np.nan
    for renorm in (True, False):
        check(x, 6, score, bias, G, keep, top, renorm=renorm, scores=True)


def test_16_bit_ties():
    x = np.round(logits(300, 128, 3) * 4) / 4
    for score in (SOFTMAX, SIGMOID):
        check(x, 8, score, dt="bf16")
        check(x, 8, score, bias=np.zeros(128, np.float32), dt="fp16")


def test_scores_that_underflow_divide():
    """Renormalised weights of logits whose scores are below fp32's range, and of saturated ones."""
    x = np.full((4, 16), -1000.0, np.float32)
    x[0, :4] = [-200, -201, -202, -203]
    x[1, :4] = [-95, -96, -97, -98]
    x[2, :4] = [300, 299, 298, 50]
    x[3, :4] = [40, -120, -121, -122]
    check(x, 4, SIGMOID)
    check(x, 4, SOFTMAX)


def test_choices_next_to_each_other():
    """Biased scores that differ by 2^-36 of their value keep their order: an fp32 choice would not."""
    T, E = 64, 16
    rng = np.random.default_rng(5)
    x = rng.standard_normal((T, E)).astype(np.float32)
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    x[:] = x[0]
    bias = (0.75 - s).astype(np.float32)                       # every choice is 0.75 to an fp32 rounding
    check(x, 8, SIGMOID, bias)
    check(x, 8, SIGMOID, bias, G=4, keep=2, top=2)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strides_and_guards(dt):
    T, E, k = 70, 60, 4
    buf = torch.full((T, 2 * E + 5), 99.0, dtype=DTS[dt])
    x = torch.from_numpy(logits(T, E, 9)).to(DTS[dt])
    buf[:, 3:3 + E] = x
    rows = buf.to(dev())[:, 3:3 + E]
    check(x, k, SOFTMAX, dt=dt, rows=rows)
    # outputs in the middle of larger buffers
    i32 = lambda n: torch.full((n + 16,), 77, dtype=torch.int32, device=dev())  # noqa: E731
    bufs = [i32(T * k), torch.full((T * k + 16,), 77.0, device=dev()), i32(T * k), i32(T * k), i32(E + 1), torch.full((T * E + 16,), 77.0, device=dev())]
    out = (bufs[0][8:-8].view(T, k), bufs[1][8:-8].view(T, k), bufs[2][8:-8], bufs[3][8:-8], bufs[4][8:-8], bufs[5][8:-8].view(T, E))
    r = m.router(rows, k, out=out)
    ref = m.router(rows.contiguous(), k, want_scores=True)
    torch.cuda.synchronize()
    for a, b, buf in zip(r, ref, bufs):
        assert torch.equal(a, b) and (buf[:8] == 77).all() and (buf[-8:] == 77).all()


def test_without_maps_and_without_tokens():
    x = torch.from_numpy(logits(100, 64, 1)).to(dev())
    r, full = m.router(x, 8, maps=False), m.router(x, 8)
    assert r.dst2src is None and r.scores is None and torch.equal(r.expert_ids, full.expert_ids) and torch.equal(r.weights, full.weights)
    e = m.router(x[:0], 8)
    assert e.expert_ids.shape == (0, 8) and (e.expert_offsets == 0).all() and e.expert_offsets.numel() == 65
    assert m.router(x[:0], 8, maps=False).expert_offsets is None
    for bad in (lambda: m.router(x.t(), 8), lambda: m.router(x, 8, bias=x[0, :63]), lambda: m.router(x, 8, bias=x[0].double()),
                lambda: m.router(x, 8, out=full._replace(route_rows=None)), lambda: m.router(x, 9, out=full)):
        with pytest.raises((AssertionError, AttributeError)):
            bad()
    with pytest.raises(m.MoeError):
        m.router(x, 8, n_group=7)


def test_agrees_with_route_prep():
    """Softmax scores renormalised, fp32 logits, no bias: moe_route_prep's case."""
    x = torch.from_numpy(logits(1000, 256, 4)).to(dev())
    r, old = m.router(x, 8), m.route_prep(x, 8)
    for a, b in zip((r.expert_ids, r.dst2src, r.route_rows, r.expert_offsets), (old[0], old[2], old[3], old[4])):
        assert torch.equal(a, b)
    torch.testing.assert_close(r.weights, old[1], rtol=1e-5, atol=0)


@pytest.mark.parametrize("T", [8, 300])
def test_captured(T):
    E, k = 128, 6
    x = torch.empty((T, E), dtype=torch.bfloat16, device=dev())
    bias = torch.linspace(-0.1, 0.1, E, device=dev())
    out = m.router(x.zero_(), k, want_scores=True)
    ws = torch.empty(max(1, m.router_workspace_size(T, E)), dtype=torch.uint8, device=dev())

    def fresh(i):
        v = torch.from_numpy(logits(T, E, i)).to(torch.bfloat16)
        v[i::5] = -float("inf")
        x.copy_(v)
    for got, want in replayed(lambda: m.router(x, k, score=SIGMOID, bias=bias, n_group=4, topk_group=2, out=out, workspace=ws), None, list(out), fresh):
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_on_another_stream():
    x = torch.from_numpy(logits(500, 64, 2)).to(dev())
    want = m.router(x, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = m.router(x, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:5], want[:5]))
