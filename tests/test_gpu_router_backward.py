"""The router's gradient against its formula in float64 and against differences of the definition."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from test_gpu_router import DTS, SIGMOID, SOFTMAX, logits, scores64
from train_util import HALF, Guarded, replayed

pytestmark = pytest.mark.gpu


def reference(x, ids, w, dw, ds, score, renorm, scale):
    """The formula of the header, and what its terms add up to in magnitude."""
    s, x = scores64(x, score)
    T, E = x.shape
    dl, u, mag = np.zeros((T, E)), np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        on = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        n = w[t, on] / scale
        mean = (n * dw[t, on]).sum()
        for j, nj in zip(on, n):
            e = ids[t, j]
            if renorm:
                f = 1 - s[t, e] if score == SIGMOID else 1.0
                dl[t, e] += scale * nj * (dw[t, j] - mean) * f
                mag[t, e] += scale * nj * (abs(dw[t, j]) + (n * np.abs(dw[t, on])).sum()) * f
            else:
                u[t, e] += scale * dw[t, j]
    if ds is not None:
        u = u + ds
    live = x > -np.inf
    u = np.where(live, u, 0)
    if score == SIGMOID:
        add, size = u * s * (1 - s), np.abs(u) * s * (1 - s)
    else:
        add = s * (u - (s * u).sum(axis=1, keepdims=True))
        size = s * (np.abs(u) + (s * np.abs(u)).sum(axis=1, keepdims=True))
    return np.where(live, dl + add, 0), mag + size


# fp32: a score's exponential is within (4 + |d|) 2^-24, |d| <= 40 here, and sums of up to 1024 terms and products add 32
# roundings; every factor enters twice at most
REL = 2 * (44 + 32) * 2.0 ** -24


def case(T, E, k, seed, dt, score, renorm, scale, aux, masked=True):
    rng = np.random.default_rng(seed)
    x = torch.from_numpy(logits(T, E, seed)).to(DTS[dt])
    if masked:
        x[::5] = -float("inf")
        x[1::7, : E // 2] = float("nan")
    r = m.router(x.to(dev()), k, score=score, renorm=renorm, scale=scale, maps=False)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    ds = None if aux == "none" else rng.standard_normal((1 if aux == "row" else T, E)).astype(np.float32) * 0.1
    return x, r.expert_ids, r.weights, torch.from_numpy(dw).to(dev()), ds


def run(x, ids, w, dw, ds, score, renorm, scale, out=None):
    out = torch.full(x.shape, 7.0, dtype=x.dtype, device=dev()) if out is None else out
    m.router_backward(x.to(dev()), ids, w, dw, out, score=score, renorm=renorm, scale=scale,
                      dscores=None if ds is None else torch.from_numpy(ds).to(dev()).expand(x.shape[0], -1))
    torch.cuda.synchronize()
    return out


@pytest.mark.parametrize("dt", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("aux", ["none", "row", "full"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (13, 7, 7), (50, 100, 5), (9, 300, 8), (6, 1024, 64)])
def test_formula(dt, score, renorm, aux, T, E, k):
    x, ids, w, dw, ds = case(T, E, k, T + E, dt, score, renorm, 2.5, aux)
    got = run(x, ids, w, dw, ds, score, renorm, 2.5).cpu().double().numpy()
    ref, mag = reference(x.double().numpy(), ids.cpu().numpy(), w.cpu().double().numpy(), dw.cpu().double().numpy(), ds, score, renorm, 2.5)
    bound = REL * mag + HALF[DTS[dt]] * (np.abs(ref) + REL * mag) + (2.0 ** -25 if dt == "fp16" else 2.0 ** -120)
    assert np.isfinite(got).all() and (np.abs(got - ref) <= bound).all(), (np.abs(got - ref) / bound).max()
    hidden = ~(x.float().numpy() > -np.inf)
    assert (got[hidden] == 0).all()


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID])
@pytest.mark.parametrize("renorm", [True, False])
def test_differences(score, renorm):
    """Central differences of sum(w dw) + sum(s ds) in float64 with the chosen experts held: step 1e-4, error of the third
    derivative's term (below 1e-8 of the factors here) and of rounding (1e-16 / 1e-4)."""
    T, E, k, scale = 4, 12, 3, 1.5
    x, ids, w, dw, ds = case(T, E, k, 3, "fp32", score, renorm, scale, "full", masked=False)
    got = run(x, ids, w, dw, ds, score, renorm, scale).cpu().double().numpy()
    sel, g = ids.cpu().numpy(), dw.cpu().double().numpy()

    def loss(v):
        s = scores64(v, score)[0]
        c = np.take_along_axis(s, sel, 1)
        c = c / c.sum(axis=1, keepdims=True) if renorm else c
        return (scale * c * g).sum() + (s * ds.astype(np.float64)).sum()
    base, h = x.double().numpy(), 1e-4
    for t in range(T):
        for e in range(E):
            d = np.zeros_like(base)
            d[t, e] = h
            want = (loss(base + d) - loss(base - d)) / (2 * h)
            assert abs(got[t, e] - want) <= 1e-5, (t, e)


def test_ids_outside_are_left_out():
    x, ids, w, dw, _ = case(20, 16, 4, 1, "fp32", SIGMOID, True, 1.0, "none", masked=False)
    ids = ids.clone()
    ids[3, 1], ids[4, 0], ids[5] = -1, 16, -7
    for score in (SOFTMAX, SIGMOID):
        for renorm in (True, False):
            got = run(x, ids, w, dw, None, score, renorm, 1.0).cpu().double().numpy()
            ref, mag = reference(x.double().numpy(), ids.cpu().numpy(), w.cpu().double().numpy(), dw.cpu().double().numpy(), None, score, renorm, 1.0)
            assert (np.abs(got - ref) <= (REL + 2.0 ** -24) * mag + 2.0 ** -120).all()


def test_an_id_named_twice_counts_twice():
    for score in (SOFTMAX, SIGMOID):
        for renorm in (True, False):
            for aux in ("none", "full"):
                x, ids, w, dw, ds = case(20, 70, 4, 2, "fp32", score, renorm, 1.5, aux, masked=False)
                ids = ids.clone()
                ids[:, 2] = ids[:, 0]
                ids[7] = ids[7, 1]
                got = run(x, ids, w, dw, ds, score, renorm, 1.5).cpu().double().numpy()
                ref, mag = reference(x.double().numpy(), ids.cpu().numpy(), w.cpu().double().numpy(), dw.cpu().double().numpy(), ds, score, renorm, 1.5)
                assert (np.abs(got - ref) <= (REL + 2.0 ** -24) * mag + 2.0 ** -120).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_strides(dt):
    x, ids, w, dw, ds = case(11, 50, 4, 2, dt, SOFTMAX, False, 1.0, "full")
    want = run(x, ids, w, dw, ds, SOFTMAX, False, 1.0)
    wide = torch.full((11, 70), 5.0, dtype=DTS[dt], device=dev())
    wide[:, 9:59] = x.to(dev())
    g = Guarded((11, 50), DTS[dt], pad=5)
    m.router_backward(wide[:, 9:59], ids, w, dw, g.view, renorm=False, dscores=torch.from_numpy(ds).to(dev()))
    torch.cuda.synchronize()
    assert torch.equal(g.view, want) and g.intact()


def test_captured():
    x, ids, w, dw, ds = case(40, 64, 6, 5, "fp32", SOFTMAX, False, 1.0, "row", masked=False)
    x, d = x.to(dev()), torch.from_numpy(ds).to(dev())
    out = torch.empty_like(x)
    call = lambda: m.router_backward(x, ids, w, dw, out, renorm=False, dscores=d.expand(40, -1))  # noqa: E731
    for got, want in replayed(call, None, [out], lambda i: dw.copy_(torch.randn(40, 6, generator=torch.Generator().manual_seed(i)))):
        assert torch.equal(got[0], want[0])


def test_refusals():
    x, ids, w, dw, _ = case(4, 16, 2, 1, "fp32", SOFTMAX, True, 1.0, "none")
    out = torch.empty((4, 16), device=dev())
    x = x.to(dev())
    for bad in (lambda: m.router_backward(x, ids.long(), w, dw, out), lambda: m.router_backward(x, ids, w[:3], dw, out),
                lambda: m.router_backward(x, ids, w, dw.double(), out), lambda: m.router_backward(x, ids, w, dw, out.bfloat16()),
                lambda: m.router_backward(x, ids, w, dw, out[:, :15]), lambda: m.router_backward(x, ids, w, dw, out, dscores=x[:3])):
        with pytest.raises(AssertionError):
            bad()
    with pytest.raises(m.MoeError):
        m.router_backward(x, ids, w, dw, out, scale=0.0)
