"""CPU pins of oracle/training.py: every gradient formula against central differences of the forward definition,
the 8-bit rounding against torch's cast, and the step as a whole against torch's float64 autograd."""
import numpy as np
import pytest
import torch

from oracle import training as tr

STEP = 1e-5     # central differences: error of order STEP^2 * third derivative + 2^-53 / STEP, below 1e-8 here


def differences(f, x):
    """Gradient of scalar f by central differences at every element of x."""
    g = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + STEP
        hi = f()
        x[i] = keep - STEP
        lo = f()
        x[i] = keep
        g[i] = (hi - lo) / (2 * STEP)
    return g


@pytest.mark.parametrize("act", [1, 2, 3, 4, 5])
def test_activation_backward_against_differences(act):
    rng = np.random.default_rng(act)
    x = rng.standard_normal((3, 10)) * 2
    x[np.abs(x) < 0.01] = 0.5                       # ReLU's kink stays outside the differences' reach
    c = rng.standard_normal((3, 5))
    want = differences(lambda: float((c * tr.gated_act(act, x)).sum()), x)
    assert np.abs(tr.gated_act_backward(act, x, c) - want).max() < 1e-8


def test_products_backward_against_differences():
    rng = np.random.default_rng(0)
    offs = np.array([0, 2, 2, 5])
    a, w, c = rng.standard_normal((5, 4)), rng.standard_normal((3, 6, 4)), rng.standard_normal((5, 6))
    f = lambda: float((c * tr.grouped_gemm(a, w, offs)[0]).sum())
    assert np.abs(tr.grouped_gemm(c, w, offs, trans=True)[0] - differences(f, a)).max() < 1e-8
    assert np.abs(tr.grouped_wgrad(c, a, offs)[0] - differences(f, w)).max() < 1e-8


@pytest.mark.parametrize("mapped", [False, True])
def test_reduce_backward_against_differences(mapped):
    rng = np.random.default_rng(1)
    slots = np.array([[0, 2, -1], [1, 0, 2]])
    rows = np.array([3, 1, -5, 0, 4, 2]) if mapped else None
    y, w, c = rng.standard_normal((6, 4)), rng.standard_normal((2, 3)), rng.standard_normal((2, 4))
    f = lambda: float((c * tr.reduce(y, slots, w, rows)).sum())
    dy, dw, _ = tr.reduce_backward(c, y, slots, w, rows)
    assert np.abs(np.nan_to_num(dy) - differences(f, y)).max() < 1e-8
    assert np.abs(dw - differences(f, w)).max() < 1e-8


def test_router_backward_against_differences():
    rng = np.random.default_rng(2)
    logits, c = rng.standard_normal((3, 7)), rng.standard_normal((3, 2))
    ids = np.array([[4, 1], [0, 6], [3, 2]])
    f = lambda: float((c * tr.route_weights(logits, ids)).sum())
    got = tr.route_backward(ids, tr.route_weights(logits, ids), c, 7)
    assert np.abs(got - differences(f, logits)).max() < 1e-8


def test_saved_rows_against_torch_cast():
    rng = np.random.default_rng(3)
    v = (rng.standard_normal((40, 300)) * np.exp(rng.uniform(-6, 6, (40, 1)))).astype(np.float32)
    v[3] = 0
    v[4, :] = 0
    v[4, 7] = 448.0                                  # exactly at the border of two scales
    v[5, :] = 0
    v[5, 7] = np.nextafter(np.float32(448), np.float32(1000))
    q, s = tr.save8(v)
    assert s[4, 0] == 1.0 and s[5, 0] == 2.0 and np.all(s[3] == 0)
    m = np.where(s > 0, np.log2(np.where(s > 0, s, 1)), 0)
    assert np.all(m == np.rint(m))
    sc = np.repeat(np.where(s == 0, 1, s), 128, axis=1)[:, :300]
    t = torch.from_numpy((v / sc).astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q, t)
    assert np.all(np.abs(v) / sc <= 448)
    top = np.array([[np.abs(v[r, 128 * j:128 * (j + 1)]).max() for j in range(3)] for r in range(40)])
    assert np.all((top == 0) | (top / np.where(s == 0, 1, s) > 224))      # the smallest such power of two


def test_step_against_autograd():
    g = torch.Generator().manual_seed(5)
    T, E, k, H, I = 4, 3, 2, 6, 4
    logits = torch.randn((T, E), generator=g, dtype=torch.float64, requires_grad=True)
    x = torch.randn((T, H), generator=g, dtype=torch.float64, requires_grad=True)
    w13 = torch.randn((E, 2 * I, H), generator=g, dtype=torch.float64, requires_grad=True)
    w2 = torch.randn((E, H, I), generator=g, dtype=torch.float64, requires_grad=True)
    c = torch.randn((T, H), generator=g, dtype=torch.float64)
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, 1)
    out = torch.zeros((T, H), dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            c1 = w13[e] @ x[t]
            out[t] = out[t] + w[t, j] * (w2[e] @ (torch.nn.functional.silu(c1[:I]) * c1[I:]))
    (out * c).sum().backward()

    ids = ids.numpy()
    slots, wn = ids.astype(np.int32), w.detach().numpy()
    order = np.argsort(ids.reshape(-1), kind="stable")
    rows = np.empty(T * k, np.int64)
    rows[order] = np.arange(T * k)
    offs = np.concatenate([[0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))])
    xr = x.detach().numpy()[order // k]
    c1, _ = tr.grouped_gemm(xr, w13.detach().numpy(), offs)
    h = tr.gated_act(1, c1)
    y, _ = tr.grouped_gemm(h, w2.detach().numpy(), offs)
    assert np.allclose(tr.reduce(y, slots, wn, rows), out.detach().numpy())
    dy, dw, _ = tr.reduce_backward(c.numpy(), y, slots, wn, rows)
    dh, _ = tr.grouped_gemm(dy, w2.detach().numpy(), offs, trans=True)
    dc1 = tr.gated_act_backward(1, c1, dh)
    dxr, _ = tr.grouped_gemm(dc1, w13.detach().numpy(), offs, trans=True)
    dx = tr.reduce(dxr, slots, np.ones_like(wn), rows)
    assert np.allclose(dx, x.grad.numpy())
    assert np.allclose(tr.grouped_wgrad(dy, h, offs)[0], w2.grad.numpy())
    assert np.allclose(tr.grouped_wgrad(dc1, xr, offs)[0], w13.grad.numpy())
    assert np.allclose(tr.route_backward(ids, wn, dw, E), logits.grad.numpy())
