"""The router and the MXFP4 experts as a layer uses them: a prefill step, a decode step, a training step's router."""
import numpy as np
import pytest
import torch

import moe_routed_expert_amd as m
from gpu_util import dev
from mx4_util import decode, quantise, to_gpu
from train_util import HALF, f64, replayed

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, T, E, k, H, I, seed=0):
        rng = np.random.default_rng(seed)
        self.T, self.E, self.k, self.H, self.I = T, E, k, H, I
        f32 = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.x = torch.from_numpy(f32(T, H)).to(torch.bfloat16).to(dev())
        self.gate = torch.from_numpy(f32(H, E) / H ** 0.5).to(dev())
        self.bias = torch.from_numpy(0.05 * f32(E)).to(dev())
        banks = []
        for n, w in ((H, 0.05 * f32(E * 2 * I, H)), (I, 0.05 * f32(E * H, I))):
            q, s = quantise(w.astype(np.float64))
            banks += [q.reshape(E, -1, n // 2), s.reshape(E, -1, n // 32)]
        self.w13, self.w2 = decode(*banks[:2]), decode(*banks[2:])
        self.g13, self.g2 = to_gpu(*banks[:2]), to_gpu(*banks[2:])
        u8 = lambda r, c: torch.empty((r, -(-c // 4) * 4), dtype=torch.uint8, device=dev())[:, :c]  # noqa: E731
        R = T * k
        self.xq, self.xs, self.hq, self.hs = u8(T, H // 2), u8(T, H // 32), u8(R, I // 2), u8(R, I // 32)
        self.y = torch.empty((R, H), dtype=torch.bfloat16, device=dev())
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=dev())
        self.logits = torch.empty((T, E), device=dev())
        self.live = torch.ones(T, dtype=torch.bool, device=dev())
        self.ws = torch.empty(max(1, m.router_workspace_size(T, E)), dtype=torch.uint8, device=dev())
        self.r = m.router(self.logits.zero_(), k)

    def route(self):
        torch.mm(self.x.float(), self.gate, out=self.logits)
        self.logits.masked_fill_(~self.live[:, None], -float("inf"))          # padding of the batch
        m.router(self.logits, self.k, score=m.MOE_SCORE_SIGMOID, bias=self.bias, n_group=4, topk_group=2, scale=2.5, out=self.r, workspace=self.ws)

    def prefill(self):
        self.route()
        m.mx4_quant(self.x, self.xq, self.xs)
        how = dict(mode=m.MOE_MODE_GROUPED, expert_offsets=self.r.expert_offsets)
        m.mx4_grouped_gemm_act_quant(self.xq, self.xs, *self.g13, self.hq, self.hs, a_rows=self.r.dst2src, **how)
        m.mx4_grouped_gemm(self.hq, self.hs, *self.g2, self.y, **how)
        m.topk_reduce(self.y, self.r.expert_ids, self.r.weights, self.out, route_rows=self.r.route_rows)

    def decode(self):
        self.route()
        m.mx4_quant(self.x, self.xq, self.xs)
        how = dict(mode=m.MOE_MODE_SLOT, slot_ids=self.r.expert_ids.view(-1))
        m.mx4_grouped_gemm_act_quant(self.xq, self.xs, *self.g13, self.hq, self.hs, a_row_div=self.k, **how)
        m.mx4_grouped_gemm(self.hq, self.hs, *self.g2, self.y, **how)
        m.topk_reduce(self.y, self.r.expert_ids, self.r.weights, self.out)

    def check(self, grouped):
        """Each step's result from the step before it as the device gave it, so no rounding to 4 bits is decided twice."""
        T, k, I = self.T, self.k, self.I
        q, s = quantise(self.x.double().cpu().numpy())
        assert np.array_equal(self.xq.cpu().numpy(), q) and np.array_equal(self.xs.cpu().numpy(), s)
        x = decode(q, s)
        ids, w = self.r.expert_ids.cpu().numpy(), self.r.weights.cpu().double().numpy()
        rows = self.r.route_rows.cpu().numpy().reshape(T, k) if grouped else np.arange(T * k).reshape(T, k)
        h = decode(self.hq.cpu().numpy(), self.hs.cpu().numpy())
        out, mag = np.zeros((T, self.H)), np.zeros((T, self.H))
        for t in range(T):
            for j in range(k):
                e, r = ids[t, j], rows[t, j]
                if e < 0:
                    continue
                c = self.w13[e] @ x[t]
                want = c[:I] / (1 + np.exp(-c[:I])) * c[I:]
                step = np.repeat(np.abs(h[r]).reshape(-1, 32).max(axis=1), 32) / 4 + 1e-6
                # the largest code is 4 or 6 scales, its half step one scale (saturation at 8 scales: two)
                assert (np.abs(h[r] - want) <= 2 * step).all()
                y = self.w2[e] @ h[r]
                out[t] += w[t, j] * y
                mag[t] += np.abs(w[t, j]) * (np.abs(self.w2[e]) @ np.abs(h[r]))
        got = f64(self.out)
        # y rounded to bf16, the weighted sum in fp32, rounded to bf16
        assert (np.abs(got - out) <= HALF[torch.bfloat16] * (mag + np.abs(out) * 1.01) + 2.0 ** -18 * mag).all()
        assert (got[(ids < 0).all(axis=1)] == 0).all()


@pytest.mark.parametrize("T,E,k,H,I", [(50, 16, 4, 256, 96), (90, 32, 6, 288, 160), (3, 8, 2, 128, 64)])
def test_prefill(T, E, k, H, I):
    L = Layer(T, E, k, H, I)
    L.live[1::4] = False
    L.prefill()
    torch.cuda.synchronize()
    L.check(True)


@pytest.mark.parametrize("T", [1, 5])
def test_decode(T):
    L = Layer(T, 16, 4, 512, 96)
    L.live[T // 2] = T == 1
    L.decode()
    torch.cuda.synchronize()
    L.check(False)


def test_prefill_and_decode_agree():
    """The two forms quantise the same rows and differ by the order of fp32 sums, which a 4-bit code may amplify; the steps
    before it are equal."""
    L = Layer(6, 8, 2, 256, 64)
    L.prefill()
    a, ids = L.out.clone(), L.r.expert_ids.clone()
    L.decode()
    assert torch.equal(ids, L.r.expert_ids)
    assert ((a.float() - L.out.float()).norm() <= 0.05 * a.float().norm()).item()


@pytest.mark.parametrize("form", ["prefill", "decode"])
def test_captured_step(form):
    L = Layer(70 if form == "prefill" else 4, 16, 4, 256, 64)

    def fresh(i):
        L.x.copy_(torch.randn(L.x.shape, generator=torch.Generator().manual_seed(i)).to(torch.bfloat16))
        L.live.copy_(torch.arange(L.T) % (i + 2) != 1)
    for got, want in replayed(getattr(L, form), None, [L.out], fresh):
        assert torch.equal(got[0], want[0])


def test_training_router_with_the_16_bit_experts():
    """logits -> router -> 16-bit experts -> reduce, and back to the logits, with padded tokens and an auxiliary loss on the mean
    scores: the gradient against differences of the same loss in float64 with the chosen experts held."""
    T, E, k, H, I, scale = 12, 8, 3, 32, 16, 1.5
    g = torch.Generator().manual_seed(2)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    logits = rand(T, E)
    logits[3] = -float("inf")
    logits[5, 2:] = -float("inf")
    x, w = rand(T, H).half(), (rand(E, I, H) * 0.2).half()
    dout, daux = rand(T, I).bfloat16(), rand(E) * 0.3
    d = lambda t: t.to(dev())  # noqa: E731
    for score in (0, 1):
        for renorm in (True, False):
            r = m.router(d(logits), k, score=score, renorm=renorm, scale=scale)
            rows = torch.empty((T * k, H), dtype=torch.float16, device=dev())
            src = r.dst2src.clamp(min=0).long()
            rows.copy_(d(x)[src])
            y = torch.zeros((T * k, I), device=dev())
            m.b16_grouped_gemm(rows, d(w), y, mode=m.MOE_MODE_GROUPED, expert_offsets=r.expert_offsets)
            out = torch.empty((T, I), dtype=torch.bfloat16, device=dev())
            m.topk_reduce(y, r.expert_ids, r.weights, out, route_rows=r.route_rows)
            assert (out[3] == 0).all()
            dy, dw = torch.zeros_like(y), torch.empty_like(r.weights)
            m.topk_reduce_backward(d(dout), y, r.expert_ids, r.weights, dy, dw, route_rows=r.route_rows)
            assert (dw[3] == 0).all() and (dw[5, 2:] == 0).all()
            dl = torch.empty((T, E), device=dev())
            m.router_backward(d(logits), r.expert_ids, r.weights, dw, dl, score=score, renorm=renorm, scale=scale,
                              dscores=d(daux).expand(T, E))
            ids = r.expert_ids.cpu().long()
            each = torch.einsum("th,eih->tei", x.double(), w.double())

            def loss(v):
                s = torch.sigmoid(v) if score else torch.softmax(v, 1).nan_to_num(0.0)
                c = torch.where(ids >= 0, s.gather(1, ids.clamp(min=0)), 0.0)
                c = c / c.sum(1, keepdim=True).clamp(min=1e-300) if renorm else c
                z = (scale * c[:, :, None] * each.gather(1, ids.clamp(min=0)[:, :, None].expand(-1, -1, I))).sum(1)
                return (z * dout.double()).sum() + (s * daux.double()).sum()
            base, h = logits.double(), 1e-5
            for t in range(T):
                for e in range(E):
                    if logits[t, e] == -float("inf"):
                        assert dl[t, e] == 0
                        continue
                    step = torch.zeros_like(base)
                    step[t, e] = h
                    want = (loss(base + step) - loss(base - step)) / (2 * h)
                    assert abs(dl[t, e].item() - want.item()) <= 2e-5 * (1 + abs(want.item())), (score, renorm, t, e)
