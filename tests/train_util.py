"""Helpers of the training operators' GPU tests: bounds, guarded outputs, replayed graphs."""
import numpy as np
import torch

from gpu_util import dev

NAMES = {torch.bfloat16: "bf16", torch.float16: "fp16", torch.float32: "fp32"}
# half a step relative to a normal value, and half the spacing below the normal range
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}


def f64(t):
    return t.detach().cpu().double().numpy()


def sum_bound(terms, mag, dt):
    """|device - exact| of a sum of `terms` exact products held in fp32: every addition, in any order, rounding or
    truncating, loses at most 2^-23 of a partial sum of at most mag; then one rounding to dt."""
    s = (terms + 8) * 2.0 ** -23 * mag
    return lambda ref: s + HALF[dt] * (np.abs(ref) + s) + TINY[dt]


def check(got, ref, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.all(np.isfinite(got)), what + ": non-finite"
    err = np.abs(got - ref)
    bad = err > bound
    assert not bad.any(), "%s: %d of %d beyond the bound, worst %.3e at %s (ref %.6e, bound %.3e)" % (
        what, bad.sum(), bad.size, err[bad].max(), np.argwhere(bad)[0], ref[bad][0], np.broadcast_to(bound, ref.shape)[bad][0])


class Guarded:
    """A [rows, cols] view in the middle of a larger buffer of a known pattern; intact() says that nothing
    outside the view changed."""

    def __init__(self, shape, dt, pad=8, row_pad=3, fill=7.0):
        *lead, rows, cols = shape
        self.lead = int(np.prod(lead)) if lead else 1
        self.buf = torch.full((self.lead * rows + 2 * row_pad, cols + 2 * pad), fill, dtype=dt, device=dev())
        v = self.buf[row_pad:row_pad + self.lead * rows, pad:pad + cols]
        self.view = v.unflatten(0, (*lead, rows)) if lead else v
        self.fill, self.mask = fill, torch.ones_like(self.buf, dtype=torch.bool)
        self.mask[row_pad:row_pad + self.lead * rows, pad:pad + cols] = False

    def intact(self):
        return bool((self.buf[self.mask] == self.fill).all())


def replayed(call, state, outputs, fresh):
    """Captures call() into a graph and replays it on three sets of inputs (fresh(i) fills the captured inputs in
    place), eager work and synchronizations between; returns the replays' and the eager outputs."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    pairs = []
    for i in range(3):
        fresh(i)
        for o in outputs:
            o.fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outputs]
        junk = torch.randn(1 << 16, device=dev()).sum()          # eager work between the replays
        for o in outputs:
            o.fill_(5)
        call()
        torch.cuda.synchronize()
        pairs.append((got, [o.clone() for o in outputs]))
    return pairs


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def randn(shape, dt, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt)
