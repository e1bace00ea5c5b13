"""The router's workspace sizes: more tokens, or more experts, never need less."""
import ctypes

import pytest

import moe_routed_expert_amd as m

P = ctypes.c_void_p
FAKE = P(0x1000)       # never dereferenced: every call below fails validation


@pytest.mark.parametrize("E", [1, 8, 64, 65, 256, 1000, 1024])
def test_never_less_for_more_tokens(E):
    at = sorted({t + d for t in [1 << s for s in range(28)] + [12288, 24576, 100000] for d in (-1, 0, 1) if 0 <= t + d <= 1 << 27})
    sizes = [m.router_workspace_size(T, E) for T in at]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), list(zip(at, sizes))


def test_never_less_for_more_experts():
    for T in (33, 65, 8192, 8193, 16384, 32769):
        sizes = [m.router_workspace_size(T, E) for E in range(1, 1025)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), T


@pytest.mark.parametrize("T,need", [(8192, 512 * 64), (8193, 129 * 64), (32769, 513 * 64 + 514 * 64 * 4)])
def test_less_than_this_call_needs_is_refused(T, need):
    """A byte of counts for each of a chunk's 64 experts, chunks of 16 tokens up to 8192, of 64 beyond; past 512 chunks their sums."""
    def call(ws_bytes, ws=FAKE):
        return m.lib().moe_router(FAKE, 1, 64, T, 64, 8, 1, None, 1, 1, 1, 1, 1.0, FAKE, FAKE, None, FAKE, FAKE, FAKE, ws, ws_bytes, None)
    assert m.router_workspace_size(T, 64) >= need and call(need - 256) == m.MOE_ERR_WORKSPACE and call(0) == m.MOE_ERR_WORKSPACE
    assert call(1 << 30, P(0x1008)) == m.MOE_ERR_ALIGN
