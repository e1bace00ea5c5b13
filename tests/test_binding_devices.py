"""CPU-only checks of the training binding's rule on devices: tensors and stream of one GPU, refused before the library is
called otherwise."""
import types

import pytest

import moe_routed_expert_amd as m


def on(index):
    return types.SimpleNamespace(get_device=lambda: index)


def stream_of(index):
    return types.SimpleNamespace(device=types.SimpleNamespace(index=index), cuda_stream=0)


@pytest.mark.parametrize("tensors,stream", [((on(0), on(1)), None), ((on(-1),), None), ((on(0), on(-1)), None), ((on(0),), stream_of(1)),
                                            ((on(1), None, on(1)), stream_of(0))])
def test_devices_that_do_not_match(tensors, stream, monkeypatch):
    monkeypatch.setattr(m, "_entry", {"moe_none": lambda *a: pytest.fail("the library was called")})
    monkeypatch.setattr(m, "_current_device", lambda: 0)
    with pytest.raises(AssertionError):
        m._call("moe_none", tensors, (), stream)


def test_devices_that_match(monkeypatch):
    seen = []
    monkeypatch.setattr(m, "_entry", {"moe_none": lambda *a: seen.append(a) or m.MOE_OK})
    monkeypatch.setattr(m, "_current_device", lambda: 0)
    m._call("moe_none", (on(0), None, on(0)), (1, 2), stream_of(0))
    assert seen == [(1, 2, 0)]
