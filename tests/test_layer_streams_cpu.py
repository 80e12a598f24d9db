"""The stream that an object of the layer module is made on: everything it allocates or
fills belongs to that stream."""
import contextlib

import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY

MADE = {"Routing": lambda stream: LY.Routing(5, 2, 4, 16, "cpu", stream),
        "ExpertMlp": lambda stream: LY.ExpertMlp(5, 2, 4, 64, 24, 16, "cpu", stream),
        "Buffers": lambda stream: LY.Buffers(LY.LayerShape(5, 64, 64, 4, 2, 16), "cpu", stream),
        "Buffers of no rows": lambda stream: LY.Buffers(LY.LayerShape(0, 64, 64, 4, 2, 16), "cpu", stream)}


@pytest.mark.parametrize("kind", MADE)
def test_buffers_are_made_on_the_stream_given(kind, monkeypatch):
    given, entered, outside = object(), [], []

    @contextlib.contextmanager
    def owner(stream):
        entered.append(stream)
        yield
        entered.append(None)

    def watched(make):
        def call(*args, **kw):
            if not entered or entered[-1] is not given:
                outside.append(make.__name__)
            return make(*args, **kw)
        return call

    monkeypatch.setattr(LY, "_owner", owner)
    for name in ("empty", "full", "zeros", "ones"):
        monkeypatch.setattr(torch, name, watched(getattr(torch, name)))
    MADE[kind](given)
    assert entered == [given, None] and not outside
