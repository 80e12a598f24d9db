"""Which backward layer.ExpertMlp accepts, with the library's calls replaced by a record
of their names."""
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N

CALLS = ("moe_route", "moe_dispatch", "moe_dispatch_bwd", "moe_combine", "moe_combine_bwd", "moe_grouped_gemm",
         "moe_grouped_gemm_dgrad", "moe_grouped_gemm_wgrad", "moe_swiglu", "moe_swiglu_bwd")


class Program:
    """A layer whose calls only record themselves; the call number `fails` raises."""

    def __init__(self, monkeypatch):
        self.calls, self.fails = [], None
        self.routing, self.mlp = LY.Routing(5, 2, 4, 16, "cpu"), LY.ExpertMlp(5, 2, 4, 64, 24, 16, "cpu")
        for name in CALLS:
            monkeypatch.setattr(N, name, lambda *args, name=name: self._call(name))

    def _call(self, name):
        if len(self.calls) == self.fails:
            raise ValueError(f"{name}: refused")
        self.calls.append(name)

    def route(self):
        self.routing(torch.zeros(5, 4))

    def forward(self):
        self.mlp.forward(None, self.routing, None, None, None)

    def backward(self, routing=None):
        self.mlp.backward(None, routing or self.routing, None, None, None, None, None, None)


def test_a_backward_of_each_forward(monkeypatch):
    p = Program(monkeypatch)
    for _ in range(2):
        p.route()
        p.forward()
        p.backward()
    assert len(p.calls) == 2 * (1 + 5 + 7)
    with pytest.raises(ValueError, match="without its forward"):
        p.backward()


@pytest.mark.parametrize("done", range(5))
def test_a_forward_that_raises_leaves_nothing_to_go_back_from(done, monkeypatch):
    """Whatever it wrote before, the forward in front of it is gone too."""
    p = Program(monkeypatch)
    p.route()
    p.forward()
    p.fails = len(p.calls) + done
    with pytest.raises(ValueError, match="refused"):
        p.forward()
    p.fails, before = None, len(p.calls)
    with pytest.raises(ValueError, match="without its forward"):
        p.backward()
    assert len(p.calls) == before
    p.forward()
    p.backward()


def test_a_routing_that_ran_again_is_refused(monkeypatch):
    """Its maps are no longer those of the rows that the forward kept; with a new forward
    they are."""
    p = Program(monkeypatch)
    p.route()
    p.forward()
    p.route()
    before = len(p.calls)
    with pytest.raises(ValueError, match="ran again"):
        p.backward()
    assert len(p.calls) == before
    p.forward()
    p.backward()


def test_a_routing_that_was_refused_midway_is_refused(monkeypatch):
    p = Program(monkeypatch)
    p.route()
    p.forward()
    p.fails = len(p.calls)
    with pytest.raises(ValueError, match="refused"):
        p.route()
    p.fails = None
    with pytest.raises(ValueError, match="ran again"):
        p.backward()


def test_another_routing_is_refused(monkeypatch):
    """And the forward's own is taken after that."""
    p = Program(monkeypatch)
    other = LY.Routing(5, 2, 4, 16, "cpu")
    p.route()
    other(torch.zeros(5, 4))
    p.forward()
    before = len(p.calls)
    with pytest.raises(ValueError, match="forward's"):
        p.backward(other)
    assert len(p.calls) == before
    p.backward()
