"""layer.ExpertMlp after a forward that was refused midway."""
import pytest
import torch

from .test_gpu_expert_mlp import Step

pytestmark = pytest.mark.gpu


def test_no_backward_after_a_forward_that_raised():
    """The second forward is refused behind its first product; the third one's gradients
    are those of a layer that never saw it."""
    s = Step(40, 2, 4, 64, 40, 16, seed=31)
    s.forward()
    s.backward()
    want = s.results()
    s.forward()
    w2 = s.w2
    s.w2 = w2[:, :, :32].contiguous()
    with pytest.raises(ValueError):
        s.forward()
    s.w2 = w2
    with pytest.raises(ValueError, match="without its forward"):
        s.backward()
    s.forward()
    s.backward()
    for a, b in zip(s.results(), want):
        assert torch.equal(a, b)


def test_no_backward_on_other_maps():
    """A routing that ran again with other logits, and another one, are refused before
    anything is written; the step after that is that of a new layer."""
    s = Step(40, 2, 4, 64, 40, 16, seed=32)
    s.forward()
    s.backward()
    want, mine = s.results(), s.routing
    other = Step(40, 2, 4, 64, 40, 16, seed=33).routing
    s.forward()
    rows = s.mlp.out_rows.clone()
    s.routing = other
    with pytest.raises(ValueError, match="forward's"):
        s.backward()
    s.routing = mine
    s.routing(-s.logits, None, s.pad, 1.5)
    with pytest.raises(ValueError, match="ran again"):
        s.backward()
    torch.cuda.synchronize()
    assert torch.equal(rows.view(torch.int16), s.mlp.out_rows.view(torch.int16))
    s.forward()
    s.backward()
    for a, b in zip(s.results(), want):
        assert torch.equal(a, b)
