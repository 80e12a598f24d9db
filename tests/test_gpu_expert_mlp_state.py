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
