"""The weight a projection is made of may be dropped right after the constructor."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from oracle import formats as F
from oracle import mx as M

from .gpu_common import DEV, dev, host, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True])
def test_weight_dropped_while_another_stream_quantizes_it(raw):
    """Its memory is not given to the current stream's next tensor before that
    stream has read it."""
    rng = np.random.default_rng(12)
    wb = F.f32_to_bf16((rng.standard_normal((2048, 4096)) / 64).astype(np.float32))
    w, side = dev(wb), torch.cuda.Stream()
    torch.cuda.synchronize()
    say("MxLinear on a busy stream")
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    lin = LY.MxLinear(w, 4, stream=side.cuda_stream if raw else side)
    del w
    taken = [torch.full((2048, 4096), 0x7F80, dtype=torch.int16, device=DEV) for _ in range(2)]
    torch.cuda.synchronize()
    codes, sf = M.quantize_mx(F.bf16_to_f64(wb).astype(np.float32), "e2m1")
    assert np.array_equal(host(lin.w_codes), codes) and np.array_equal(host(lin.w_sf), sf)
    assert all(int(t[0, 0]) == 0x7F80 for t in taken)
