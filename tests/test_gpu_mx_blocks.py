"""The product's fp32 output from every size of block, and the same bits from
call to call for every kernel of the product."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import mx as M

from .gpu_common import DEV, dev, say
from .test_gpu_mx import FMT, FORMATS, _check_gemm, _gemm, _values

pytestmark = pytest.mark.gpu

# blocks of 64 x 64, 64 x 128, 128 x 128 and 256 x 256, ragged at both edges of the output
BLOCKS = [(130, 200), (1030, 2200), (1700, 3300), (2817, 3841)]


@pytest.mark.parametrize("T,Nn", BLOCKS)
@pytest.mark.parametrize("K", [640, 1152, 1056])
@pytest.mark.parametrize("pad", [0, 3])
def test_fp32_output(T, Nn, K, pad):
    """K with aligned scales (whole and cut chunks of them) and without; rows of
    the output that start at multiples of 16 bytes and that do not."""
    # stride Nn + pad: a multiple of 4 floats, or odd
    _check_gemm(T, Nn, K, "e2m1", "e2m1", True, pad + (-Nn) % 4)


@pytest.mark.parametrize("T,Nn", BLOCKS)
@pytest.mark.parametrize("K", [1024, 1056])
def test_fp32_output_of_whole_numbers(T, Nn, K):
    """Products of e2m1 values are whole quarters up to 36, their sums below 2^18:
    exact in fp32 in any order, so the output is."""
    rng = np.random.default_rng(T + K)
    ac, wc = (rng.integers(0, 256, (r, K // 2), dtype=np.uint8) for r in (T, Nn))
    asf, wsf = (np.full((r, K // 32), 127, np.uint8) for r in (T, Nn))
    got = _gemm(ac, asf, "e2m1", wc, wsf, "e2m1", True)
    ref, _ = M.gemm(M.dequantize_mx(ac, asf, "e2m1"), M.dequantize_mx(wc, wsf, "e2m1"))
    assert np.array_equal(got, ref)


@pytest.mark.parametrize("af,wf", FORMATS)
@pytest.mark.parametrize("T,Nn", [(5, 300), (31, 4500), *BLOCKS])
@pytest.mark.parametrize("K", [1056, 2048])
def test_the_same_bits_from_call_to_call(T, Nn, K, af, wf):
    """Every sum has one order; two streams at once too."""
    rng = np.random.default_rng(T + K)
    (ac, asf), (wc, wsf) = _values(rng, T, K, af), _values(rng, Nn, K, wf)
    args = [dev(ac), dev(asf), FMT[af], dev(wc), dev(wsf), FMT[wf]]
    say(f"mx_gemm repeated T={T} N={Nn} K={K} {af} x {wf}")
    outs = [torch.full((T, Nn), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(6)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i, out in enumerate(outs):
        N.mx_gemm(*args, out, stream=side if i % 3 == 2 else None)
    torch.cuda.synchronize()
    for out in outs[1:]:
        assert torch.equal(out.view(torch.int16), outs[0].view(torch.int16))
