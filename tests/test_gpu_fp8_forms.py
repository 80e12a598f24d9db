"""fp8_gemm through each of its kernels, asserted to be the one it is about: strides, NaN,
the same bits from call to call, and more than 64 blocks of K, after which the weight's
scales are read again."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N

from . import kernel_choice as C
from .gpu_common import DEV, say
from .test_gpu_fp8 import _operands, _product

pytestmark = pytest.mark.gpu

FORMS = [  # kernel, T, N, K
    ("16 tokens", 9, 200, 528), ("16 tokens", 11, 300, 8336), ("32 tokens", 30, 300, 528), ("32 tokens", 17, 200, 8336),
    ("64 x 64", 70, 300, 528), ("64 x 64", 70, 300, 2048), ("64 x 64, two groups", 70, 300, 2064), ("64 x 64, two groups", 70, 300, 8336),
    ("64 x 128, two groups", 517, 2085, 528), ("64 x 128, two groups", 517, 2085, 8336), ("64 x 128", 1100, 3000, 528),
    ("64 x 128", 1100, 3000, 8336), ("128 x 128", 2000, 2100, 528), ("128 x 128", 2000, 2100, 8336), ("256 x 256", 2900, 2901, 528),
    ("256 x 256", 2900, 2901, 8336)]
CASES = pytest.mark.parametrize("form,T,Nn,K", FORMS)


@CASES
def test_strides(form, T, Nn, K):
    assert C.fp8_gemm(T, Nn, K) == form
    _product(T, Nn, K, w_pad=48, out_pad=3)
    if K < 8192:
        _product(T, Nn, K, w_pad=16, out_pad=8 + -Nn % 8)


@CASES
def test_nan_scales_and_codes(form, T, Nn, K):
    """In the first block of K, the last whole one and the last, which K ends in."""
    assert C.fp8_gemm(T, Nn, K) == form
    last = -(-K // 128) - 1
    _, (ac, asf, wc, wsf) = _operands(np.random.default_rng(T + K), T, Nn, K)
    asf[last - 1, 3], asf[last, T - 1], asf[0, 5] = (float("nan"),) * 3
    ac[7, K - 1] = 0x7F
    wc[150, 0] = 0xFF
    wsf[0, last] = float("nan")
    out = torch.empty((T, Nn), dtype=torch.bfloat16, device=DEV)
    say(f"fp8_gemm with NaN, {form}: T={T} N={Nn} K={K}")
    N.fp8_gemm(ac, asf, wc, wsf, out)
    torch.cuda.synchronize()
    bad = ~np.isfinite(out.float().cpu().numpy())
    want = np.zeros_like(bad)
    want[[3, 5, 7, T - 1]] = True
    want[:, 150] = want[:, :128] = True
    assert np.array_equal(bad, want)


@CASES
def test_same_bits_from_call_to_call(form, T, Nn, K):
    """Also into rows of another stride, and behind an output that was all NaN."""
    assert C.fp8_gemm(T, Nn, K) == form
    _, t = _operands(np.random.default_rng(T + K), T, Nn, K)
    outs = [torch.full((T, Nn + pad), float("nan"), dtype=torch.bfloat16, device=DEV)[:, :Nn] for pad in (0, 0, 0, 3, 16)]
    say(f"fp8_gemm again, {form}: T={T} N={Nn} K={K}")
    for o in outs:
        N.fp8_gemm(*t, o)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)
