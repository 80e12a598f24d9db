"""MxLinear's calls are its parts' calls, bit for bit, at each kernel of the product."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F

from .gpu_common import DEV, dev, host, say

pytestmark = pytest.mark.gpu

E2M1, E4M3 = N.MOE_MX_E2M1, N.MOE_MX_E4M3


def _bf16(rng, dims, scale=1.0):
    return dev(F.f32_to_bf16((rng.standard_normal(dims) * scale).astype(np.float32)))


@pytest.mark.parametrize("a_fmt,w_fmt,f32", [(E4M3, E2M1, False), (E4M3, E4M3, False), (E2M1, E2M1, False), (E2M1, E2M1, True)])
@pytest.mark.parametrize("Nn,K", [(264, 1056), (4160, 512)])
def test_calls_are_their_parts(Nn, K, a_fmt, w_fmt, f32):
    rng = np.random.default_rng(Nn)
    wb, gain = _bf16(rng, (Nn, K), K ** -0.5), _bf16(rng, K, 0.1)
    lin = LY.MxLinear(wb, 2600, w_fmt=w_fmt, a_fmt=a_fmt)
    width = {E2M1: 2, E4M3: 1}
    wc, wsf = (torch.empty(s, dtype=torch.uint8, device=DEV) for s in ((Nn, K // width[w_fmt]), (Nn, K // 32)))
    N.mx_quant(wb, w_fmt, wc, wsf)
    for T in (1, 20, 33, 700, 2600):
        say(f"MxLinear T={T} N={Nn} K={K} {a_fmt} {w_fmt} f32={f32}")
        x, res = _bf16(rng, (T, K)), _bf16(rng, (T, K), 3.0)
        c, s = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in ((T, K // width[a_fmt]), (T, K // 32)))
        got, want = (torch.full((T, Nn), 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV) for _ in range(2))
        lin(x, got)
        N.mx_quant(x, a_fmt, c, s)
        N.mx_gemm(c, s, a_fmt, wc, wsf, w_fmt, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and float(want.float().abs().max()) < 100
        h = torch.empty_like(x)
        sums = torch.empty_like(x)
        lin.after_norm(x, res, gain, 1.0, 1e-6, h, got)
        N.mx_add_norm_quant(x, res, gain, 1.0, 1e-6, a_fmt, sums, c, s)
        N.mx_gemm(c, s, a_fmt, wc, wsf, w_fmt, want)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and np.array_equal(host(h), host(sums))
