"""A projection that has no product is refused when it is made, before anything
is allocated or quantized."""
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N


@pytest.mark.parametrize("kw", [dict(a_fmt=N.MOE_MX_E2M1, w_fmt=N.MOE_MX_E4M3), dict(a_fmt=2), dict(a_fmt=-1), dict(w_fmt=7)])
def test_formats_without_a_product(kw):
    with pytest.raises(N.MoeError, match="mx_gemm"):
        LY.MxLinear(torch.zeros((96, 64), dtype=torch.bfloat16), 8, **kw)


@pytest.mark.parametrize("K", [16, 40, (1 << 20) + 32])
def test_widths_without_a_product(K):
    with pytest.raises(N.MoeError, match="mx_gemm"):
        LY.MxLinear(torch.zeros((1, K), dtype=torch.bfloat16), 8)


@pytest.mark.parametrize("a,w", [(N.MOE_MX_E2M1, N.MOE_MX_E2M1), (N.MOE_MX_E4M3, N.MOE_MX_E2M1), (N.MOE_MX_E4M3, N.MOE_MX_E4M3)])
def test_products_that_there_are(a, w):
    N.mx_gemm_validate(a, w, 96, 64)
