"""Sizes past the library's 32-bit ones: ctypes would pass their low half, and a
call would quietly do the wrong part of the work (meta tensors: no memory)."""
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N

BF, U8, I32, F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
BIG = (1 << 32) + 32


def _t(rows, cols, dtype=BF):
    return torch.empty((rows, cols), dtype=dtype, device="meta")


def _v(n, dtype=I32):
    return torch.empty((n,), dtype=dtype, device="meta")


CALLS = {
    "mx_quant rows": lambda: N.mx_quant(_t(BIG, 32), N.MOE_MX_E4M3, _t(BIG, 32, U8), _t(BIG, 1, U8)),
    "mx_quant row": lambda: N.mx_quant(_t(1, BIG), N.MOE_MX_E2M1, _t(1, BIG // 2, U8), _t(1, BIG // 32, U8)),
    "mx_dequant": lambda: N.mx_dequant(_t(1, BIG, U8), _t(1, BIG // 32, U8), N.MOE_MX_E4M3, _t(1, BIG)),
    "mx_add_norm_quant": lambda: N.mx_add_norm_quant(_t(BIG, 32), None, None, 0.0, 1e-6, N.MOE_MX_E4M3, None,
                                                     _t(BIG, 32, U8), _t(BIG, 1, U8)),
    "mx_gemm tokens": lambda: N.mx_gemm(_t(BIG, 32, U8), _t(BIG, 1, U8), N.MOE_MX_E4M3, _t(4, 16, U8), _t(4, 1, U8),
                                        N.MOE_MX_E2M1, _t(BIG, 4)),
    "mx_gemm K": lambda: N.mx_gemm(_t(4, BIG, U8), _t(4, BIG // 32, U8), N.MOE_MX_E4M3, _t(4, BIG // 2, U8),
                                   _t(4, BIG // 32, U8), N.MOE_MX_E2M1, _t(4, 4)),
    "mx_gemm_validate": lambda: N.mx_gemm_validate(N.MOE_MX_E4M3, N.MOE_MX_E2M1, 4, BIG),
    "moe_dispatch": lambda: N.moe_dispatch(_t(BIG, 16, U8), _t(BIG, 1, I32), _v(64), _v(1), _t(64, 16, U8)),
    "moe_dispatch_bwd": lambda: N.moe_dispatch_bwd(_t(64, 8), _t(BIG, 1, I32), _t(BIG, 8)),
    "moe_combine": lambda: N.moe_combine(_t(64, 8), _t(4, BIG, I32), _t(4, BIG, F32), _t(4, 8)),
    "moe_combine_bwd": lambda: N.moe_combine_bwd(_t(BIG, 8), _t(64, 8), _t(BIG, 1, I32), _v(64), _v(1), _t(BIG, 1, F32),
                                                 _t(64, 8), _t(BIG, 1, F32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_sizes_past_32_bits_are_refused(name):
    with pytest.raises(N.MoeError, match="too large"):
        CALLS[name]()
