"""mx_add_norm_quant at the limits of fp32: against the definition, beside the
comparison with the oracle."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F
from oracle import mx as M

from .gpu_common import DEV, dev, host, say
from .mx_near import assert_codes_near, norm64

pytestmark = pytest.mark.gpu

FMT = {"e2m1": N.MOE_MX_E2M1, "e4m3": N.MOE_MX_E4M3}


def _norm(xb, rb, wb, center, eps, fmt):
    T, H = xb.shape
    c = torch.full((T, H // 2 if fmt == "e2m1" else H), 0xAB, dtype=torch.uint8, device=DEV)
    s = torch.full((T, H // 32), 0xCD, dtype=torch.uint8, device=DEV)
    out = torch.zeros((T, H), dtype=torch.int16, device=DEV)
    say(f"mx_add_norm_quant limits T={T} H={H} {fmt} residual={rb is not None} weight={wb is not None}")
    N.mx_add_norm_quant(dev(xb), None if rb is None else dev(rb), None if wb is None else dev(wb), center, eps, FMT[fmt],
                        out, c, s)
    torch.cuda.synchronize()
    h, codes, sf = host(out), host(c), host(s)
    oh, oc, os_ = M.add_norm_mx(xb, rb, wb, center, eps, fmt)
    assert np.array_equal(h, oh) and np.array_equal(sf, os_) and np.array_equal(codes, oc)
    return h, codes, sf


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("H", [32, 4096, 16384])
def test_finite_rows_of_any_size_are_normalized(H, fmt):
    rng = np.random.default_rng(H)
    sizes = np.array([1.0, 1e15, 1e18, 1.9e19, 3e19, 1e25, 8e37])[:, None]
    xb, rb = (F.f32_to_bf16((rng.standard_normal((7, H)) * sizes).clip(-1.5e38, 1.5e38).astype(np.float32)) for _ in range(2))
    wb = F.f32_to_bf16((rng.standard_normal(H) * 0.1).astype(np.float32))
    for r, w, center in ((None, None, 0.0), (rb, wb, 1.0)):
        h, codes, sf = _norm(xb, r, w, center, 1e-6, fmt)
        assert_codes_near(codes, sf, norm64(h, w, center, 1e-6), fmt)


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("H", [32, 128, 4096, 16384])
def test_a_row_with_an_infinity_or_a_nan_is_nan_in_every_block(H, fmt):
    """In x, in the residual, or made by their sum; the rows beside are not touched."""
    rng = np.random.default_rng(H)
    a, b = (rng.standard_normal((9, H)).astype(np.float32) for _ in range(2))
    a[1, 0], a[2, H - 1], b[3, H // 2], a[4, 7], b[5, 3] = np.inf, -np.inf, np.inf, np.nan, np.nan
    a[6, 9] = b[6, 9] = 3e38                        # their sum is infinite
    a[7, 1], b[7, 1] = np.inf, -np.inf              # theirs NaN
    wb = F.f32_to_bf16((rng.standard_normal(H) * 0.1).astype(np.float32))
    for w, center in ((None, 0.0), (wb, 1.0)):
        _, codes, sf = _norm(F.f32_to_bf16(a), F.f32_to_bf16(b), w, center, 1e-6, fmt)
        assert (sf[1:8] == 255).all() and not codes[1:8].any()
        assert (sf[[0, 8]] != 255).all()
    _, codes, sf = _norm(F.f32_to_bf16(a), None, wb, 1.0, 1e-6, fmt)
    assert (sf[[1, 2, 4, 7]] == 255).all() and (sf[[0, 3, 5, 6, 8]] != 255).all()
