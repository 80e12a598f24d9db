"""The MX oracle's residual norm at the limits of fp32, against the definition."""
import numpy as np
import pytest

from oracle import formats as F
from oracle import mx as M

from .mx_near import assert_codes_near, norm64


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("size", [1.0, 1e15, 1e18, 3e19, 1e25, 8e37])
def test_finite_rows_of_any_size_are_normalized(size, fmt):
    """Also where the mean square passes fp32's range (3.4e38: sizes above 1.8e19)."""
    rng = np.random.default_rng(3)
    xb = F.f32_to_bf16((rng.standard_normal((6, 256)) * size).clip(-3e38, 3e38).astype(np.float32))
    wb = F.f32_to_bf16((rng.standard_normal(256) * 0.1).astype(np.float32))
    for w, center in ((None, 0.0), (wb, 1.0)):
        h, codes, sf = M.add_norm_mx(xb, None, w, center, 1e-6, fmt)
        assert np.array_equal(h, xb)
        assert_codes_near(codes, sf, norm64(xb, w, center, 1e-6), fmt)


BAD = [(0, np.inf), (5, -np.inf), (100, np.nan), (255, np.inf)]


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_a_row_with_an_infinity_or_a_nan_is_nan_in_every_block(fmt):
    x = np.random.default_rng(4).standard_normal((6, 256)).astype(np.float32)
    for t, (j, v) in enumerate(BAD):
        x[t, j] = v
    _, codes, sf = M.add_norm_mx(F.f32_to_bf16(x), None, None, 0.0, 1e-6, fmt)
    assert (sf[:4] == 255).all() and not codes[:4].any()
    assert (sf[4:] != 255).all()
