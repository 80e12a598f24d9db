"""Codes and scales of a row that the quantizer got with a small error."""
import numpy as np

from oracle import formats as F
from oracle import mx as M

TOP = {"e2m1": 6.0, "e4m3": 448.0}


def norm64(h_bits, norm_weight_bits, gain_center, eps):
    """The RMSNorm of bf16 rows in extended precision."""
    h = F.bf16_to_f64(h_bits).astype(np.longdouble)
    w = 1.0 if norm_weight_bits is None else F.bf16_to_f64(norm_weight_bits)[None, :]
    r = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + np.longdouble(np.float32(eps)))
    return h * r * (w + np.longdouble(gain_center))


def assert_codes_near(codes, sf, y, fmt):
    """`codes` and `sf` are the MX block of values within 2^-22 of y (relative): three
    fp32 roundings, of h * r, of the gain and of their product, are 3 * 2^-24. The
    scale: of the exponent of a block's largest value so far off. A code: half its
    step from the scaled value, or the format's largest where that is larger."""
    y = np.asarray(y, dtype=np.float64)
    T, H = y.shape
    assert np.isfinite(y).all()
    off = 2.0 ** -22
    top = np.abs(y).reshape(T, H // 32, 32).max(-1)
    byte = [np.maximum(0, np.frexp(top * (1 + d))[1] - 1 + 127 - M.EMAX[fmt]) for d in (-off, off)]
    assert ((sf >= byte[0]) & (sf <= byte[1])).all()
    scale = np.repeat(np.ldexp(1.0, sf.astype(np.int64) - 127), 32, axis=1)
    q, got = np.abs(y) / scale, M.dequantize_mx(codes, sf, fmt) / scale
    expo = np.floor(np.log2(np.maximum(q * (1 + off), 2.0 ** -60)))
    step = np.exp2(np.maximum(expo - 1, -1)) if fmt == "e2m1" else np.exp2(np.maximum(expo - 3, -9))
    near = np.abs(got - y / scale) <= step / 2 + off * q
    near |= (np.abs(got) == TOP[fmt]) & (q >= TOP[fmt]) & (np.sign(got) == np.sign(y))
    assert near.all(), np.argwhere(~near)[:3]
