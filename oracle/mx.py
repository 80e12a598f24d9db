"""MX blocks (OCP microscaling): quantizer, inverse, the residual norm whose
output is MX, and the dense product. Test infrastructure (see
``oracle/__init__``).

A block is 32 consecutive elements of a row under one e8m0 byte b of value
2^(b - 127); elements are e2m1 or e4m3. The pages name no MX format; the rules
are those of the OCP specification with its recommended scale:
  * b = floor(log2 m) + 127 - emax of the block's largest magnitude m, emax the
    exponent of the format's largest binade (2 for e2m1, 8 for e4m3), clamped at
    0 from below; 0 for m = 0;
  * codes are v / 2^(b - 127) to nearest even, saturating, the sign bit v's;
  * a block that holds a NaN or an infinity: b = 255, codes 0.
v / 2^(b - 127) is formed in fp64, where it is exact for every fp32 v but for
underflow far below the smallest code, so a code is one rounding of v.
"""
from __future__ import annotations

import numpy as np

from .formats import (E2M1, E4M3, bf16_to_f64, encode_e2m1, encode_e4m3, f64_to_bf16, pack_nibbles,
                      unpack_nibbles)
from .norm_quant import gamma

BLOCK = 32
EMAX = {"e2m1": 2, "e4m3": 8}


def quantize_mx(x: np.ndarray, fmt: str) -> tuple[np.ndarray, np.ndarray]:
    """fp32 values [T, H] -> (codes uint8 [T, H/2] or [T, H], scale bytes uint8 [T, H/32])."""
    x = np.asarray(x, dtype=np.float32)
    T, H = x.shape
    v = x.reshape(T, H // BLOCK, BLOCK).astype(np.float64)
    bad = ~np.isfinite(v).all(axis=-1)
    m = np.where(bad, 0.0, np.abs(np.where(np.isfinite(v), v, 0.0)).max(axis=-1))
    _, e = np.frexp(m)                                  # m = f * 2^e, 0.5 <= f < 1
    b = np.where(m == 0, 0, np.maximum(0, e - 1 + 127 - EMAX[fmt]))
    q = np.ldexp(np.where(bad[..., None], 0.0, v), (127 - b)[..., None])
    # q holds v's significand: fp32 loses nothing but what underflows below 2^-149
    q = q.astype(np.float32).reshape(T, H)
    codes = pack_nibbles(encode_e2m1(q)) if fmt == "e2m1" else encode_e4m3(q)
    return codes, np.where(bad, 255, b).astype(np.uint8)


def dequantize_mx(codes: np.ndarray, sf: np.ndarray, fmt: str) -> np.ndarray:
    """Codes and scale bytes -> fp64 values [T, H]."""
    c = E2M1[unpack_nibbles(codes).astype(np.int64)] if fmt == "e2m1" else E4M3[np.asarray(codes, dtype=np.int64)]
    s = np.asarray(sf, dtype=np.int64)
    scale = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return c * np.repeat(scale, BLOCK, axis=1)


def add_norm_mx(x_bf16, residual_bf16, norm_weight_bf16, gain_center: float, eps: float, fmt: str):
    """bf16 bits [T, H] -> (sum bf16 bits, codes, scale bytes): the sum rounded
    to bf16 from its fp32 rounding, then the norm of those values step by step
    in fp32 (the mean square from an exact fp64 sum), then quantize_mx. Where the
    mean square passes fp32's range, r and h * r are formed in fp64; r is NaN for
    a row that holds an infinity."""
    x = bf16_to_f64(x_bf16)
    if residual_bf16 is not None:
        with np.errstate(over="ignore", invalid="ignore"):
            x = (x.astype(np.float32) + bf16_to_f64(residual_bf16).astype(np.float32)).astype(np.float64)
    h = f64_to_bf16(x)
    v = bf16_to_f64(h).astype(np.float32)
    T, H = v.shape
    with np.errstate(all="ignore"):
        s = (v.astype(np.float64) ** 2).sum(axis=1, dtype=np.longdouble).astype(np.float64)
        ms = (s / H).astype(np.float32)
        r = (np.float32(1.0) / np.sqrt(ms + np.float32(eps)).astype(np.float32)).astype(np.float32)
        rd = np.where(np.isinf(s), np.nan, 1.0 / np.sqrt(s / H + np.float64(np.float32(eps))))
        n = np.where(np.isinf(ms)[:, None], (v.astype(np.float64) * rd[:, None]).astype(np.float32), v * r[:, None])
        y = n * gamma(norm_weight_bf16, gain_center, H)[None, :]
    codes, sf = quantize_mx(y.astype(np.float32), fmt)
    return h, codes, sf


def gemm(a: np.ndarray, w: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """fp64 values [T, K] and [N, K] -> (products [T, N] in fp64, the sums of
    the products' magnitudes: the scale of a summation's error)."""
    return a @ w.T, np.abs(a) @ np.abs(w).T
