"""e4m3 with one fp32 scale for a block of 128, and the product of such operands.
Test infrastructure (see ``oracle/__init__``).

A block is 128 consecutive elements of a row (activations) or 128 x 128 (weights),
less at the edges. Of its largest magnitude m (at least 2^-100) the scale is
fp32(m / 448) and a code the e4m3 value nearest to v * 448 / m, ties to the even
code; a block that holds a NaN or an infinity has scale NaN and codes 0.

The quotient is formed in fp64 and rounded to fp32 before the search of the grid:
v and m are bf16, so a quotient is a tie of the grid exactly or 2^-14 away from one.
"""
from __future__ import annotations

import numpy as np

from .formats import E4M3, encode_e4m3

BLOCK, LEAST = 128, 2.0 ** -100


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def _expand(sf: np.ndarray, tall: int, T: int, H: int) -> np.ndarray:
    """A scale for each element of [T, H], of blocks of `tall` x 128."""
    return np.repeat(np.repeat(sf, tall, axis=0)[:T], BLOCK, axis=1)[:, :H]


def quantize(x: np.ndarray, tall: int) -> tuple[np.ndarray, np.ndarray]:
    """fp64 values [T, H] (bf16 numbers) -> codes uint8 [T, H], scales fp32 [ceil(T/tall), ceil(H/128)]."""
    T, H = x.shape
    up, across = -(-T // tall), blocks(H)
    wide = np.zeros((up * tall, across * BLOCK))
    wide[:T, :H] = np.abs(x)
    m = wide.reshape(up, tall, across, BLOCK).max(axis=(1, 3))      # NaN wins over every number
    bad = ~np.isfinite(m)
    m = np.where(bad, 1.0, np.maximum(m, LEAST))
    sf = np.where(bad, np.nan, m).astype(np.float32) / np.float32(448.0)
    with np.errstate(invalid="ignore", over="ignore"):
        q = (x * 448.0 / _expand(m, tall, T, H)).astype(np.float32)
    return encode_e4m3(np.where(_expand(bad, tall, T, H), np.float32(0), q)), sf.astype(np.float32)


def values(codes: np.ndarray, sf: np.ndarray, tall: int) -> np.ndarray:
    """Codes [T, H] and scales [.., ceil(H/128)] -> fp64 values."""
    T, H = codes.shape
    return E4M3[codes.astype(np.int64)] * _expand(sf.astype(np.float64), tall, T, H)


def gemm(a: np.ndarray, w: np.ndarray) -> tuple[np.ndarray, np.ndarray, np.ndarray]:
    """fp64 values [T, K] and [N, K] -> (products [T, N], sums of the products'
    magnitudes, sums over groups of 8 along K of the products of the operands'
    largest magnitudes in the group)."""
    K = a.shape[1]
    g = [np.abs(v).reshape(len(v), K // 8, 8).max(-1) for v in (a, w)]
    return a @ w.T, np.abs(a) @ np.abs(w).T, g[0] @ g[1].T
