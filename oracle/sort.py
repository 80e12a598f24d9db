"""Token rows by expert and back, and the gradients. Test infrastructure (see
``oracle/__init__``). Plain loops over the routes in fp64; the maps are those of
``oracle/permute``."""
from __future__ import annotations

import numpy as np


def dispatch(x: np.ndarray, exp2perm: np.ndarray, total_rows: int, rows: np.ndarray) -> np.ndarray:
    """rows (its present contents) -> rows after the sort: zeros below
    total_rows, then every route's token row; the rest stays."""
    out = rows.copy()
    out[:total_rows] = 0
    for t, k in np.argwhere(exp2perm >= 0):
        out[exp2perm[t, k]] = x[t]
    return out


def combine(rows: np.ndarray, exp2perm: np.ndarray, weights: np.ndarray) -> np.ndarray:
    """fp64 rows [R, H] -> out [T, H] = sum_k w[t, k] rows[exp2perm[t, k]]."""
    out = np.zeros((exp2perm.shape[0], rows.shape[1]), dtype=np.float64)
    for t, k in np.argwhere(exp2perm >= 0):
        out[t] += weights[t, k] * rows[exp2perm[t, k]]
    return out


def dispatch_bwd(d_rows: np.ndarray, exp2perm: np.ndarray) -> np.ndarray:
    return combine(d_rows, exp2perm, np.ones(exp2perm.shape))


def combine_bwd(d_out: np.ndarray, rows: np.ndarray, exp2perm: np.ndarray, total_rows: int, weights: np.ndarray,
                d_rows: np.ndarray) -> tuple[np.ndarray, np.ndarray]:
    """-> (d_rows after the call, from its present contents; d_weights)."""
    dr, dw = d_rows.copy(), np.zeros(exp2perm.shape, dtype=np.float64)
    dr[:total_rows] = 0
    for t, k in np.argwhere(exp2perm >= 0):
        p = exp2perm[t, k]
        dr[p] = weights[t, k] * d_out[t]
        dw[t, k] = rows[p] @ d_out[t]
    return dr, dw
