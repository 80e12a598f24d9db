"""Products grouped by expert with their gradients, and the gated activation with
its own, in fp64. Test infrastructure (see ``oracle/__init__``).

Expert e's rows are [offsets[e], offsets[e] + counts[e]); rows up to the next offset
are padding (zeros in outputs of rows), rows from the last offset on are left.
"""
from __future__ import annotations

import numpy as np


def _live(offsets, counts, e):
    return slice(int(offsets[e]), int(offsets[e]) + int(counts[e]))


def forward(x, w, offsets, counts, out):
    """out (fp64 [R, N], in place): w[e] x[r]; also returns the sums of magnitudes."""
    mags = np.zeros_like(out)
    for e in range(len(counts)):
        s = _live(offsets, counts, e)
        out[s.stop:int(offsets[e + 1])] = 0.0
        out[s] = x[s] @ w[e].T
        mags[s] = np.abs(x[s]) @ np.abs(w[e]).T
    return out, mags


def input_grad(d_out, w, offsets, counts, d_x):
    return forward(d_out, np.swapaxes(w, 1, 2), offsets, counts, d_x)


def weight_grad(d_out, x, offsets, counts, N, D):
    E = len(counts)
    d_w, mags = np.zeros((E, N, D)), np.zeros((E, N, D))
    for e in range(E):
        s = _live(offsets, counts, e)
        d_w[e] = d_out[s].T @ x[s]
        mags[e] = np.abs(d_out[s]).T @ np.abs(x[s])
    return d_w, mags


def sigmoid(g):
    t = np.exp(-np.abs(g))
    return np.where(g < 0, t, 1.0) / (1.0 + t)


def swiglu(gate_up):
    g, u = np.split(gate_up, 2, axis=1)
    return g * sigmoid(g) * u


def swiglu_grad(d, gate_up):
    """d_gate_up [R, 2 I], and the sum of magnitudes of the two terms of its gate half."""
    g, u = np.split(gate_up, 2, axis=1)
    s, rest = sigmoid(g), sigmoid(-g)
    return np.concatenate([d * u * (s + g * s * rest), d * g * s], axis=1)


def expert_mlp(x, ids, weights, w13, w2):
    """out [T, H] of the whole layer, fp64; ids [T, K] (-1: no route)."""
    out = np.zeros_like(x)
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = ids[t, k]
            if e >= 0:
                out[t] += weights[t, k] * (w2[e] @ swiglu((w13[e] @ x[t])[None])[0])
    return out


def expert_mlp_grads(x, ids, weights, w13, w2, d_out):
    d_x, d_w13, d_w2, d_weights = (np.zeros_like(v) for v in (x, w13, w2, weights))
    for t in range(x.shape[0]):
        for k in range(ids.shape[1]):
            e = ids[t, k]
            if e < 0:
                continue
            gate_up = w13[e] @ x[t]
            inter = swiglu(gate_up[None])[0]
            d_weights[t, k] = (w2[e] @ inter) @ d_out[t]
            d_row = weights[t, k] * d_out[t]
            d_w2[e] += np.outer(d_row, inter)
            d_gate_up = swiglu_grad((w2[e].T @ d_row)[None], gate_up[None])[0]
            d_w13[e] += np.outer(d_gate_up, x[t])
            d_x[t] += w13[e].T @ d_gate_up
    return d_x, d_w13, d_w2, d_weights
