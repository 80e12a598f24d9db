"""Pins of the MX oracle (oracle/mx.py) and of the sort's (oracle/sort.py):
exact rational brute force, torch's own casts, and invariants."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import mx as M
from oracle import sort as S
from oracle.norm_quant import normalize
from oracle.permute import permute


def _brute(block, fmt):
    """One block by exact rationals: the scale by search, every code by search of
    the whole value table."""
    vals = [Fraction(float(v)) for v in block]
    m = max(abs(v) for v in vals)
    e = -300
    if m:
        while Fraction(2) ** (e + 1) <= m:
            e += 1
    b = max(0, e + 127 - M.EMAX[fmt]) if m else 0
    table = F.E2M1[:8] if fmt == "e2m1" else F.E4M3[:127]
    grid = [Fraction(float(g)) for g in table]
    codes = []
    for v, f in zip(vals, block):
        q = abs(v) / Fraction(2) ** (b - 127)
        best = min(range(len(grid)), key=lambda i: (abs(grid[i] - q), i & 1))
        codes.append(best | ((8 if fmt == "e2m1" else 128) if np.signbit(f) else 0))
    return b, codes


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantize_is_the_definition(fmt):
    rng = np.random.default_rng(5)
    rows = [rng.standard_normal(64) * s for s in (1.0, 1e-30, 3e37, 1e-39)]
    rows += [np.zeros(64), np.where(np.arange(64) % 3, -0.0, 5.0), np.full(64, 6.0), np.full(64, 7.75),
             np.concatenate([np.full(32, 2.0 ** -149), np.full(32, 2.0 ** -126)]),
             rng.standard_normal(64) * np.logspace(-20, 20, 64)]
    x = np.array(rows).astype(np.float32)
    codes, sf = M.quantize_mx(x, fmt)
    for t in range(len(x)):
        for j in range(2):
            b, want = _brute(x[t, 32 * j:32 * j + 32], fmt)
            got = (F.unpack_nibbles(codes[t]) if fmt == "e2m1" else codes[t])[32 * j:32 * j + 32]
            assert sf[t, j] == b
            assert got.tolist() == want


def test_quantize_non_finite_blocks():
    x = np.ones((3, 96), np.float32)
    x[0, 40], x[1, 3], x[2, 95] = np.nan, np.inf, -np.inf
    for fmt in ("e2m1", "e4m3"):
        codes, sf = M.quantize_mx(x, fmt)
        assert (sf == 255).tolist() == [[False, True, False], [True, False, False], [False, False, True]]
        v = M.dequantize_mx(codes, sf, fmt).reshape(3, 3, 32)
        assert np.array_equal(np.isnan(v).all(-1), sf == 255) and (v[sf != 255] == 1.0).all()


def test_e4m3_codes_are_torchs():
    x = np.random.default_rng(1).standard_normal((16, 256)).astype(np.float32)
    codes, sf = M.quantize_mx(x, "e4m3")
    scaled = torch.from_numpy(x.reshape(16, 8, 32)) * torch.exp2(127.0 - torch.from_numpy(sf.astype(np.float32)))[..., None]
    want = scaled.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(16, 256)
    assert np.array_equal(codes, want)


@pytest.mark.parametrize("fmt,worst", [("e2m1", 2.0 / 8.0), ("e4m3", 64.0 / 512.0)])
def test_round_trip_error_is_bounded(fmt, worst):
    """Off by at most half a step of the code, or by the saturation of the
    largest values: (2^(emax+1) - max) / 2^(emax+1) of them."""
    x = np.random.default_rng(2).standard_normal((8, 512)).astype(np.float32)
    v = M.dequantize_mx(*M.quantize_mx(x, fmt), fmt)
    amax = np.abs(x.reshape(8, 16, 32)).max(-1, keepdims=True)
    assert (np.abs(v - x).reshape(8, 16, 32) <= worst * amax + 1e-12).all()


def test_add_norm_without_residual_is_the_norm_of_the_layer():
    xb = F.f32_to_bf16(np.random.default_rng(3).standard_normal((5, 320)).astype(np.float32) * 3)
    wb = F.f32_to_bf16(np.random.default_rng(4).uniform(-0.1, 0.1, 320).astype(np.float32))
    for fmt in ("e2m1", "e4m3"):
        h, codes, sf = M.add_norm_mx(xb, None, wb, 1.0, 1e-6, fmt)
        assert np.array_equal(h, xb)
        c2, s2 = M.quantize_mx(normalize(xb, wb, 1.0, 1e-6), fmt)
        assert np.array_equal(codes, c2) and np.array_equal(sf, s2)


def test_add_norm_sum_is_torchs():
    g = np.random.default_rng(6)
    a, b = (torch.from_numpy(g.standard_normal((4, 64)).astype(np.float32)).bfloat16() for _ in range(2))
    bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
    h, _, _ = M.add_norm_mx(bits(a), bits(b), None, 0.0, 1e-6, "e4m3")
    assert np.array_equal(h, bits((a.float() + b.float()).bfloat16()))


def test_sort_and_its_gradients_are_adjoint():
    """<dispatch(x), g> = <x, dispatch_bwd(g)>; combine is linear in rows and in
    weights with the gradients as its adjoints; both against central differences."""
    rng = np.random.default_rng(7)
    T, K, E, H = 9, 3, 5, 4
    ids = np.array([rng.permutation(E + 2)[:K] for _ in range(T)])
    maps = permute(ids, 1, E, 16)
    p, R, total = maps["exp2perm"], maps["rows_max"], maps["total_rows"]
    assert (p < 0).any()
    x, w = rng.standard_normal((T, H)), rng.random((T, K))
    g, d_out = rng.standard_normal((R, H)), rng.standard_normal((T, H))
    keep = rng.standard_normal((R, H))
    rows = S.dispatch(x, p, total, keep)
    assert np.array_equal(rows[total:], keep[total:])
    assert np.isclose((rows[:total] * g[:total]).sum(), (x * S.dispatch_bwd(g, p)).sum())
    dr, dw = S.combine_bwd(d_out, rows, p, total, w, keep)
    assert np.array_equal(dr[total:], keep[total:])
    loss = lambda r, v: (S.combine(r, p, v) * d_out).sum()  # noqa: E731
    for t, k in ((0, 0), (3, 2), (8, 1)):
        e = np.zeros_like(w)
        e[t, k] = 0.5
        assert np.isclose(loss(rows, w + e) - loss(rows, w - e), dw[t, k])
    for i in range(0, total, 3):
        e = np.zeros_like(rows)
        e[i, 1] = 0.5
        assert np.isclose(loss(rows + e, w) - loss(rows - e, w), dr[i, 1])
