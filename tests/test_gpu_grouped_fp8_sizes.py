"""The products by expert and the 8-bit product at their largest rows, widths and strides:
offsets past 32 bits, the rows at both ends against the oracle."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F
from oracle import fp8 as Q

from .gpu_common import DEV, dev, host, say
from .test_gpu_fp8 import _bits, _bound as _fp8_bound
from .test_gpu_grouped import _bound, _near

pytestmark = pytest.mark.gpu

MOST = 0x7FFFF000


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.empty_cache()


def _f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("grad", [False, True])
def test_the_most_rows(grad):
    """One expert of all but the last 300 rows, one of 290 of those."""
    cols = 8
    x, out = torch.empty((MOST, cols), dtype=torch.bfloat16, device=DEV), torch.empty((MOST, cols), dtype=torch.bfloat16, device=DEV)
    rows = [0, 1, 255, 256, (1 << 28) + 1, 1 << 30, MOST - 301, MOST - 300, MOST - 11]
    xs = torch.randn(len(rows), cols, device=DEV).bfloat16()
    x[rows] = xs
    w = torch.randn(2, cols, cols, device=DEV).bfloat16()
    off, cnt = np.array([0, MOST - 300, MOST], np.int32), np.array([MOST - 300, 290], np.int32)
    say(f"grouped R={MOST} grad={grad}")
    (N.moe_grouped_gemm_dgrad if grad else N.moe_grouped_gemm)(x, w, dev(off), dev(cnt), out)
    torch.cuda.synchronize()
    wv, xv = _f64(w), _f64(xs)
    for i, r in enumerate(rows):
        e = int(r >= MOST - 300)
        m = wv[e] if grad else wv[e].T
        ref, mags = xv[i] @ m, np.abs(xv[i]) @ np.abs(m)
        _near(_f64(out[r]), ref, _bound(ref, mags, cols, "bf16"), f"row {r}")
    assert (out[MOST - 10:] == 0).all()


def test_the_widest_weights():
    wide, rows = 32768, 40
    w = torch.randn(1, 512, wide, device=DEV).bfloat16().repeat(3, wide // 512, 1)      # 6.4 GB, of equal bands
    x = torch.randn(rows, wide, device=DEV).bfloat16()
    off, cnt = dev(np.array([0, 7, 7, 40], np.int32)), dev(np.array([7, 0, 33], np.int32))
    out = torch.empty((rows, wide), device=DEV)
    say(f"grouped N=D={wide}")
    N.moe_grouped_gemm(x, w, off, cnt, out)
    torch.cuda.synchronize()
    ref, mags = _f64(x) @ _f64(w[0, :512]).T, np.abs(_f64(x)) @ np.abs(_f64(w[0, :512])).T
    tol = _bound(ref, mags, wide, "f32")
    for n in (0, 512, wide - 512):
        _near(_f64(out[:, n:n + 512]), ref, tol, f"columns from {n}")
    d_w = torch.zeros((3, wide, wide), dtype=torch.bfloat16, device=DEV)
    N.moe_grouped_gemm_wgrad(out.bfloat16(), x, off, cnt, d_w)
    torch.cuda.synchronize()
    assert (d_w[1] == 0).all()
    dv, xv = _f64(out.bfloat16())[7:, -256:], _f64(x)[7:]
    ref, mags = dv.T @ xv, np.abs(dv).T @ np.abs(xv)
    _near(_f64(d_w[2, -256:]), ref, _bound(ref, mags, 33, "bf16"), "d_w")


def test_the_longest_strides():
    rows, stride, D, Nn = 600, 1 << 21, 72, 4000
    x = torch.empty((rows, stride), dtype=torch.bfloat16, device=DEV)[:, :D]
    d = torch.empty((rows, stride), dtype=torch.bfloat16, device=DEV)[:, :Nn]
    x.copy_(torch.randn(rows, D, device=DEV)), d.copy_(torch.randn(rows, Nn, device=DEV))
    w = torch.randn(1, Nn, D, device=DEV).bfloat16()
    off, cnt = dev(np.array([0, rows], np.int32)), dev(np.array([rows - 3], np.int32))
    xv, dv, wv = _f64(x)[:rows - 3], _f64(d)[:rows - 3], _f64(w)[0]
    out, d_x, d_w = (torch.empty(s, device=DEV) for s in ((rows, Nn), (rows, D), (1, Nn, D)))
    say(f"grouped stride={stride}")
    N.moe_grouped_gemm(x, w, off, cnt, out)
    N.moe_grouped_gemm_dgrad(d, w, off, cnt, d_x)
    N.moe_grouped_gemm_wgrad(d, x, off, cnt, d_w)
    torch.cuda.synchronize()
    for got, a, b, K in ((out[:rows - 3], xv, wv.T, D), (d_x[:rows - 3], dv, wv, Nn), (d_w[0], dv.T, xv, rows)):
        ref, mags = a @ b, np.abs(a) @ np.abs(b)
        _near(_f64(got), ref, _bound(ref, mags, K, "f32"), K)


def _codes(rng, rows, K, tall):
    return Q.quantize(F.bf16_to_f64(_bits(rng, rows, K)), tall)


def test_the_most_tokens():
    K, Nn, rng = 16, 1, np.random.default_rng(0)
    rows = [0, 255, 256, 1 << 28, (1 << 30) + 5, MOST - 257, MOST - 1]
    ac, asf = _codes(rng, len(rows), K, 1)
    wc, wsf = _codes(rng, Nn, K, 128)
    a, sf = torch.empty((MOST, K), dtype=torch.uint8, device=DEV), torch.empty((1, MOST), device=DEV)
    a[rows], sf[0, rows] = dev(ac), dev(np.ascontiguousarray(asf[:, 0]))
    out = torch.empty((MOST, Nn), dtype=torch.bfloat16, device=DEV)
    say(f"fp8_gemm T={MOST}")
    N.fp8_gemm(a, sf, dev(wc), dev(wsf), out)
    torch.cuda.synchronize()
    av, wv = Q.values(ac, asf, 1), Q.values(wc, wsf, 128)
    ref, mags, tops = Q.gemm(av, wv)
    _near(_f64(out[rows]), ref, _fp8_bound(av, wv, ref, mags, tops, K), "rows")


@pytest.mark.parametrize("T", [5, 40, 700])
def test_the_longest_stride_of_weights(T):
    K, Nn, rng = 272, 1100, np.random.default_rng(T)
    ac, asf = _codes(rng, T, K, 1)
    wc, wsf = _codes(rng, Nn, K, 128)
    w = torch.empty((Nn, 1 << 22), dtype=torch.uint8, device=DEV)[:, :K]
    w.copy_(dev(wc))
    out = torch.empty((T, Nn), dtype=torch.int16, device=DEV)
    say(f"fp8_gemm T={T} stride={1 << 22}")
    N.fp8_gemm(dev(ac), dev(np.ascontiguousarray(asf.T)), w, dev(wsf), out)
    torch.cuda.synchronize()
    av, wv = Q.values(ac, asf, 1), Q.values(wc, wsf, 128)
    ref, mags, tops = Q.gemm(av, wv)
    _near(F.bf16_to_f64(host(out)), ref, _fp8_bound(av, wv, ref, mags, tops, K), "rows")
