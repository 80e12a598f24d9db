"""The MX and sort calls on buffers whose offsets pass 32 bits (in elements or in
bytes): the rows at both ends and around 2^32 against the oracle."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F
from oracle import mx as M

from .gpu_common import DEV, dev, host, say
from .test_gpu_sort import Maps

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.empty_cache()


def _bf16(rng, dims, scale=1.0):
    return F.f32_to_bf16((rng.standard_normal(dims) * scale).astype(np.float32))


def _ends(T, at):
    """Rows at both ends and around row `at`."""
    return [0, 1, at - 1, at, at + 1, T - 2, T - 1]


def test_quantizer_and_its_inverse():
    H = 2048
    T = (1 << 32) // H + 5
    rows = _ends(T, (1 << 32) // H)
    xb = _bf16(np.random.default_rng(1), (len(rows), H))
    x = torch.zeros((T, H), dtype=torch.int16, device=DEV)
    x[rows] = dev(xb)
    c, s = torch.empty((T, H), dtype=torch.uint8, device=DEV), torch.empty((T, H // 32), dtype=torch.uint8, device=DEV)
    say(f"mx_quant T={T} H={H}")
    N.mx_quant(x, N.MOE_MX_E4M3, c, s)
    oc, os_ = M.quantize_mx(F.bf16_to_f64(xb).astype(np.float32), "e4m3")
    assert np.array_equal(host(c[rows]), oc) and np.array_equal(host(s[rows]), os_)
    x.fill_(1)
    N.mx_dequant(c, s, N.MOE_MX_E4M3, x)
    assert np.array_equal(host(x[rows]), F.f64_to_bf16(M.dequantize_mx(oc, os_, "e4m3")))
    assert int((x != 0).sum(dtype=torch.int64)) == int((M.dequantize_mx(oc, os_, "e4m3") != 0).sum() + ((oc == 0x80).sum()))


def test_residual_norm():
    H = 16384
    T = (1 << 32) // H + 3
    rows = _ends(T, (1 << 31) // H)
    rng = np.random.default_rng(2)
    xb, rb = _bf16(rng, (len(rows), H)), _bf16(rng, (len(rows), H), 4.0)
    x, r = (torch.zeros((T, H), dtype=torch.int16, device=DEV) for _ in range(2))
    x[rows], r[rows] = dev(xb), dev(rb)
    c, s = torch.empty((T, H // 2), dtype=torch.uint8, device=DEV), torch.empty((T, H // 32), dtype=torch.uint8, device=DEV)
    say(f"mx_add_norm_quant T={T} H={H}")
    N.mx_add_norm_quant(x, r, None, 0.0, 1e-6, N.MOE_MX_E2M1, r, c, s)
    oh, oc, os_ = M.add_norm_mx(xb, rb, None, 0.0, 1e-6, "e2m1")
    assert np.array_equal(host(r[rows]), oh) and np.array_equal(host(c[rows]), oc) and np.array_equal(host(s[rows]), os_)


def _operand(rng, rows, K, picked, fmt):
    """Zeros but for the picked rows; scales of 1."""
    width = K // 2 if fmt == "e2m1" else K
    codes = torch.zeros((rows, width), dtype=torch.uint8, device=DEV)
    sf = torch.full((rows, K // 32), 127, dtype=torch.uint8, device=DEV)
    c, s = M.quantize_mx(rng.standard_normal((len(picked), K)).astype(np.float32), fmt)
    codes[picked], sf[picked] = dev(c), dev(s)
    return codes, sf, M.dequantize_mx(c, s, fmt)


def _near(got, ref):
    # every value's rounding to bf16 is at most 2^-8 of it; 1e-4 for the sums (e4m3 products cut in the
    # matrix unit: 3.3e-5 measured at most, fp32 sums of 65664 products far below)
    assert np.linalg.norm(got - ref) <= (2.0 ** -8 + 1e-4) * np.linalg.norm(ref)


@pytest.mark.parametrize("T,Nn,K,af,wf", [(66000, 65600, 512, "e2m1", "e2m1"), (66000, 65600, 32, "e4m3", "e2m1"),
                                          (66000, 40, 65664, "e4m3", "e4m3"), (20, 66000, 65664, "e4m3", "e4m3")])
def test_product(T, Nn, K, af, wf):
    rng = np.random.default_rng(K)
    rows, cols = _ends(T, T * 2 // 3), _ends(Nn, Nn // 2)
    ac, asf, av = _operand(rng, T, K, rows, af)
    wc, wsf, wv = _operand(rng, Nn, K, cols, wf)
    out = torch.full((T, Nn), 3.0, dtype=torch.bfloat16, device=DEV)
    fmt = {"e2m1": N.MOE_MX_E2M1, "e4m3": N.MOE_MX_E4M3}
    say(f"mx_gemm T={T} N={Nn} K={K} {af} x {wf}")
    N.mx_gemm(ac, asf, fmt[af], wc, wsf, fmt[wf], out)
    torch.cuda.synchronize()
    _near(out[rows][:, cols].double().cpu().numpy(), av @ wv.T)
    out[rows] = out[rows].index_fill(1, torch.tensor(cols, device=DEV), 0.0)
    for part in out.split(8192):        # everything else is zero times something
        assert not bool(part.any())


def test_sort_and_gradients():
    T, K, H = 20000, 8, 16384
    m = Maps(T, K, 64, 128)
    rng = np.random.default_rng(5)
    toks = [0, 1, 7777, 13000, 13001, T - 1]
    x = torch.zeros((T, H), dtype=torch.bfloat16, device=DEV)
    xv = torch.from_numpy(rng.standard_normal((len(toks), H)).astype(np.float32)).bfloat16().to(DEV)
    x[toks] = xv
    rows = torch.empty((m.R, H), dtype=torch.bfloat16, device=DEV)
    say(f"sort T={T} K={K} R={m.R} H={H}")
    N.moe_dispatch(x, *m.dev, rows)
    p = torch.from_numpy(m.p[toks]).long().to(DEV)
    assert int(p.max()) * H * 2 > 1 << 32
    assert torch.equal(rows[p], xv[:, None].expand(-1, K, -1))
    w = torch.from_numpy(m.w).to(DEV)
    N.moe_combine(rows, m.dev[0], w, x)
    ref = w[toks].double().sum(1, keepdim=True) * xv.double()
    mags = w[toks].double().abs().sum(1, keepdim=True) * xv.double().abs()
    assert bool(((x[toks].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (K + 1) * 2.0 ** -24 * mags).all())
    x.zero_()
    x[toks] = xv
    d_w = torch.empty_like(w)
    N.moe_combine_bwd(x, rows, *m.dev, w, rows, d_w)        # in place of the rows
    ref = w[toks].double()[..., None] * xv.double()[:, None]
    assert bool(((rows[p].double() - ref).abs() <= (2.0 ** -8 + 2.0 ** -23) * ref.abs()).all())
    dot = xv.double().square().sum(1, keepdim=True)
    assert bool(((d_w[toks].double() - dot).abs() <= 56 * 2.0 ** -24 * dot).all())
    assert float(d_w.abs().sum(dtype=torch.float64)) <= float(d_w[toks].double().abs().sum()) * (1 + 1e-9)
