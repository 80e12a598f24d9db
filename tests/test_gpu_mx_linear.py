"""The dense projections around the expert layer as a model calls them: residual
norm and pooler in front of the layer, the layer, the unpooler behind it, each
against the CPU oracle on what the step before it gave."""
import dataclasses

import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N
from nvfp4_block_scaled_route_amd import workloads as W
from oracle import formats as F
from oracle import mx as M
from oracle.layer import layer as o_layer
from oracle.layer import rel_l2

from .gpu_common import DEV, dev, host, say, upload_weights

pytestmark = pytest.mark.gpu


def _bf16(rng, dims, scale=1.0):
    return F.f32_to_bf16((rng.standard_normal(dims) * scale).astype(np.float32))


def _product(codes, sf, a_fmt, wb, w_fmt):
    """The exact products, what bf16 makes of them, and the sums of magnitudes."""
    w = M.dequantize_mx(*M.quantize_mx(F.bf16_to_f64(wb).astype(np.float32), w_fmt), w_fmt)
    return M.gemm(M.dequantize_mx(codes, sf, a_fmt), w)


def _near(got_bits, ref, mags):
    # half a bf16 step; the sums: fp32, and e4m3 products cut at 2^-13 of the largest of 8, at most
    # 8 * 2^-13 of the magnitudes
    err = 2.0 ** -10 * mags
    assert (np.abs(F.bf16_to_f64(got_bits) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err)).all()


def test_pooler_layer_unpooler():
    wl = W.WORKLOADS["tiny"]
    inp = W.make_inputs(wl)
    D, rng = 512, np.random.default_rng(21)
    pool_w, unpool_w = _bf16(rng, (wl.H, D), D ** -0.5), _bf16(rng, (D, wl.H), wl.H ** -0.5)
    norm_w, xb, rb = _bf16(rng, D, 0.1), _bf16(rng, (wl.T, D)), _bf16(rng, (wl.T, D), 4.0)
    pooler = LY.MxLinear(dev(pool_w), 8)
    unpooler = LY.MxLinear(dev(unpool_w), 8, a_fmt=N.MOE_MX_E2M1)
    x, res = dev(xb), dev(rb)
    pooled = torch.empty((wl.T, wl.H), dtype=torch.int16, device=DEV)
    back = torch.empty((wl.T, D), dtype=torch.int16, device=DEV)
    bufs = LY.Buffers(LY.LayerShape(wl.T, wl.H, wl.I, wl.E, wl.K, wl.tile_m), DEV)
    say("pooler, layer, unpooler")
    pooler.after_norm(x, res, dev(norm_w), 1.0, 1e-6, res, pooled)
    LY.run_layer(bufs, pooled, dev(inp.a1_gscale), dev(inp.logits), None, None, upload_weights(inp),
                 dev(inp.norm_weight_bf16), wl.gain_center, wl.eps, bool(wl.weight_before_norm), check=True)
    unpooler(bufs.out, back)
    torch.cuda.synchronize()
    h, codes, sf = M.add_norm_mx(xb, rb, norm_w, 1.0, 1e-6, "e4m3")
    assert np.array_equal(host(res), h)
    _near(host(pooled), *_product(codes, sf, "e4m3", pool_w, "e2m1"))
    ref = o_layer(dataclasses.replace(inp, x_bf16=host(pooled)))
    assert np.array_equal(host(bufs.ids), ref["ids"])
    out = host(bufs.out)
    assert rel_l2(F.bf16_to_f64(out), F.bf16_to_f64(ref["out"])) < 1e-2
    _near(host(back), *_product(*M.quantize_mx(F.bf16_to_f64(out).astype(np.float32), "e2m1"), "e2m1", unpool_w, "e2m1"))


def test_token_counts_and_refusals():
    rng = np.random.default_rng(3)
    wb = _bf16(rng, (96, 64), 0.125)
    lin = LY.MxLinear(dev(wb), 40, w_fmt=N.MOE_MX_E4M3)
    for T in (0, 1, 33, 40):
        xb = _bf16(rng, (T, 64))
        out = torch.full((T, 96), 5, dtype=torch.int16, device=DEV)
        lin(dev(xb), out)
        torch.cuda.synchronize()
        if T:
            _near(host(out), *_product(*M.quantize_mx(F.bf16_to_f64(xb).astype(np.float32), "e4m3"), "e4m3", wb, "e4m3"))
    x, out = torch.zeros((41, 64), dtype=torch.int16, device=DEV), torch.zeros((41, 96), dtype=torch.int16, device=DEV)
    with pytest.raises(ValueError, match="tokens"):
        lin(x, out)
    with pytest.raises((ValueError, N.MoeError)):
        lin(x[:4, :32], out[:4])


@pytest.mark.parametrize("raw", [False, True])
def test_made_on_another_stream(raw):
    """Memory that the current stream freed with work still to come is not the weight's."""
    rng = np.random.default_rng(8)
    wb = _bf16(rng, (2048, 4096), 4096 ** -0.5)
    w, side = dev(wb), torch.cuda.Stream()
    torch.cuda.synchronize()
    late = torch.empty((2048, 2048), dtype=torch.uint8, device=DEV)      # the codes' size
    torch.cuda._sleep(20_000_000)
    late.fill_(0x77)
    del late
    lin = LY.MxLinear(w, 4, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    codes, sf = M.quantize_mx(F.bf16_to_f64(wb).astype(np.float32), "e2m1")
    assert np.array_equal(host(lin.w_codes), codes) and np.array_equal(host(lin.w_sf), sf)


def test_made_on_the_null_stream():
    """Raw stream 0 is the default one: behind the work that makes the weight there."""
    rng = np.random.default_rng(9)
    wb = _bf16(rng, (256, 1024), 2.0 ** -5)
    w, made, side = torch.zeros((256, 1024), dtype=torch.int16, device=DEV), dev(wb), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    w.copy_(made)
    with torch.cuda.stream(side):
        lin = LY.MxLinear(w, 4, stream=0)
    torch.cuda.synchronize()
    codes, sf = M.quantize_mx(F.bf16_to_f64(wb).astype(np.float32), "e2m1")
    assert np.array_equal(host(lin.w_codes), codes) and np.array_equal(host(lin.w_sf), sf)
