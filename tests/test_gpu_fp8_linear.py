"""Fp8Linear as a program uses it: forward and both gradients equal their parts, the
weight again after a step, fewer tokens than it was made for, streams and captures."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from oracle import formats as F
from oracle import fp8 as Q

from .gpu_common import DEV, dev, host, say

pytestmark = pytest.mark.gpu


def _bits(rng, T, H, scale=1.0):
    return F.f32_to_bf16((rng.standard_normal((T, H)) * scale).astype(np.float32))


def _check(got, x_bits, w_values):
    """out against the exact product of the quantized values (bounds as the product's own
    tests derive them)."""
    K = x_bits.shape[1]
    av = Q.values(*Q.quantize(F.bf16_to_f64(x_bits), 1), 1)
    ref, mags, tops = Q.gemm(av, w_values)
    err = 2.0 ** -10 * tops + (13 + K / 128) * 2.0 ** -23 * mags
    assert (np.abs(F.bf16_to_f64(host(got)) - ref) <= err + 2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -134).all()


def _out(*dims):
    return torch.empty(dims, dtype=torch.int16, device=DEV)


@pytest.mark.parametrize("Nn,K", [(16, 16), (272, 400), (1040, 144)])
def test_forward_and_gradients(Nn, K):
    rng = np.random.default_rng(Nn)
    wb = _bits(rng, Nn, K, K ** -0.5)
    lin = LY.Fp8Linear(dev(wb), 130, grads=True)
    for T in (130, 1, 33):
        xb, db = _bits(rng, T, K), _bits(rng, T, Nn)
        x, d = dev(xb), dev(db)
        out, d_x, d_w = _out(T, Nn), _out(T, K), torch.empty((Nn, K), device=DEV)
        say(f"Fp8Linear N={Nn} K={K} T={T}")
        lin(x, out)
        lin.input_grad(d, d_x)
        lin.weight_grad(d, x, d_w)
        torch.cuda.synchronize()
        wv = Q.values(*Q.quantize(F.bf16_to_f64(wb), 128), 128)
        _check(out, xb, wv)
        _check(d_x, db, wv.T)
        dv, xv = F.bf16_to_f64(db), F.bf16_to_f64(xb)
        ref, mags = dv.T @ xv, np.abs(dv).T @ np.abs(xv)
        err = (T / 16 + 6) * 2.0 ** -23 * mags
        got = d_w.double().cpu().numpy()
        assert (np.abs(got - ref) <= err + 2.0 ** -24 * (np.abs(ref) + err)).all()
        again = d_w.clone()
        lin.weight_grad(d, x, again, accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(again, d_w + d_w)
    wb = _bits(rng, Nn, K)          # after a step
    lin.load(dev(wb))
    lin(x, out)
    torch.cuda.synchronize()
    _check(out, xb, Q.values(*Q.quantize(F.bf16_to_f64(wb), 128), 128))


def test_refusals():
    w = torch.zeros((48, 32), dtype=torch.bfloat16, device=DEV)
    lin = LY.Fp8Linear(w, 4)
    x, out = (torch.zeros((5, c), dtype=torch.bfloat16, device=DEV) for c in (32, 48))
    with pytest.raises(ValueError, match="more than the 4"):
        lin(x, out)
    with pytest.raises(ValueError, match="without grads"):
        lin.input_grad(out[:4], x[:4])
    with pytest.raises(ValueError, match="rows of 48"):
        lin(out[:4], x[:4])
    with pytest.raises(ValueError, match="a weight of"):
        lin.load(w[:32])


def test_no_tokens():
    """Empty calls; the weight's gradient of none is zeros, or what was there."""
    lin = LY.Fp8Linear(torch.zeros((48, 144), dtype=torch.bfloat16, device=DEV), 4, grads=True)
    x, d = (torch.zeros((0, c), dtype=torch.bfloat16, device=DEV) for c in (144, 48))
    lin(x, torch.empty_like(d))
    lin.input_grad(d, torch.empty_like(x))
    d_w = torch.ones((48, 144), device=DEV)
    lin.weight_grad(d, x, d_w, accumulate=True)
    assert (d_w == 1).all()
    lin.weight_grad(d, x, d_w)
    assert (d_w == 0).all()


def test_captured_with_a_step_of_the_weight():
    """Quantizing the weight, the product and its gradients in one graph: replays follow
    the weight and the tokens."""
    rng = np.random.default_rng(3)
    Nn, K, T = 272, 144, 40
    w, x, d = dev(_bits(rng, Nn, K)), dev(_bits(rng, T, K)), dev(_bits(rng, T, Nn))
    lin = LY.Fp8Linear(w, T, grads=True)
    out, d_x, d_w = _out(T, Nn), _out(T, K), torch.empty((Nn, K), device=DEV)

    def step():
        lin.load(w)
        lin(x, out)
        lin.input_grad(d, d_x)
        lin.weight_grad(d, x, d_w)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for it in range(4):
        for t in (w, x, d):
            t.copy_(dev(_bits(rng, *t.shape)))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (out, d_x, d_w)]
        for t in (out, d_x, d_w):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((out, d_x, d_w), want))


@pytest.mark.parametrize("raw", [False, True])
def test_on_its_own_stream(raw):
    """Made and called on a stream, as an object or as its number; the weight may go."""
    rng = np.random.default_rng(4)
    wb, xb = _bits(rng, 272, 400), _bits(rng, 20, 400)
    stream = torch.cuda.Stream()
    handle = stream.cuda_stream if raw else stream
    w, x, out = dev(wb), dev(xb), _out(20, 272)
    stream.wait_stream(torch.cuda.current_stream())
    lin = LY.Fp8Linear(w, 32, stream=handle)
    del w
    junk = [torch.full((272, 400), 0x7F7F, dtype=torch.int16, device=DEV) for _ in range(4)]
    lin(x, out, handle)
    torch.cuda.synchronize()
    assert junk
    _check(out, xb, Q.values(*Q.quantize(F.bf16_to_f64(wb), 128), 128))
