"""The products grouped by expert and their gradients against the oracle in 64 bits:
every block size, ragged and empty experts, offsets of any kind, NaN in whatever
may not be read, strides, accumulation, wrong maps."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F
from oracle import grouped as G

from .gpu_common import DEV, dev, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # half a step, relative
LEFT = 7.25                                        # what the outputs hold before


def _bound(ref, mags, K, dt):
    """A step of 16 products is summed in at most 4 levels of additions and added to an
    fp32 accumulator: each addition is off by at most 2^-23 (rounded or cut) of its
    sum, itself at most the magnitudes': (K / 16 + 4) 2^-23 in all, rounded up by a step
    for a ragged K and one for a sum onto the output. Then half a step of the output."""
    err = (K / 16 + 6) * 2.0 ** -23 * mags
    return err + HALF[dt] * (np.abs(ref) + err) + 2.0 ** -149


def _near(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} values, first at {np.argwhere(bad)[0]}"


class Rows:
    """Experts of the given rows, each padded to a multiple of `align` and by `gap`
    rows more; `behind` rows behind the last. Random bf16 values, NaN in the others."""

    def __init__(self, counts, align=1, gap=0, behind=5, seed=0):
        self.counts = np.array(counts, np.int32)
        padded = [-(-c // align) * align + gap for c in counts]
        self.offsets = np.concatenate([[0], np.cumsum(padded)]).astype(np.int32)
        self.E, self.R = len(counts), int(self.offsets[-1]) + behind
        self.rng = np.random.default_rng(seed)
        self.live = np.zeros(self.R, bool)
        for e in range(self.E):
            self.live[self.offsets[e]:self.offsets[e] + self.counts[e]] = True
        self.maps = dev(self.offsets), dev(self.counts)

    def matrix(self, cols, pad=0):
        """A device matrix (a view of wider rows with pad) and its fp64 values."""
        v = self.rng.standard_normal((self.R, cols + pad)).astype(np.float32)
        v[~self.live] = np.nan
        t = torch.from_numpy(v).to(torch.bfloat16).to(DEV)[:, :cols]
        return t, np.nan_to_num(t.double().cpu().numpy())

    def weights(self, Nn, D):
        w = self.rng.standard_normal((self.E, Nn, D)).astype(np.float32)
        w[self.counts == 0] = np.nan            # of experts without rows nothing is read
        t = torch.from_numpy(w).to(torch.bfloat16).to(DEV)
        return t, np.nan_to_num(t.double().cpu().numpy())

    def out(self, cols, dt, pad=0):
        wide = torch.full((self.R, cols + pad), LEFT, dtype=DT[dt], device=DEV)
        return wide, wide[:, :cols]


def _rows_call(r: Rows, Nn, D, dt, grad, pad=0, out_pad=0):
    cols_in, cols_out = (Nn, D) if grad else (D, Nn)
    say(f"{'input grad' if grad else 'forward'} E={r.E} R={r.R} N={Nn} D={D} {dt} pad={pad},{out_pad}")
    x, xv = r.matrix(cols_in, pad)
    w, wv = r.weights(Nn, D)
    wide, out = r.out(cols_out, dt, out_pad)
    (N.moe_grouped_gemm_dgrad if grad else N.moe_grouped_gemm)(x, w, *r.maps, out)
    torch.cuda.synchronize()
    ref, mags = (G.input_grad if grad else G.forward)(xv, wv, r.offsets, r.counts, np.full((r.R, cols_out), LEFT))
    got = wide.double().cpu().numpy()
    _near(got[:, :cols_out], ref, np.where(r.live[:, None], _bound(ref, mags, cols_in, dt), 0.0), "rows")
    assert (got[:, cols_out:] == LEFT).all()


def _weight_call(r: Rows, Nn, D, dt, accumulate, pad=0):
    say(f"weight grad E={r.E} R={r.R} N={Nn} D={D} {dt} accumulate={accumulate} pad={pad}")
    d, dv = r.matrix(Nn, pad)
    x, xv = r.matrix(D, pad)
    old = torch.from_numpy(r.rng.standard_normal((r.E, Nn, D)).astype(np.float32)).to(DT[dt]).to(DEV)
    d_w = old.clone() if accumulate else torch.full_like(old, float("nan"))
    N.moe_grouped_gemm_wgrad(d, x, *r.maps, d_w, accumulate)
    torch.cuda.synchronize()
    ref, mags = G.weight_grad(dv, xv, r.offsets, r.counts, Nn, D)
    if accumulate:
        ref, mags = ref + old.double().cpu().numpy(), mags + np.abs(old.double().cpu().numpy())
    tol = _bound(ref, mags, r.counts.max(initial=0), dt)
    empty = r.counts == 0
    tol[empty] = 0.0            # zeros, or what was there
    _near(d_w.double().cpu().numpy(), ref, tol, "d_w")


SMALL = [  # counts, alignment, gap, N, D: the 32-row blocks
    ([1], 1, 0, 8, 8), ([0, 1, 0], 16, 0, 16, 24), ([3, 0, 17, 32, 33], 16, 0, 72, 136), ([5, 31, 64], 1, 3, 128, 64),
    ([2] * 40, 16, 0, 264, 200), ([0, 0, 0], 16, 16, 40, 48), ([1, 2, 3, 4], 1, 0, 136, 1032)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("counts,align,gap,Nn,D", SMALL)
def test_few_rows(counts, align, gap, Nn, D, dt):
    r = Rows(counts, align, gap, seed=len(counts))
    _rows_call(r, Nn, D, dt, False)
    _rows_call(r, Nn, D, dt, True)
    for accumulate in (False, True):
        _weight_call(r, Nn, D, dt, accumulate)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
def test_blocks_of_128_rows(grad, dt):
    """4 experts, at least 150 blocks of 128 x 128: rows that leave 1 or 2 row tiles of a
    wave live, a whole block, and none."""
    r = Rows([130, 0, 257, 413], 16, 0, seed=1)
    wide, deep = 2600, 200
    _rows_call(r, *((deep, wide) if grad else (wide, deep)), dt, grad, pad=8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("deep", [72, 8, 328])
def test_blocks_of_256_rows(deep, grad, dt):
    """8 experts, at least 448 blocks of 256 x 256: the last block of an expert with 1,
    2, 3 and 4 row tiles of a wave live, of padding alone, and experts without rows."""
    r = Rows([0, 1, 256, 257, 330, 450, 511, 640], 1, 270, seed=2)
    wide = 9000
    _rows_call(r, *((deep, wide) if grad else (wide, deep)), dt, grad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("counts,align,gap,out_pad", [
    ([257, 288, 300, 320, 321, 513, 640, 641], 1, 0, 0), ([769, 961, 1100, 640, 257, 1], 128, 0, 3),
    ([300, 257, 620, 0, 255, 1500], 16, 400, 0), ([4500], 128, 0, 8)])
def test_blocks_of_320_rows(counts, align, gap, out_pad, grad, dt):
    """Experts whose rows fill fewer blocks of 320 x 192 than of 256 x 256, beside others:
    equal sides, a last block of padding alone, rows that start anywhere."""
    r = Rows(counts, align, gap, seed=len(counts))
    wide, deep = 6400, 136
    _rows_call(r, *((deep, wide) if grad else (wide, deep)), dt, grad, out_pad=out_pad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_grad_blocks_of_256(accumulate, dt):
    r = Rows([0, 1, 63, 64, 65, 400, 700, 300], 16, 0, seed=3)
    _weight_call(r, 1272, 1528, dt, accumulate)


@pytest.mark.parametrize("way", ["forward", "input", "weight"])
@pytest.mark.parametrize("counts", [[1000], [0, 2000]])
def test_long_contractions(counts, way):
    """Many stages: the ring goes round often, its last stage whole or not."""
    r = Rows(counts, 1, 0, seed=4)
    if way == "weight":
        _weight_call(r, 136, 72, "f32", False)
    elif way == "forward":
        _rows_call(r, 136, 4104, "f32", False)
    else:
        _rows_call(r, 4160, 136, "f32", True)


@pytest.mark.parametrize("out_pad", [1, 4, 8])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_output_rows_of_any_stride(dt, out_pad):
    r = Rows([7, 40, 0, 20], 16, 0, seed=5)
    _rows_call(r, 72, 64, dt, False, pad=16, out_pad=out_pad)
    _rows_call(r, 64, 200, dt, True, pad=8, out_pad=out_pad)
    _weight_call(r, 72, 40, dt, False, pad=8)


@pytest.mark.parametrize("E", [1, 255, 256, 257, 1000, 1024])
def test_experts_in_number(E):
    """The search for a block's expert: a thread looks at 1 to 4 of them."""
    rng = np.random.default_rng(E)
    r = Rows(rng.integers(0, 4, E).tolist(), 1, 0, seed=6)
    _rows_call(r, 16, 24, "f32", False)
    _rows_call(r, 16, 24, "f32", True)
    _weight_call(r, 16, 24, "f32", False)


def test_no_rows():
    w = torch.ones((3, 16, 8), dtype=torch.bfloat16, device=DEV)
    zero = torch.zeros(4, dtype=torch.int32, device=DEV)
    x, d = (torch.empty((0, c), dtype=torch.bfloat16, device=DEV) for c in (8, 16))
    N.moe_grouped_gemm(x, w, zero, zero[:3].clone(), torch.empty((0, 16), device=DEV))
    N.moe_grouped_gemm_wgrad(d, x, zero, zero[:3].clone(), w)
    torch.cuda.synchronize()
    assert (w == 0).all()
    w.fill_(3.0)
    N.moe_grouped_gemm_wgrad(d, x, zero, zero[:3].clone(), w, True)
    torch.cuda.synchronize()
    assert (w == 3.0).all()


def test_no_contraction():
    """D = 0 of the forward product: zeros in the experts' rows."""
    r = Rows([3, 0, 9], 16, 0, seed=7)
    wide, out = r.out(32, "f32")
    N.moe_grouped_gemm(torch.empty((r.R, 0), dtype=torch.bfloat16, device=DEV),
                       torch.empty((3, 32, 0), dtype=torch.bfloat16, device=DEV), *r.maps, out)
    torch.cuda.synchronize()
    got, end = out.cpu().numpy(), int(r.offsets[-1])
    assert (got[:end] == 0).all() and (got[end:] == np.float32(LEFT)).all()


def test_infinities_and_nans_stay_in_their_rows():
    r = Rows([20, 40], 16, 0, seed=8)
    x, xv = r.matrix(64)
    w, wv = r.weights(48, 64)
    x[3, 5], x[40, 7] = float("inf"), float("nan")
    w[1, 9, 11] = float("nan")
    wide, out = r.out(48, "bf16")
    N.moe_grouped_gemm(x, w, *r.maps, out)
    torch.cuda.synchronize()
    bad = ~np.isfinite(out.float().cpu().numpy())
    want = np.zeros_like(bad)
    want[3] = want[40] = True
    want[int(r.offsets[1]):int(r.offsets[1]) + 40, 9] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("offsets,counts", [([-5, 10, 1 << 30], [1 << 30, -3]), ([40, 20, 10], [7, 7]),
                                            ([0, 100, 200], [1 << 31 - 1, 5]), ([90, 95, 97], [50, 50])])
def test_wrong_maps_stay_inside_the_rows(offsets, counts):
    """Rows on both sides of the buffers stay; the values are not looked at."""
    guard, R = 64, 96
    o, c = dev(np.array(offsets, np.int32)), dev(np.array(counts, np.int32))
    w = torch.ones((2, 40, 72), dtype=torch.bfloat16, device=DEV)
    for grad in (False, True):
        cols_in, cols_out = (40, 72) if grad else (72, 40)
        x = torch.ones((R, cols_in), dtype=torch.bfloat16, device=DEV)
        out = torch.full((guard + R + guard, cols_out), LEFT, device=DEV)
        say("wrong maps", offsets, counts, grad)
        (N.moe_grouped_gemm_dgrad if grad else N.moe_grouped_gemm)(x, w, o, c, out[guard:guard + R])
        torch.cuda.synchronize()
        assert (out[:guard] == LEFT).all() and (out[guard + R:] == LEFT).all()
    d_w = torch.zeros((2, 40, 72), device=DEV)
    N.moe_grouped_gemm_wgrad(torch.ones((R, 40), dtype=torch.bfloat16, device=DEV),
                             torch.ones((R, 72), dtype=torch.bfloat16, device=DEV), o, c, d_w)
    torch.cuda.synchronize()
    assert (d_w <= R).all()


def test_one_expert_of_all_rows():
    """The limits of the maps: {0, INT32_MAX} and {INT32_MAX}."""
    r = Rows([77], 1, 0, behind=0, seed=9)
    x, xv = r.matrix(64)
    d, dv = r.matrix(40)
    big = np.int32(2 ** 31 - 1)
    d_w = torch.empty((1, 40, 64), device=DEV)
    N.moe_grouped_gemm_wgrad(d, x, dev(np.array([0, big], np.int32)), dev(np.array([big], np.int32)), d_w)
    torch.cuda.synchronize()
    ref, mags = G.weight_grad(dv, xv, r.offsets, r.counts, 40, 64)
    _near(d_w.double().cpu().numpy(), ref, _bound(ref, mags, 77, "f32"), "d_w")


def test_same_bits_from_call_to_call_and_stream_to_stream():
    r = Rows([130, 0, 257, 413], 16, 0, seed=10)
    x, _ = r.matrix(200)
    w, _ = r.weights(2600, 200)
    _, first = r.out(2600, "bf16")
    N.moe_grouped_gemm(x, w, *r.maps, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side, side.cuda_stream):
        _, out = r.out(2600, "bf16")
        side.wait_stream(torch.cuda.current_stream())
        N.moe_grouped_gemm(x, w, *r.maps, out, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, first)


def test_gradients_are_those_of_the_product():
    """<d_out, forward(x + t v)> is linear in x: its difference is <d_x, v>, and with w
    likewise; on whole numbers, which every product and sum holds exactly."""
    r = Rows([9, 0, 33], 16, 0, seed=11)
    rng = np.random.default_rng(12)

    def whole(*dims):
        return torch.from_numpy(rng.integers(-3, 4, dims).astype(np.float32)).to(torch.bfloat16).to(DEV)

    live = torch.from_numpy(r.live).to(DEV)[:, None]
    x, v, d = (torch.where(live, whole(r.R, c), 0.0) for c in (40, 40, 24))
    w, wv = whole(3, 24, 40), whole(3, 24, 40)

    def loss(x, w):
        out = torch.zeros((r.R, 24), device=DEV)
        N.moe_grouped_gemm(x, w, *r.maps, out)
        return (out.double() * d.double()).sum()

    d_x, d_w = torch.zeros((r.R, 40), device=DEV), torch.empty((3, 24, 40), device=DEV)
    N.moe_grouped_gemm_dgrad(d, w, *r.maps, d_x)
    N.moe_grouped_gemm_wgrad(d, x, *r.maps, d_w)
    assert (loss(x + v, w) - loss(x, w)).item() == (d_x.double() * v.double()).sum().item()
    assert (loss(x, w + wv) - loss(x, w)).item() == (d_w.double() * wv.double()).sum().item()


def test_rows_past_32_bits():
    """Rows 128 KiB apart, the second expert's behind 4 GiB; the last of 9 experts'
    weights behind 2^32 elements."""
    R, stride = 40000, 65536
    x = torch.empty((R, stride), dtype=torch.bfloat16, device=DEV)[:, :64]
    x.zero_()
    x[-40:] = torch.randn(40, 64, device=DEV).bfloat16()
    w = torch.randn(2, 24, 64, device=DEV).bfloat16()
    maps = dev(np.array([0, R - 40, R], np.int32)), dev(np.array([1, 40], np.int32))
    out, d_w = torch.zeros((R, 24), device=DEV), torch.empty((2, 24, 64), device=DEV)
    d_out = torch.randn(R, 24, device=DEV).bfloat16()
    say("rows past 32 bits")
    N.moe_grouped_gemm(x, w, *maps, out)
    N.moe_grouped_gemm_wgrad(d_out, x, *maps, d_w)
    torch.cuda.synchronize()
    xv, wv, dv = (t.double().cpu().numpy() for t in (x[-40:], w[1], d_out[-40:]))
    _near(out[-40:].double().cpu().numpy(), xv @ wv.T, _bound(xv @ wv.T, np.abs(xv) @ np.abs(wv).T, 64, "f32"), "out")
    _near(d_w[1].double().cpu().numpy(), dv.T @ xv, _bound(dv.T @ xv, np.abs(dv).T @ np.abs(xv), 40, "f32"), "d_w")
    del x, out, d_w, d_out
    E, Nn, D = 9, 32768, 16384
    w = torch.empty((E, Nn, D), dtype=torch.bfloat16, device=DEV)
    w[8].zero_()
    w[8, -24:] = torch.randn(24, D, device=DEV).bfloat16()
    x = torch.randn(3, D, device=DEV).bfloat16()
    maps = dev(np.array([0] * 9 + [3], np.int32)), dev(np.array([0] * 8 + [3], np.int32))
    out = torch.empty((3, Nn), device=DEV)
    N.moe_grouped_gemm(x, w, *maps, out)
    torch.cuda.synchronize()
    xv, wv = x.double().cpu().numpy(), w[8, -24:].double().cpu().numpy()
    _near(out[:, -24:].double().cpu().numpy(), xv @ wv.T, _bound(xv @ wv.T, np.abs(xv) @ np.abs(wv).T, D, "f32"), "out")
    assert (out[:, :-24] == 0).all()
