"""The grouped products through the blocks that their tests are about, asserted: the edges
of the tall ones, each side, and maps with the largest counts and offsets."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N

from . import kernel_choice as C
from .gpu_common import DEV, dev, say
from .test_gpu_grouped import LEFT, Rows, _rows_call, _weight_call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("deep", [72, 264])
def test_edges_of_the_tall_blocks(deep, grad, dt):
    """One row below, at and above what one block of 320 x 192 holds, and two."""
    counts, wide = [257, 288, 300, 320, 321, 513, 640, 641], 7200
    r = Rows(counts, 1, 0, seed=41)
    assert C.grouped_side(r.R, r.E, wide) == 256
    assert [C.grouped_tall(c, c, wide) for c in counts] == [True, True, True, True, False, True, True, False]
    _rows_call(r, *((deep, wide) if grad else (wide, deep)), dt, grad, pad=8, out_pad=3)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("gap,full", [(0, True), (159, True), (160, True), (161, False), (500, False)])
def test_padding_behind_tall_blocks(gap, full, grad, dt):
    """Up to half a block more is the last one's (160 rows behind 320), more than that
    blocks of its own, which may make square ones the fewer."""
    counts, wide, deep = [290, 600, 320, 300], 16640, 72
    r = Rows(counts, 1, gap, seed=42)
    assert C.grouped_side(r.R, r.E, wide) == 256
    assert [C.grouped_tall(c, c + gap, wide) for c in counts] == [True, True, full, True]
    _rows_call(r, *((deep, wide) if grad else (wide, deep)), dt, grad)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("side,counts,wide", [(32, [31, 32, 33, 63, 64, 65, 0, 1], 264), (128, [127, 128, 129, 255, 256, 257, 0, 1], 2608),
                                              (256, [255, 256, 511, 512, 767, 768, 0, 1], 7208)])
def test_edges_of_each_side(side, counts, wide, grad, dt):
    r = Rows(counts, 1, 0, seed=43)
    assert C.grouped_side(r.R, r.E, wide) == side
    assert side < 256 or not any(C.grouped_tall(c, c, wide) for c in counts)
    _rows_call(r, *((136, wide) if grad else (wide, 136)), dt, grad, pad=8, out_pad=8)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("side,counts,Nn,D", [(128, [127, 128, 129, 0, 1], 136, 264), (256, [191, 192, 193, 600, 0, 64, 300, 129], 1272, 1288)])
def test_weight_gradients_of_each_side(side, counts, Nn, D, accumulate, dt):
    r = Rows(counts, 1, 0, seed=44)
    assert C.weight_side(r.R, r.E, Nn, D) == side
    _weight_call(r, Nn, D, dt, accumulate, pad=8)


@pytest.mark.parametrize("offsets,counts", [([0, 2 ** 31 - 1, 2 ** 31 - 1], [2 ** 31 - 1, 2 ** 31 - 1]), ([0, 48, 2 ** 31 - 1], [2 ** 31 - 1] * 2),
                                            ([-2 ** 31, 50, 96], [2 ** 31 - 1, 46]), ([0, 100, 200], [2 ** 31 - 1, 5]),
                                            ([2 ** 31 - 1, 0, -2 ** 31], [2 ** 31 - 1, -2 ** 31])])
def test_maps_of_the_largest_numbers(offsets, counts):
    """What each expert gets is its rows inside the buffers, [clamped first, clamped next),
    where those maps leave no doubt; nothing outside is touched."""
    guard, R, Nn, D = 64, 96, 40, 72
    o, c = np.array(offsets, np.int64), np.array(counts, np.int64)
    first = np.clip(o[:2], 0, R)
    end = np.maximum(np.clip(o[1:], 0, R), first)
    rows = np.clip(c, 0, end - first)
    maps = dev(o.astype(np.int32)), dev(c.astype(np.int32))
    w = torch.ones((2, Nn, D), dtype=torch.bfloat16, device=DEV)
    w[1] = 2.0
    say("maps", offsets, counts)
    for grad in (False, True):
        cols_in, cols_out = (Nn, D) if grad else (D, Nn)
        x = torch.ones((R, cols_in), dtype=torch.bfloat16, device=DEV)
        out = torch.full((guard + R + guard, cols_out), LEFT, device=DEV)
        (N.moe_grouped_gemm_dgrad if grad else N.moe_grouped_gemm)(x, w, *maps, out[guard:guard + R])
        torch.cuda.synchronize()
        want = np.full((R, cols_out), LEFT)
        for e in range(2):
            want[first[e]:first[e] + rows[e]] = cols_in * (e + 1)
            want[first[e] + rows[e]:end[e]] = 0.0
        assert np.array_equal(out[guard:guard + R].cpu().numpy(), want)
        assert (out[:guard] == LEFT).all() and (out[guard + R:] == LEFT).all()
    d_w = torch.full((2, Nn, D), float("nan"), device=DEV)
    N.moe_grouped_gemm_wgrad(torch.ones((R, Nn), dtype=torch.bfloat16, device=DEV),
                             torch.ones((R, D), dtype=torch.bfloat16, device=DEV), *maps, d_w)
    torch.cuda.synchronize()
    assert np.array_equal(d_w.cpu().numpy(), np.broadcast_to(rows.reshape(2, 1, 1), d_w.shape).astype(np.float32))
