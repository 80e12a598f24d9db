"""Pins of the oracles of the grouped products, the gated activation and the 8-bit
blocks: hand-computed values, and gradients against differences."""
import numpy as np

from oracle import fp8 as Q
from oracle import grouped as G


def test_forward_and_gradients_of_two_experts_by_hand():
    off, cnt = np.array([0, 2, 3]), np.array([1, 1])
    x = np.array([[1.0, 2.0], [9.0, 9.0], [3.0, -1.0], [7.0, 7.0]])
    w = np.array([[[1.0, 0.0], [1.0, 1.0]], [[2.0, 1.0], [0.0, 4.0]]])
    out, mags = G.forward(x, w, off, cnt, np.full((4, 2), 5.0))
    assert np.array_equal(out, [[1, 3], [0, 0], [5, -4], [5, 5]]) and np.array_equal(mags[2], [7, 4])
    d = np.array([[1.0, 1.0], [8.0, 8.0], [2.0, -1.0], [6.0, 6.0]])
    d_x, _ = G.input_grad(d, w, off, cnt, np.full((4, 2), 5.0))
    assert np.array_equal(d_x, [[2, 1], [0, 0], [4, -2], [5, 5]])
    d_w, _ = G.weight_grad(d, x, off, cnt, 2, 2)
    assert np.array_equal(d_w, [[[1, 2], [1, 2]], [[6, -2], [-3, 1]]])


def test_swiglu_values():
    y = G.swiglu(np.array([[0.0, 1.0, -1.0, 700.0, -700.0, 2.0, 3.0, 4.0, 2.0, 1.0]]))
    s1 = 1 / (1 + np.exp(-1))
    assert np.allclose(y, [[0.0, s1 * 3, -(1 - s1) * 4, 1400.0, -700.0 * np.exp(-700.0)]], rtol=1e-14, atol=0)


def test_layer_gradients_against_differences():
    rng = np.random.default_rng(0)
    T, K, E, H, I = 3, 2, 4, 5, 3
    x, w13, w2 = rng.standard_normal((T, H)), rng.standard_normal((E, 2 * I, H)), rng.standard_normal((E, H, I))
    ids, weights, d = np.array([[0, 2], [3, -1], [2, 1]]), rng.random((T, K)), rng.standard_normal((T, H))
    grads = G.expert_mlp_grads(x, ids, weights, w13, w2, d)
    args, h = [x, w13, w2, weights], 1e-5

    def loss(x, w13, w2, weights):
        return (G.expert_mlp(x, ids, weights, w13, w2) * d).sum()

    for i, g in zip((0, 1, 2, 3), grads):
        v = rng.standard_normal(args[i].shape)
        up, down = list(args), list(args)
        up[i], down[i] = args[i] + h * v, args[i] - h * v
        # h^2 of third derivatives of values about 10, and 1e-16 / h of them
        assert abs((loss(*up) - loss(*down)) / (2 * h) - (g * v).sum()) < 1e-6


def test_blocks_of_a_row_and_of_a_weight():
    x = np.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 129], x[1, 5] = 7.0, 0.21875, -3.5, np.inf
    codes, sf = Q.quantize(x, 1)
    assert np.array_equal(sf[0], np.float32([7 / 448, 3.5 / 448])) and np.isnan(sf[1, 0])
    assert sf[1, 1] == np.float32(2.0 ** -100) / np.float32(448)
    assert codes[0, 0] == 0x7E and codes[0, 129] == 0xFE and not codes[1].any()
    assert Q.values(codes, sf, 1)[0, 1] == 14.0 * np.float64(np.float32(7 / 448))      # 448 * 0.21875 / 7, a value of the grid
    codes, sf = Q.quantize(np.where(np.isinf(x), 0, x), 128)
    assert sf.shape == (1, 2) and sf[0, 0] == np.float32(7 / 448)


def test_ties_go_to_the_even_code_whatever_the_scale():
    """v = m * t / 448 for the ties t = 17, 19, 21 of the grid's steps of 2 (m a multiple
    of 7 has them in bf16; 21 is one for any m)."""
    for m, t, want in ((7.0, 17.0, 16.0), (7.0, 19.0, 20.0), (9.1875, 21.0, 20.0), (0.0703125, 21.0, 20.0)):
        x = np.zeros((1, 16))
        x[0, 0], x[0, 1] = m, m * t / 448
        codes, sf = Q.quantize(x, 1)
        assert np.isclose(Q.values(codes, sf, 1)[0, 1] / np.float64(sf[0, 0]), want, rtol=0, atol=1e-12)
