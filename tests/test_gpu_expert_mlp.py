"""The trained experts as a program runs them: routing, forward and backward, each
call against the oracle on what the call before it gave, the whole against the
formula's gradients, captured and replayed with other tokens."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from oracle import grouped as G
from oracle import sort as S

from .gpu_common import DEV, say

pytestmark = pytest.mark.gpu

SHAPES = [  # T, K, E, H, I, tile
    (1, 1, 1, 8, 8, 16), (5, 2, 4, 64, 24, 16), (64, 4, 8, 136, 72, 32), (300, 2, 4, 128, 264, 128)]


class Step:
    """One layer's tensors, and a forward and a backward on them."""

    def __init__(self, T, K, E, H, I, tile, seed=0, padding=0.2):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)

        def normal(*dims, scale=1.0):
            return (scale * torch.randn(*dims, generator=g, device=DEV)).bfloat16()

        self.dims = T, K, E, H, I
        self.routing = LY.Routing(T, K, E, tile)
        self.mlp = LY.ExpertMlp(T, K, E, H, I, tile)
        self.logits = torch.randn(T, E, generator=g, device=DEV)
        self.pad = (torch.rand(T, generator=g, device=DEV) < padding).to(torch.uint8)
        self.x, self.d_out = normal(T, H), normal(T, H)
        self.w13, self.w2 = normal(E, 2 * I, H, scale=H ** -0.5), normal(E, H, I, scale=I ** -0.5)
        self.out, self.d_x = (torch.empty((T, H), dtype=torch.bfloat16, device=DEV) for _ in range(2))
        self.d_w13, self.d_w2 = torch.empty(E, 2 * I, H, device=DEV), torch.empty(E, H, I, device=DEV)
        self.d_weights = torch.empty(T, K, device=DEV)

    def forward(self, stream=None):
        self.routing(self.logits, None, self.pad, 1.5, stream)
        self.mlp.forward(self.x, self.routing, self.w13, self.w2, self.out, stream)

    def backward(self, accumulate=False, stream=None):
        self.mlp.backward(self.d_out, self.routing, self.w13, self.w2, self.d_x, self.d_w13, self.d_w2, self.d_weights,
                          accumulate, stream)

    def results(self):
        torch.cuda.synchronize()
        return [t.clone() for t in (self.out, self.d_x, self.d_w13, self.d_w2, self.d_weights)]


def _v(t):
    return t.double().cpu().numpy()


def _near(got, ref, err, half, what):
    bad = ~(np.abs(got - ref) <= err + half * (np.abs(ref) + err) + 2.0 ** -134)
    assert not bad.any(), f"{what}: {int(bad.sum())} values, first at {np.argwhere(bad)[0]}"


BF16, F32 = 2.0 ** -8, 2.0 ** -24


def _sum_err(mags, K):
    """Of a product over K, as in the grouped products' own tests."""
    return (K / 16 + 6) * 2.0 ** -23 * mags


@pytest.mark.parametrize("T,K,E,H,I,tile", SHAPES)
def test_every_call_on_what_the_one_before_gave(T, K, E, H, I, tile):
    s = Step(T, K, E, H, I, tile, seed=T)
    say(f"ExpertMlp T={T} K={K} E={E} H={H} I={I} tile={tile}")
    s.forward()
    torch.cuda.synchronize()
    r, m = s.routing, s.mlp
    p, total = r.exp2perm.cpu().numpy(), int(r.total_rows.item())
    off, cnt = r.expert_offsets.cpu().numpy(), r.expert_counts.cpu().numpy()
    held = r.perm2tok.cpu().numpy() >= 0
    used = np.arange(m.R) < total
    wv, w13, w2 = _v(r.weights), _v(s.w13), _v(s.w2)
    rows, gate_up, inter, out_rows = (_v(t) for t in (m.rows, m.gate_up, m.inter, m.out_rows))
    assert np.array_equal(rows[used], S.dispatch(_v(s.x), p, total, rows)[used])

    def product(got, x, w, K, what):
        ref, mags = G.forward(x, w, off, cnt, np.zeros((m.R, w.shape[1])))
        _near(got[used], ref[used], _sum_err(mags, K)[used], BF16, what)

    product(gate_up, rows, w13, H, "gate_up")
    _near(inter[held], G.swiglu(gate_up)[held], 11 * F32 * np.abs(G.swiglu(gate_up)[held]), BF16, "inter")
    assert (inter[used & ~held] == 0).all()
    product(out_rows, inter, w2, I, "out_rows")
    _near(_v(s.out), S.combine(out_rows, p, wv), K * F32 * S.combine(np.abs(out_rows), p, np.abs(wv)), BF16, "out")

    s.backward()
    torch.cuda.synchronize()
    d_out, d_rows2, d_gate_up, d_inter, d_rows = _v(s.d_out), _v(m.out_rows), _v(m.gate_up), _v(m.d_inter), _v(m.d_rows)
    want = np.zeros_like(d_rows2)
    for t, k in np.argwhere(p >= 0):
        want[p[t, k]] = wv[t, k] * d_out[t]
    _near(d_rows2[used], want[used], 0.0, BF16, "d_rows2")

    def grads(got, d, x, what):
        ref, mags = G.weight_grad(d, x, off, cnt, d.shape[1], x.shape[1])
        _near(_v(got), ref, _sum_err(mags, cnt.max()), F32, what)

    def inputs(got, d, w, K, what):
        ref, mags = G.input_grad(d, w, off, cnt, np.zeros((m.R, w.shape[2])))
        _near(got[used], ref[used], _sum_err(mags, K)[used], BF16, what)

    grads(s.d_w2, d_rows2, inter, "d_w2")
    inputs(d_inter, d_rows2, w2, H, "d_inter")
    ref = G.swiglu_grad(d_inter, gate_up)
    g, u = np.split(gate_up, 2, axis=1)
    sg, rest = G.sigmoid(g), G.sigmoid(-g)
    mags = np.concatenate([np.abs(d_inter * u) * (sg + np.abs(g) * sg * rest), np.abs(ref[:, I:])], axis=1)
    _near(d_gate_up[held], ref[held], 11 * F32 * mags[held], BF16, "d_gate_up")
    grads(s.d_w13, d_gate_up, rows, "d_w13")
    inputs(d_rows, d_gate_up, w13, 2 * I, "d_rows")
    ones = np.ones((T, K))
    _near(_v(s.d_x), S.combine(d_rows, p, ones), K * F32 * S.combine(np.abs(d_rows), p, ones), BF16, "d_x")
    dots = np.zeros((T, K))
    mags = np.zeros((T, K))
    for t, k in np.argwhere(p >= 0):
        dots[t, k], mags[t, k] = out_rows[p[t, k]] @ d_out[t], np.abs(out_rows[p[t, k]]) @ np.abs(d_out[t])
    _near(_v(s.d_weights), dots, (H / 8 + 16) * F32 * mags, F32, "d_weights")


def test_gradients_of_the_whole_layer():
    """Against the formula's, in norm: the longest path rounds 7 times to bf16 (gate_up,
    inter, out_rows' gradient, d_inter, d_gate_up, d_rows, d_x), each off by at most 2^-8 of
    a value; on random signs products and sums keep the relative size of errors, so 7 *
    2^-8 even if they all added up."""
    s = Step(64, 4, 8, 136, 72, 32, seed=3)
    s.forward()
    s.backward()
    got = [_v(t) for t in s.results()]
    ids = np.where(s.routing.exp2perm.cpu().numpy() >= 0, s.routing.ids.cpu().numpy(), -1)
    args = _v(s.x), ids, _v(s.routing.weights), _v(s.w13), _v(s.w2)
    want = [G.expert_mlp(*args), *G.expert_mlp_grads(*args, _v(s.d_out))]
    for a, b, name in zip(got, want, ("out", "d_x", "d_w13", "d_w2", "d_weights")):
        err = np.linalg.norm(a - b) / np.linalg.norm(b)
        say(f"{name}: {err:.2e}")
        assert err <= 7 * 2.0 ** -8, name


def test_accumulated_gradients_and_second_batches():
    """Two batches' gradients in one buffer: the second added in fp32 to the first."""
    s = Step(40, 2, 4, 64, 40, 16, seed=4)
    s.forward()
    s.backward()
    first = s.results()
    s.forward()
    s.backward(accumulate=True)
    twice = s.results()
    for a, b in zip(first[2:4], twice[2:4]):
        assert torch.equal(a + a, b)
    assert torch.equal(first[0], twice[0]) and torch.equal(first[1], twice[1]) and torch.equal(first[4], twice[4])
    with pytest.raises(ValueError, match="forward"):
        s.backward()


@pytest.mark.parametrize("T,K,E,H,I,tile", [(8, 2, 8, 64, 24, 16), (300, 2, 4, 128, 264, 128)])
def test_replays_of_a_captured_step(T, K, E, H, I, tile):
    """Forward and backward in one graph, replayed with other tokens and routings, eager
    work on the same buffers in between: every replay equals the eager step bit for bit."""
    s = Step(T, K, E, H, I, tile, seed=5)
    s.forward()
    s.backward()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.forward()
        s.backward()
    say("captured a step; replaying")
    for it in range(4):
        s.logits.copy_(torch.randn(T, E, device=DEV))
        s.x.copy_(torch.randn(T, H, device=DEV))
        s.pad.copy_(torch.rand(T, device=DEV) < 0.3 * it)
        s.forward()
        s.backward()
        eager = s.results()
        for t in (s.out, s.d_x, s.d_w13, s.d_w2, s.d_weights):
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        for a, b in zip(s.results(), eager):
            assert torch.equal(a, b)


def test_on_another_stream_beside_other_work():
    a, b = Step(64, 4, 8, 136, 72, 32, seed=6), Step(64, 4, 8, 136, 72, 32, seed=7)
    want = []
    for s in (a, b):
        s.forward()
        s.backward()
        want.append(s.results())
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for it in range(3):
        for s, stream in zip((a, b), streams):
            stream.wait_stream(torch.cuda.current_stream())
            s.forward(stream)
            s.backward(stream=stream.cuda_stream)
        for s, w in zip((a, b), want):
            for x, y in zip(s.results(), w):
                assert torch.equal(x, y)


def test_a_batch_of_padding_alone_and_of_no_tokens():
    s = Step(6, 2, 4, 64, 24, 16, seed=8, padding=1.1)
    s.forward()
    s.backward()
    out = s.results()
    assert all((t == 0).all() for t in out)
    s = Step(0, 2, 4, 64, 24, 16)
    s.mlp.forward(s.x, s.routing, s.w13, s.w2, s.out)


def test_the_backward_of_no_tokens():
    s = Step(0, 2, 4, 64, 24, 16)
    s.forward()
    for accumulate, want in ((True, 1.0), (False, 0.0)):
        for t in (s.d_w13, s.d_w2):
            t.fill_(1.0)
        s.mlp.forward(s.x, s.routing, s.w13, s.w2, s.out)
        s.backward(accumulate=accumulate)
        assert (s.d_w13 == want).all() and (s.d_w2 == want).all()
