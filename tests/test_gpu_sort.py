"""The sort of tokens by expert and back, and its gradients, against the CPU
oracle, on moe_route's own maps."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N
from oracle import formats as F
from oracle import sort as S
from oracle.permute import permute

from .gpu_common import DEV, dev, host, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}     # half a step, relative


class Maps:
    """A routing of T tokens to K of E experts by moe_route, `local` of them here,
    some tokens padding; the maps as the calls take them, and on the host."""

    def __init__(self, T, K, E, tile, local=None, padding=0.0, seed=0):
        rng = np.random.default_rng(seed)
        local = E if local is None else local
        shape = LY.LayerShape(T, 64, 64, local, K, tile)
        bufs = LY.Buffers(shape, DEV)
        first = (E - local) // 2
        pad = (rng.random(T) < padding).astype(np.uint8)
        say(f"moe_route T={T} K={K} E={E} local={local} tile={tile} padding={padding}")
        N.moe_route(dev(rng.standard_normal((T, E)).astype(np.float32)), None, dev(pad), K, 1.0, tile, first, local,
                    bufs.ids, bufs.weights, bufs.meta)
        torch.cuda.synchronize()
        self.bufs, self.T, self.K, self.R = bufs, T, K, bufs.layout.rows_max
        self.dev = (bufs.exp2perm, bufs.perm2tok, bufs.meta[1:2])
        self.p, self.total = host(bufs.exp2perm), int(bufs.meta[1].item())
        want = permute(host(bufs.ids), first, local, tile)
        assert np.array_equal(self.p, want["exp2perm"]) and self.total == want["total_rows"]
        self.w = rng.random((T, K)).astype(np.float32) - 0.3


def _rand(rng, rows, H, dt, pad=0):
    """A device matrix of type dt (a view of wider rows with pad) and its fp64 values."""
    wide = torch.from_numpy(rng.standard_normal((rows, H + pad)).astype(np.float32)).to(DT[dt]).to(DEV)
    return wide[:, :H], wide[:, :H].double().cpu().numpy()


def _near(got, ref, tol, what):
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} values, first at {np.argwhere(bad)[0]}"


def _check_all(m: Maps, H, dt, pad=0, seed=1, inplace=False):
    rng = np.random.default_rng(seed)
    say(f"sort T={m.T} K={m.K} R={m.R} total={m.total} H={H} {dt} pad={pad} inplace={inplace}")
    x, xv = _rand(rng, m.T, H, dt, pad)
    rows, keep = _rand(rng, m.R, H, dt, pad)
    N.moe_dispatch(x, *m.dev, rows)
    torch.cuda.synchronize()
    assert np.array_equal(rows.double().cpu().numpy(), S.dispatch(xv, m.p, m.total, keep))

    rows, rv = _rand(rng, m.R, H, dt, pad)
    ones = np.ones((m.T, m.K))
    for w in (m.w, None):
        out, _ = _rand(rng, m.T, H, dt, pad)
        if w is None:
            N.moe_dispatch_bwd(rows, m.dev[0], out)
        else:
            N.moe_combine(rows, m.dev[0], dev(w), out)
        torch.cuda.synchronize()
        ref = S.combine(rv, m.p, (ones if w is None else w).astype(np.float64))
        mags = S.combine(np.abs(rv), m.p, np.abs(ones if w is None else w).astype(np.float64))
        # K fused multiply-adds of one fp32 rounding each, then the output's
        err = m.K * 2.0 ** -24 * mags
        _near(out.double().cpu().numpy(), ref, err + HALF[dt] * (np.abs(ref) + err), "combine" if w is not None else "dispatch_bwd")

    d_out, dv = _rand(rng, m.T, H, dt, pad)
    d_rows, keep = (rows, rv) if inplace else _rand(rng, m.R, H, dt, pad)
    d_w = torch.full((m.T, m.K), 9.0, device=DEV)
    N.moe_combine_bwd(d_out, rows, *m.dev, dev(m.w), d_rows, d_w)
    torch.cuda.synchronize()
    dr, dw = S.combine_bwd(dv, rv, m.p, m.total, m.w.astype(np.float64), keep)
    # one product rounded to fp32 and then to the rows' type
    _near(d_rows.double().cpu().numpy()[:m.total], dr[:m.total], (HALF[dt] + 2.0 ** -23) * np.abs(dr[:m.total]), "d_rows")
    assert np.array_equal(d_rows.double().cpu().numpy()[m.total:], keep[m.total:])
    mags = S.combine_bwd(np.abs(dv), np.abs(rv), m.p, m.total, m.w, np.abs(keep))[1]
    # a chain of at most 32 fused multiply-adds a thread, 6 additions in the wave, 16 over the waves
    _near(d_w.double().cpu().numpy(), dw, 56 * 2.0 ** -24 * mags, "d_weights")
    assert (d_w.cpu().numpy()[m.p < 0] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,K,E,tile,local,padding", [
    (1, 1, 1, 16, None, 0.0), (1, 8, 64, 16, None, 0.0), (4, 2, 8, 16, None, 0.5), (8, 8, 64, 16, 32, 0.0), (33, 3, 8, 32, 3, 0.2),
    (64, 8, 128, 16, None, 0.0), (100, 32, 40, 256, None, 0.1), (5, 2, 8, 16, 4, 1.0), (600, 8, 64, 128, 32, 0.1),
    (777, 9, 16, 64, None, 0.0)])
def test_routings(T, K, E, tile, local, padding, dt):
    """One token to many, all experts here or some, padding tokens (all of them
    too: no row), more routes than one batch of loads."""
    m = Maps(T, K, E, tile, local, padding)
    _check_all(m, 136, dt)
    _check_all(m, 136, dt, seed=2, inplace=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T", [20, 520])
@pytest.mark.parametrize("H,pad", [(8, 0), (8, 8), (1024, 16), (1032, 0), (2056, 8), (4096, 0), (4104, 0), (8200, 8), (16384, 0)])
def test_widths(H, pad, T, dt):
    _check_all(Maps(T, 4, 16, 16, padding=0.1), H, dt, pad)


@pytest.mark.parametrize("T", [1, 30, 700])
def test_dispatch_moves_any_type(T):
    """Quantized rows: codes and scales as bytes, in rows of any multiple of 16 bytes."""
    m = Maps(T, 4, 16, 16)
    rng = np.random.default_rng(3)
    for W, dt in ((16, np.uint8), (48, np.uint8), (4112, np.uint8), (8, np.int16), (16384, np.float32)):
        x = rng.integers(0, 100, (T, W)).astype(dt)
        keep = rng.integers(100, 120, (m.R, W)).astype(dt)
        rows = torch.from_numpy(keep).to(DEV)
        N.moe_dispatch(torch.from_numpy(x).to(DEV), *m.dev, rows)
        torch.cuda.synchronize()
        assert np.array_equal(rows.cpu().numpy(), S.dispatch(x, m.p, m.total, keep))


def test_special_values_stay_with_their_routes():
    """NaN and infinity in padding rows, in rows behind the last tile and in rows
    of absent routes' tokens reach nothing; in a routed row, its token alone."""
    m = Maps(40, 4, 16, 16, local=8)
    rng = np.random.default_rng(5)
    rows, rv = _rand(rng, m.R, 64, "bf16")
    held = np.zeros(m.R, bool)
    held[m.p[m.p >= 0]] = True
    rows[torch.from_numpy(~held).to(DEV)] = float("nan")
    hit = m.p[m.p >= 0][0]
    rows[int(hit), 3] = float("inf")
    out = torch.empty(40, 64, dtype=torch.bfloat16, device=DEV)
    N.moe_combine(rows, m.dev[0], dev(np.abs(m.w) + 1), out)
    d_out, _ = _rand(rng, 40, 64, "bf16")
    d_out[torch.from_numpy((m.p < 0).all(1)).to(DEV)] = float("nan")
    d_rows, d_w = torch.empty_like(rows), torch.empty(40, 4, device=DEV)
    N.moe_combine_bwd(d_out, rows, *m.dev, dev(m.w), d_rows, d_w)
    torch.cuda.synchronize()
    o = out.float().cpu().numpy()
    t = np.argwhere(m.p == hit)[0][0]
    assert np.isinf(o[t, 3]) and np.isfinite(np.delete(o.reshape(-1), t * 64 + 3)).all()
    assert torch.isfinite(d_rows[:m.total]).all()
    assert np.isfinite(np.delete(d_w.cpu().numpy().reshape(-1), np.argwhere(m.p.reshape(-1) == hit)[0])).all()


def test_gradients_against_differences():
    """The training step of a caller's own experts: dispatch, a product per
    expert, combine, and back through the calls; the loss against central
    differences along random directions, in fp32 with fp64 products between."""
    m = Maps(48, 3, 8, 16, padding=0.1)
    rng = np.random.default_rng(9)
    H, L = 32, m.bufs.layout
    off = host(m.bufs.field("expert_offsets", 9))
    wt = [torch.from_numpy(rng.standard_normal((H, H)) / H ** 0.5).to(DEV) for _ in range(8)]
    seed_out = torch.from_numpy(rng.standard_normal((m.T, H)).astype(np.float32)).to(DEV)

    def experts(rows, transpose=False):
        out = torch.zeros_like(rows)
        for e in range(8):
            a, b = int(off[e]), int(off[e + 1])
            out[a:b] = torch.tanh(rows[a:b].double() @ wt[e]).float()
        return out

    def forward(x, w):
        rows = torch.zeros(m.R, H, device=DEV)
        N.moe_dispatch(x, *m.dev, rows)
        y, out = experts(rows), torch.empty(m.T, H, device=DEV)
        N.moe_combine(y, m.dev[0], w, out)
        return rows, y, out

    x = torch.from_numpy(rng.standard_normal((m.T, H)).astype(np.float32)).to(DEV)
    w = dev(m.w)
    rows, y, out = forward(x, w)
    d_y, d_w = torch.zeros_like(y), torch.empty_like(w)
    N.moe_combine_bwd(seed_out, y, *m.dev, w, d_y, d_w)
    d_rows = torch.zeros_like(rows)
    for e in range(8):
        a, b = int(off[e]), int(off[e + 1])
        d_rows[a:b] = ((d_y[a:b].double() * (1 - y[a:b].double() ** 2)) @ wt[e].t()).float()
    d_x = torch.empty_like(x)
    N.moe_dispatch_bwd(d_rows, m.dev[0], d_x)

    def loss(x, w):
        return float((forward(x, w)[2].double() * seed_out.double()).sum())

    h = 2.0 ** -6
    for _ in range(3):
        vx = torch.from_numpy(rng.standard_normal((m.T, H)).astype(np.float32)).to(DEV)
        vw = torch.from_numpy(rng.standard_normal(m.w.shape).astype(np.float32)).to(DEV)
        for along, got in (((vx, 0 * vw), float((d_x.double() * vx.double()).sum())),
                           ((0 * vx, vw), float((d_w.double() * vw.double()).sum()))):
            diff = (loss(x + h * along[0], w + h * along[1]) - loss(x - h * along[0], w - h * along[1])) / (2 * h)
            # third-order term of the difference: h^2 / 6 times a third derivative of the order of the
            # sum's size; fp32 roundings of the outputs (2^-24 of each, divided by h) are far below it
            size = float((seed_out.abs().double().sum()))
            assert abs(diff - got) <= h * h * size, (diff, got)


def test_captured_calls_replay_with_eager_work_between():
    """Forward and gradients in a graph, replayed on changed inputs, each replay
    equal to the eager calls bit for bit; on a stream of their own."""
    m = Maps(64, 8, 32, 16)
    H = 256
    x = torch.empty(m.T, H, dtype=torch.bfloat16, device=DEV)
    w, d_w = torch.empty(m.T, m.K, device=DEV), torch.zeros(m.T, m.K, device=DEV)
    rows = torch.zeros(m.R, H, dtype=torch.bfloat16, device=DEV)
    d_rows, out, d_x = torch.zeros_like(rows), torch.zeros_like(x), torch.zeros_like(x)

    def step():
        N.moe_dispatch(x, *m.dev, rows)
        N.moe_combine(rows, m.dev[0], w, out)
        N.moe_combine_bwd(out, rows, *m.dev, w, d_rows, d_w)
        N.moe_dispatch_bwd(d_rows, m.dev[0], d_x)

    def load(seed):
        g = torch.Generator().manual_seed(seed)
        x.copy_(torch.randn(m.T, H, generator=g))
        w.copy_(torch.rand(m.T, m.K, generator=g))

    load(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(1, 5):
        load(seed)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (rows, out, d_rows, d_w, d_x)]
        step()
        torch.cuda.synchronize()
        for a, b in zip(got, (rows, out, d_rows, d_w, d_x)):
            assert torch.equal(a, b)


def test_binding_refusals():
    m = Maps(8, 2, 8, 16)
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device=DEV)
    rows, w = torch.zeros(m.R, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(8, 2, device=DEV)
    p, t, n = m.dev
    bad = [lambda: N.moe_dispatch(x.float(), p, t, n, rows), lambda: N.moe_dispatch(x, p, t[:-1], n, rows),
           lambda: N.moe_dispatch(x, p.long(), t, n, rows), lambda: N.moe_dispatch(x, p, t, m.bufs.meta[:2], rows),
           lambda: N.moe_dispatch(x[:, :4], p, t, n, rows[:, :4]), lambda: N.moe_dispatch(x.t(), p, t, n, rows),
           lambda: N.moe_dispatch_bwd(rows, p, x.float()), lambda: N.moe_dispatch_bwd(rows.half(), p, x),
           lambda: N.moe_combine(rows, p, w.double(), x), lambda: N.moe_combine(rows, p, w.t().contiguous(), x),
           lambda: N.moe_combine(rows, p, w.cpu(), x),
           lambda: N.moe_combine_bwd(x, rows, p, t, n, w, rows[:-1], w),
           lambda: N.moe_combine_bwd(x, rows, p, t, n, w, rows, w[:, :1])]
    for call in bad:
        with pytest.raises((ValueError, TypeError, N.MoeError)):
            call()
