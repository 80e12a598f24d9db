"""moe_swiglu and its gradient against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N
from oracle import grouped as G

from .gpu_common import DEV, dev, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
LEFT = 7.25


def _maps(R, total, seed):
    rng = np.random.default_rng(seed)
    tok = np.where(rng.random(R) < 0.7, rng.integers(0, 50, R), -1).astype(np.int32)
    tok[total:] = -1
    return tok, dev(tok), dev(np.array([total], np.int32))


def _run(gate_up, tok, total, dt, d=None, pad=0, inplace=False):
    """gate_up, d: fp32 arrays; NaN goes into rows that may not be read."""
    R, I = gate_up.shape[0], gate_up.shape[1] // 2
    held = tok >= 0

    def matrix(v):
        wide = np.full((R, v.shape[1] + pad), np.nan, np.float32)
        wide[held, :v.shape[1]] = v[held]
        t = torch.from_numpy(wide).to(DT[dt]).to(DEV)[:, :v.shape[1]]
        return t, t.double().cpu().numpy()

    g, gv = matrix(gate_up)
    say(f"swiglu R={R} I={I} total={total} {dt} pad={pad} grad={d is not None} inplace={inplace}")
    maps = dev(tok), dev(np.array([total], np.int32))
    if d is None:
        out = torch.full((R, I + pad), LEFT, dtype=DT[dt], device=DEV)[:, :I]
        N.moe_swiglu(g, *maps, out)
        ref = G.swiglu(gv)
    else:
        dd, dv = matrix(d)
        out = g if inplace else torch.full((R, 2 * I + pad), LEFT, dtype=DT[dt], device=DEV)[:, :2 * I]
        N.moe_swiglu_bwd(dd, g, *maps, out)
        ref = G.swiglu_grad(dv, gv)
    torch.cuda.synchronize()
    got = out.double().cpu().numpy()
    # exp is off by at most 2 steps of fp32, and there are at most 7 more fp32 roundings of
    # factors; the two terms of the gate's gradient may cancel: of their magnitudes
    mags = np.abs(ref)
    if d is not None:
        gg, u = np.split(gv, 2, axis=1)
        s, rest = G.sigmoid(gg), G.sigmoid(-gg)
        mags = np.concatenate([np.abs(dv * u) * (s + np.abs(gg) * s * rest), mags[:, I:]], axis=1)
    # below fp32's normal numbers roundings are absolute: of the sigmoid, 2^-149, times the other factors
    tiny = 2.0 ** -140 * (1 + np.abs(np.nan_to_num(gv)).max()) ** 2 * (1 if d is None else 1 + np.abs(np.nan_to_num(dv)).max())
    err = 11 * 2.0 ** -24 * mags + tiny
    tol = err + HALF[dt] * (np.abs(ref) + err) + 2.0 ** -134
    assert (np.abs(got[held] - ref[held]) <= tol[held]).all(), np.argwhere(~(np.abs(got[held] - ref[held]) <= tol[held]))[:3]
    assert (got[:total][~held[:total]] == 0).all()
    behind = got[total:]
    assert np.isnan(behind).all() if inplace else (behind == LEFT).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("R,total,I,pad", [(1, 1, 8, 0), (3, 2, 8, 8), (16, 16, 24, 0), (100, 64, 136, 16), (37, 37, 4096, 0),
                                           (1025, 1000, 40, 8), (5, 0, 16, 0), (20, 20, 16384, 0)])
def test_shapes(R, total, I, pad, dt):
    rng = np.random.default_rng(R + I)
    tok, _, _ = _maps(R, total, I)
    x = (3 * rng.standard_normal((R, 2 * I))).astype(np.float32)
    d = rng.standard_normal((R, I)).astype(np.float32)
    _run(x, tok, total, dt, None, pad)
    _run(x, tok, total, dt, d, pad)
    _run(x, tok, total, dt, d, pad, inplace=True)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_gates_of_every_size(dt):
    """From where the sigmoid is 1 to where it underflows, both signs."""
    g = np.concatenate([np.linspace(-110, 110, 2008), [0.0, -0.0, 1e-30, -1e-30, 1e4, -1e4, 3e38, -3e38]]).astype(np.float32)
    x = np.stack([np.concatenate([g, np.ones_like(g)]), np.concatenate([g, np.full_like(g, -2.5)])])
    d = np.stack([np.ones_like(g), np.full_like(g, 0.75)])
    tok = np.array([0, 1], np.int32)
    x = np.where(np.abs(x) > 1e30, np.sign(x) * 1e30, x)        # products stay finite
    for dd in (None, d):
        wide = np.abs(x[:, :len(g)]) > 1e3
        xx = x.copy()
        xx[:, :len(g)][wide] = np.sign(xx[:, :len(g)][wide]) * 200.0
        _run(xx, tok, 2, dt, dd)


def test_huge_and_infinite_values():
    """A gate far below 0 gives 0 whatever stands beside it; one far above passes the
    other half; NaN and infinite gates give NaN or infinity in their own place alone."""
    g = torch.tensor([[-1e30, 1e30, float("inf"), float("nan"), 1.0, 1.0, -float("inf"), 2.0] + [2.0] * 8], device=DEV)
    out = torch.empty((1, 8), device=DEV)
    maps = dev(np.array([0], np.int32)), dev(np.array([1], np.int32))
    N.moe_swiglu(g, *maps, out)
    got = out.cpu().numpy()[0]
    assert got[0] == 0 and got[1] == np.float32(2e30) and got[2] == np.inf and np.isnan(got[3]) and np.isnan(got[6])
    assert abs(got[4] - 2 / (1 + np.exp(-1))) < 1e-6 and np.isfinite(got[7])


def test_gradient_against_differences():
    """Central differences of the oracle's formula, in 64 bits: off by h^2 of the third
    derivative (below 1) and by 2^-52 / h of the values."""
    rng = np.random.default_rng(5)
    x, d, v = (rng.standard_normal((4, c)) for c in (32, 16, 32))
    h = 2.0 ** -17
    slope = ((G.swiglu(x + h * v) - G.swiglu(x - h * v)) * d).sum() / (2 * h)
    assert abs(slope - (G.swiglu_grad(d, x) * v).sum()) <= 64 * (h * h * 27 + 2.0 ** -50 / h)
