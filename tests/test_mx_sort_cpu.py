"""Refusals of the MX and sort calls, by the library (fake aligned addresses,
never dereferenced: every call here returns before a launch) and by the binding."""
import ctypes

import pytest
import torch

from nvfp4_block_scaled_route_amd import native as N

f = ctypes.c_float
P = 4096        # an aligned address no call reads


def quant(x=P, ld=64, T=4, H=64, fmt=N.MOE_MX_E4M3, codes=P, sf=P):
    return N.lib().mx_quant(x, ld, T, H, fmt, codes, sf, None)


def dequant(codes=P, sf=P, T=4, H=64, fmt=N.MOE_MX_E4M3, out=P, ld=64):
    return N.lib().mx_dequant(codes, sf, T, H, fmt, out, ld, None)


def norm(x=P, ld=64, res=P, ldr=64, w=P, gain=1.0, eps=1e-6, T=4, H=64, fmt=N.MOE_MX_E4M3, out=2 * P, ldo=64, codes=P,
         sf=P):
    return N.lib().mx_add_norm_quant(x, ld, res, ldr, w, f(gain), f(eps), T, H, fmt, out, ldo, codes, sf, None)


def gemm(a=P, asf=P, af=N.MOE_MX_E4M3, w=P, wsf=P, wf=N.MOE_MX_E2M1, T=4, Nn=48, K=64, out=P, ld=48, dt=N.MOE_BF16):
    return N.lib().mx_gemm(a, asf, af, w, wsf, wf, T, Nn, K, out, ld, dt, None)


def dispatch(x=P, ldx=64, nb=64, e2p=P, p2t=P, tot=P, T=4, K=2, R=64, rows=P, ldr=64):
    return N.lib().moe_dispatch(x, ldx, nb, e2p, p2t, tot, T, K, R, rows, ldr, None)


def dispatch_bwd(rows=P, ldr=64, dt=N.MOE_BF16, e2p=P, T=4, K=2, R=64, H=64, dx=P, ldx=64):
    return N.lib().moe_dispatch_bwd(rows, ldr, dt, e2p, T, K, R, H, dx, ldx, None)


def combine(rows=P, ldr=64, dt=N.MOE_BF16, e2p=P, w=P, T=4, K=2, R=64, H=64, out=P, ldo=64):
    return N.lib().moe_combine(rows, ldr, dt, e2p, w, T, K, R, H, out, ldo, None)


def combine_bwd(do=P, ldo=64, rows=P, ldr=64, dt=N.MOE_BF16, e2p=P, p2t=P, tot=P, w=P, T=4, K=2, R=64, H=64, dr=2 * P,
                ldd=64, dw=P):
    return N.lib().moe_combine_bwd(do, ldo, rows, ldr, dt, e2p, p2t, tot, w, T, K, R, H, dr, ldd, dw, None)


CASES = [
    (quant, N.MOE_EINVAL, [dict(T=-1), dict(fmt=2), dict(fmt=-1), dict(x=0), dict(codes=0), dict(sf=0), dict(x=P + 8),
                           dict(sf=P + 1), dict(ld=56), dict(ld=68)]),
    (quant, N.MOE_EUNSUPPORTED, [dict(H=48, ld=48), dict(H=16)]),
    (dequant, N.MOE_EINVAL, [dict(H=-32), dict(fmt=7), dict(codes=0), dict(sf=0), dict(out=0), dict(out=P + 2),
                             dict(ld=32), dict(ld=65)]),
    (dequant, N.MOE_EUNSUPPORTED, [dict(H=33)]),
    (norm, N.MOE_EINVAL, [dict(T=-2), dict(fmt=9), dict(x=0), dict(codes=0), dict(sf=0), dict(out=0), dict(eps=0.0),
                          dict(eps=2.0), dict(eps=float("nan")), dict(gain=float("nan")), dict(res=P + 4),
                          dict(out=P + 6), dict(w=P + 8), dict(ldr=60), dict(ldo=32), dict(ld=63),
                          dict(out=P, res=P, ldr=128), dict(out=P, x=P, res=3 * P, ld=72)]),
    (norm, N.MOE_EUNSUPPORTED, [dict(H=40, ld=64), dict(H=16384 + 32, ld=32768)]),
    (gemm, N.MOE_EINVAL, [dict(T=-1), dict(Nn=-1), dict(K=-32), dict(af=3), dict(wf=-2), dict(dt=4), dict(a=0), dict(asf=0),
                          dict(w=0), dict(wsf=0), dict(out=0), dict(a=P + 8), dict(wsf=P + 4), dict(out=P + 2), dict(ld=47)]),
    (gemm, N.MOE_EUNSUPPORTED, [dict(K=0), dict(K=48), dict(K=(1 << 20) + 32), dict(af=N.MOE_MX_E2M1, wf=N.MOE_MX_E4M3),
                                dict(dt=N.MOE_F32), dict(wf=N.MOE_MX_E4M3, dt=N.MOE_F32)]),
    (dispatch, N.MOE_EINVAL, [dict(T=-1), dict(K=0), dict(K=33), dict(R=-1), dict(R=1 << 31), dict(x=0), dict(e2p=0),
                              dict(p2t=0), dict(tot=0), dict(rows=0), dict(x=P + 8), dict(tot=P + 2), dict(ldx=48),
                              dict(ldr=72)]),
    (dispatch, N.MOE_EUNSUPPORTED, [dict(nb=24), dict(nb=-16), dict(nb=4 * 16384 + 16, ldx=1 << 17, ldr=1 << 17),
                                    dict(T=1 << 30, K=32)]),
    (dispatch_bwd, N.MOE_EINVAL, [dict(T=-1), dict(K=0), dict(dt=2), dict(H=-8), dict(rows=0), dict(e2p=0), dict(dx=0),
                                  dict(dx=P + 8), dict(ldr=56), dict(ldx=68)]),
    (dispatch_bwd, N.MOE_EUNSUPPORTED, [dict(H=60), dict(H=16392, ldr=16392, ldx=16392)]),
    (combine, N.MOE_EINVAL, [dict(T=-1), dict(K=40), dict(dt=-1), dict(w=0), dict(rows=0), dict(out=0), dict(w=P + 4),
                             dict(ldo=56)]),
    (combine, N.MOE_EUNSUPPORTED, [dict(H=4)]),
    (combine_bwd, N.MOE_EINVAL, [dict(T=-1), dict(K=0), dict(dt=5), dict(do=0), dict(rows=0), dict(e2p=0), dict(p2t=0),
                                 dict(tot=0), dict(w=0), dict(dr=0), dict(dw=0), dict(tot=P + 1), dict(dw=P + 4),
                                 dict(ldo=32), dict(ldr=60), dict(ldd=4), dict(dr=P, rows=P, ldd=128)]),
    (combine_bwd, N.MOE_EUNSUPPORTED, [dict(H=12)]),
]


@pytest.mark.parametrize("call,want,kw", [(c, w, k) for c, w, ks in CASES for k in ks],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_library_refuses(call, want, kw):
    assert call(**kw) == want, N.lib().moe_last_error()
    assert N.lib().moe_last_error()


@pytest.mark.parametrize("call,kw", [
    (quant, dict(T=1 << 30, H=64)), (dequant, dict(T=1 << 30, H=64)), (norm, dict(T=1 << 23)), (gemm, dict(T=1, Nn=2 ** 31 - 1, ld=2 ** 31 - 1)),
    (gemm, dict(T=1 << 20, Nn=1 << 20, ld=1 << 20)), (dispatch, dict(T=1 << 24, K=8)), (dispatch_bwd, dict(T=1 << 27)),
    (combine, dict(T=1 << 25)), (combine_bwd, dict(T=1 << 26, K=1)),
    (combine_bwd, dict(T=1 << 22, K=1, H=16384, ldo=16384, ldr=16384, ldd=16384))])
def test_library_refuses_more_threads_than_a_launch_counts(call, kw):
    assert call(**kw) == N.MOE_EUNSUPPORTED, N.lib().moe_last_error()


@pytest.mark.parametrize("call,kw", [(quant, dict(T=0, x=0)), (quant, dict(H=0, x=0, ld=0)), (dequant, dict(T=0)),
                                     (norm, dict(T=0, x=0)), (gemm, dict(T=0, a=0)), (gemm, dict(Nn=0, w=0)),
                                     (dispatch, dict(T=0, x=0)), (dispatch, dict(nb=0)), (dispatch_bwd, dict(T=0)),
                                     (combine, dict(T=0)), (combine_bwd, dict(T=0)), (combine_bwd, dict(H=0))])
def test_empty_calls_launch_nothing(call, kw):
    assert call(**kw) == N.MOE_OK, N.lib().moe_last_error()


def test_binding_refuses_before_the_library():
    """Types and shapes first, then the device: a host tensor never reaches a launch."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c, s = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)
    fmt = N.MOE_MX_E4M3
    with pytest.raises(ValueError, match="device"):
        N.mx_quant(x, fmt, c, s)
    with pytest.raises(TypeError):
        N.mx_quant(x.float(), fmt, c, s)
    with pytest.raises(ValueError, match="dimensions"):
        N.mx_quant(x[0], fmt, c, s)
    with pytest.raises(TypeError):
        N.moe_combine(x.half(), torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, 2), x)
    with pytest.raises(ValueError):
        N.moe_dispatch(x, torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32),
                       torch.zeros(1, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        N.mx_gemm(c, s, fmt, c, s, fmt, x[0])
