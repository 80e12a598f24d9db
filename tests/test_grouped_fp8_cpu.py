"""Refusals of the grouped products, the gated activation and the 8-bit products, by
the library (fake aligned addresses, never dereferenced: every call here returns
before a launch) and by the binding."""
import pytest
import torch

from nvfp4_block_scaled_route_amd import layer as LY
from nvfp4_block_scaled_route_amd import native as N

P = 4096        # an aligned address no call reads


def grouped(x=P, ldx=64, w=P, off=P, cnt=P, R=64, E=4, Nn=48, D=64, out=P, ldo=48, dt=N.MOE_BF16):
    return N.lib().moe_grouped_gemm(x, ldx, w, off, cnt, R, E, Nn, D, out, ldo, dt, None)


def dgrad(d=P, ldd=48, w=P, off=P, cnt=P, R=64, E=4, Nn=48, D=64, dx=P, ldx=64, dt=N.MOE_BF16):
    return N.lib().moe_grouped_gemm_dgrad(d, ldd, w, off, cnt, R, E, Nn, D, dx, ldx, dt, None)


def wgrad(d=P, ldd=48, x=P, ldx=64, off=P, cnt=P, R=64, E=4, Nn=48, D=64, acc=0, dw=P, dt=N.MOE_F32):
    return N.lib().moe_grouped_gemm_wgrad(d, ldd, x, ldx, off, cnt, R, E, Nn, D, acc, dw, dt, None)


def swiglu(g=P, ldg=64, dt=N.MOE_BF16, p2t=P, tot=P, R=64, I=32, y=P, ldy=32):
    return N.lib().moe_swiglu(g, ldg, dt, p2t, tot, R, I, y, ldy, None)


def swiglu_bwd(d=P, ldd=32, g=P, ldg=64, dt=N.MOE_BF16, p2t=P, tot=P, R=64, I=32, dg=2 * P, lddg=64):
    return N.lib().moe_swiglu_bwd(d, ldd, g, ldg, dt, p2t, tot, R, I, dg, lddg, None)


def quant(x=P, ld=64, T=4, H=64, codes=P, sf=P, lds=4):
    return N.lib().fp8_quant(x, ld, T, H, codes, sf, lds, None)


def quant_weight(w=P, ld=64, Nn=20, K=64, codes=P, sf=P, ct=P, ldt=32, st=P):
    return N.lib().fp8_quant_weight(w, ld, Nn, K, codes, sf, ct, ldt, st, None)


def gemm(a=P, asf=P, lds=4, w=P, ldw=64, wsf=P, T=4, Nn=48, K=64, out=P, ldo=48):
    return N.lib().fp8_gemm(a, asf, lds, w, ldw, wsf, T, Nn, K, out, ldo, None)


CASES = [
    (grouped, N.MOE_EINVAL, [dict(R=-1), dict(R=1 << 31), dict(E=0), dict(E=1025), dict(Nn=-8), dict(D=-8), dict(dt=2), dict(x=0),
                             dict(w=0), dict(off=0), dict(cnt=0), dict(out=0), dict(x=P + 8), dict(w=P + 2), dict(off=P + 4),
                             dict(cnt=P + 8), dict(out=P + 4), dict(ldx=56), dict(ldx=68), dict(ldx=(1 << 21) + 8), dict(ldo=47)]),
    (grouped, N.MOE_EUNSUPPORTED, [dict(Nn=44), dict(D=60), dict(Nn=32776, ldo=32776), dict(D=32776, ldx=32776)]),
    (dgrad, N.MOE_EINVAL, [dict(R=-1), dict(E=-4), dict(dt=-1), dict(d=0), dict(w=0), dict(off=0), dict(cnt=0), dict(dx=0),
                           dict(d=P + 4), dict(dx=P + 2), dict(ldd=40), dict(ldd=50), dict(ldx=63)]),
    (dgrad, N.MOE_EUNSUPPORTED, [dict(Nn=50), dict(D=4)]),
    (wgrad, N.MOE_EINVAL, [dict(R=-1), dict(E=0), dict(dt=3), dict(d=0), dict(x=0), dict(off=0), dict(cnt=0), dict(dw=0),
                           dict(d=P + 8), dict(x=P + 1), dict(dw=P + 4), dict(ldd=40), dict(ldx=68), dict(ldx=56)]),
    (wgrad, N.MOE_EUNSUPPORTED, [dict(Nn=2), dict(D=63)]),
    (swiglu, N.MOE_EINVAL, [dict(R=-1), dict(R=1 << 31), dict(I=-8), dict(dt=7), dict(g=0), dict(p2t=0), dict(tot=0), dict(y=0),
                            dict(g=P + 8), dict(p2t=P + 4), dict(tot=P + 2), dict(y=P + 8), dict(ldg=56), dict(ldg=68), dict(ldy=24)]),
    (swiglu, N.MOE_EUNSUPPORTED, [dict(I=12), dict(I=16392, ldg=1 << 16, ldy=1 << 15)]),
    (swiglu_bwd, N.MOE_EINVAL, [dict(R=-1), dict(dt=-2), dict(d=0), dict(g=0), dict(p2t=0), dict(tot=0), dict(dg=0), dict(d=P + 4),
                                dict(dg=P + 8), dict(ldd=24), dict(ldd=36), dict(lddg=32), dict(ldg=60), dict(dg=P, lddg=128)]),
    (swiglu_bwd, N.MOE_EUNSUPPORTED, [dict(I=20)]),
    (quant, N.MOE_EINVAL, [dict(T=-1), dict(H=-16), dict(x=0), dict(codes=0), dict(sf=0), dict(x=P + 2), dict(codes=P + 8),
                           dict(sf=P + 4), dict(ld=56), dict(ld=68), dict(lds=3)]),
    (quant, N.MOE_EUNSUPPORTED, [dict(H=56), dict(H=8)]),
    (quant_weight, N.MOE_EINVAL, [dict(Nn=-1), dict(K=-16), dict(w=0), dict(codes=0), dict(sf=0), dict(ct=0), dict(st=0),
                                  dict(w=P + 8), dict(sf=P + 4), dict(ct=P + 8), dict(st=P + 4), dict(ld=60), dict(ldt=16),
                                  dict(ldt=40)]),
    (quant_weight, N.MOE_EUNSUPPORTED, [dict(K=40)]),
    (gemm, N.MOE_EINVAL, [dict(T=-1), dict(Nn=-1), dict(K=-16), dict(a=0), dict(asf=0), dict(w=0), dict(wsf=0), dict(out=0),
                          dict(a=P + 8), dict(asf=P + 4), dict(w=P + 8), dict(wsf=P + 2), dict(out=P + 8), dict(lds=3), dict(ldw=48),
                          dict(ldw=72), dict(ldw=(1 << 22) + 16), dict(ldo=47)]),
    (gemm, N.MOE_EUNSUPPORTED, [dict(K=0), dict(K=24), dict(K=(1 << 20) + 16)]),
]


@pytest.mark.parametrize("call,want,kw", [(c, w, k) for c, w, ks in CASES for k in ks],
                         ids=lambda v: v.__name__ if callable(v) else str(v))
def test_library_refuses(call, want, kw):
    assert call(**kw) == want, N.lib().moe_last_error()
    assert N.lib().moe_last_error()


@pytest.mark.parametrize("call,kw", [
    (grouped, dict(R=(1 << 31) - 1, Nn=32768, ldo=32768)), (dgrad, dict(R=(1 << 31) - 1, D=32768, ldx=32768)),
    (wgrad, dict(E=1024, Nn=32768, ldd=32768, D=32768, ldx=32768)), (swiglu, dict(R=(1 << 31) - 1, I=16384, ldg=1 << 16, ldy=1 << 16)),
    (quant, dict(T=(1 << 31) - 1, H=1 << 20, ld=1 << 20, lds=1 << 31)),
    (quant_weight, dict(Nn=(1 << 31) - 1, K=(1 << 31) - 16, ld=1 << 32, ct=None, st=None)),
    (gemm, dict(T=(1 << 31) - 1, Nn=(1 << 31) - 1, lds=1 << 31, ldo=1 << 31))])
def test_library_refuses_more_threads_than_a_launch_counts(call, kw):
    assert call(**kw) == N.MOE_EUNSUPPORTED, N.lib().moe_last_error()


BIG = 0x7FFFF001     # one more than a side may have


@pytest.mark.parametrize("call,kw", [
    (grouped, dict(R=BIG, Nn=8, D=8)), (dgrad, dict(R=BIG, Nn=8, D=8)), (wgrad, dict(R=BIG, Nn=8, D=8)),
    (quant, dict(T=BIG, H=16, lds=1 << 31)), (quant, dict(T=1, H=BIG + 15, ld=1 << 31)),
    (quant_weight, dict(Nn=BIG, K=16, ct=None, st=None)), (quant_weight, dict(Nn=1, K=BIG + 15, ld=1 << 31)),
    (gemm, dict(T=BIG, Nn=1, K=16, lds=1 << 31)), (gemm, dict(T=1, Nn=BIG, K=16, ldo=1 << 31))])
def test_library_refuses_sides_whose_last_block_leaves_31_bits(call, kw):
    assert call(**kw) == N.MOE_EUNSUPPORTED, N.lib().moe_last_error()
    assert b"more than" in N.lib().moe_last_error()


@pytest.mark.parametrize("call,kw", [
    (grouped, dict(R=0, x=0)), (grouped, dict(Nn=0, w=0)), (dgrad, dict(R=0, d=0)), (dgrad, dict(D=0)), (wgrad, dict(Nn=0, dw=0)),
    (wgrad, dict(D=0)), (swiglu, dict(R=0, g=0)), (swiglu, dict(I=0)), (swiglu_bwd, dict(R=0)), (quant, dict(T=0, x=0)),
    (quant, dict(H=0, ld=0)), (quant_weight, dict(Nn=0)), (quant_weight, dict(K=0)), (gemm, dict(T=0, a=0)), (gemm, dict(Nn=0, w=0))])
def test_empty_calls_launch_nothing(call, kw):
    assert call(**kw) == N.MOE_OK, N.lib().moe_last_error()


def test_transposed_outputs_go_together():
    assert quant_weight(ct=None) == N.MOE_EINVAL and quant_weight(st=None) == N.MOE_EINVAL


def test_binding_refuses_before_the_library():
    """Types and shapes first, then the device: a host tensor never reaches a launch."""
    b, i = torch.bfloat16, torch.int32
    x, w, out = torch.zeros(8, 64, dtype=b), torch.zeros(2, 48, 64, dtype=b), torch.zeros(8, 48, dtype=b)
    off, cnt = torch.zeros(3, dtype=i), torch.zeros(2, dtype=i)
    with pytest.raises(ValueError, match="device"):
        N.moe_grouped_gemm(x, w, off, cnt, out)
    with pytest.raises(TypeError):
        N.moe_grouped_gemm(x.float(), w, off, cnt, out)
    with pytest.raises(ValueError, match="three dimensions"):
        N.moe_grouped_gemm(x, w[0], off, cnt, out)
    with pytest.raises(ValueError, match="d_out"):
        N.moe_grouped_gemm_dgrad(x, w, off, cnt, x)         # rows of D, not N
    with pytest.raises(ValueError, match="three dimensions"):
        N.moe_grouped_gemm_wgrad(out, x, off, cnt, w[0])
    with pytest.raises(ValueError, match="device"):
        N.moe_grouped_gemm_wgrad(out, x, off, cnt, w)
    tok, tot = torch.zeros(8, dtype=i), torch.zeros(1, dtype=i)
    with pytest.raises(ValueError, match="device"):
        N.moe_swiglu(x, tok, tot, torch.zeros(8, 32, dtype=b))
    with pytest.raises(TypeError):
        N.moe_swiglu(x, tok, tot, torch.zeros(8, 32, dtype=torch.float16))
    with pytest.raises(ValueError):
        N.moe_swiglu_bwd(torch.zeros(8, 32, dtype=b), torch.zeros(8, 48, dtype=b), tok, tot, x)
    c = torch.zeros(8, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        N.fp8_quant(x, c, torch.zeros(1, 8))
    with pytest.raises(ValueError):
        N.fp8_gemm(c, torch.zeros(1, 8), c[:, :48], torch.zeros(1, 1), torch.zeros(8, 8, dtype=b))
    with pytest.raises(ValueError, match="dimensions"):
        N.fp8_quant_weight(x[0], c, torch.zeros(1, 1))


def test_projections_without_a_product_are_refused_when_made():
    with pytest.raises(N.MoeError):
        LY.Fp8Linear(torch.zeros(16, 24, dtype=torch.bfloat16), 4)
    with pytest.raises(N.MoeError):
        LY.Fp8Linear(torch.zeros(24, 16, dtype=torch.bfloat16), 4, grads=True)
    with pytest.raises(N.MoeError):
        N.fp8_gemm_validate(1 << 31, 16)
    N.fp8_gemm_validate(24, 16)
