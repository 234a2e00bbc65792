"""The router, row and few-token calls refuse bad arguments on the host, before
any device work (these calls return before touching HIP)."""

import ctypes
import os

import pytest
import torch

import fp4_grouped_gemm_amd as fgg

pytestmark = pytest.mark.skipif(not os.path.exists(fgg.library_path()),
                                reason="libfgg.so not built (run __graft_entry__.build())")

g = ctypes.c_void_p(4096)
odd = ctypes.c_void_p(4097)
F32, BF16 = fgg.FGG_F32, fgg.FGG_BF16
INVALID, UNSUPPORTED = 1, 2


def route(logits=g, dtype=F32, T=4, E=8, ld=8, k=2, gate=0, bias=None, renorm=0, scale=1.0, ids=g, w=g):
    return fgg.load_library().fgg_moe_route(logits, dtype, T, E, ld, k, gate, bias, renorm, scale, ids, w, None)


def route_bwd(logits=g, dtype=F32, T=4, E=8, ld=8, k=2, gate=0, renorm=0, scale=1.0, ids=g, dw=g, out=g, ldd=8):
    return fgg.load_library().fgg_moe_route_backward(logits, dtype, T, E, ld, k, gate, renorm, scale, ids, dw, out,
                                                     ldd, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(E=1025, ld=1025), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(E=128, ld=128, k=65), INVALID), (dict(ld=7), INVALID), (dict(gate=2), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID), (dict(dtype=fgg.FGG_E4M3), UNSUPPORTED),
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(logits=odd), INVALID),
    (dict(logits=odd, dtype=BF16), INVALID), (dict(ids=odd), INVALID), (dict(T=1 << 31), UNSUPPORTED),
])
def test_route_refuses(bad, status):
    assert route(**bad) == status
    assert route_bwd(**bad) == status


def test_route_refuses_more():
    assert route(w=None) == INVALID and route(bias=odd) == INVALID
    assert route_bwd(dw=None) == INVALID and route_bwd(out=None) == INVALID and route_bwd(ldd=7) == INVALID
    assert route(T=0, logits=None, ids=None, w=None) == 0
    assert route_bwd(T=0, logits=None, ids=None, dw=None, out=None) == 0


def permute(x=g, dtype=F32, T=4, k=2, N=8, ldx=8, w=None, s2r=g, r2s=g, off=g, E=3, M=32, rows=g, ldr=8):
    return fgg.load_library().fgg_moe_permute_rows(x, dtype, T, k, N, ldx, w, s2r, r2s, off, E, M, rows, ldr, None)


def permute_bwd(drows=g, dtype=F32, M=32, lddr=8, x=g, ldx=8, w=None, s2r=g, T=4, k=2, N=8, dx=g, lddx=8, dw=g):
    return fgg.load_library().fgg_moe_permute_rows_backward(drows, dtype, M, lddr, x, ldx, w, s2r, T, k, N, dx, lddx,
                                                            dw, None)


def unpermute(rows=g, dtype=F32, M=32, ldr=8, w=None, s2r=g, T=4, k=2, N=8, out=g, ldo=8):
    return fgg.load_library().fgg_moe_unpermute_rows(rows, dtype, M, ldr, w, s2r, T, k, N, out, ldo, None)


def unpermute_bwd(dout=g, dtype=F32, T=4, k=2, N=8, lddo=8, rows=g, ldr=8, w=None, s2r=g, r2s=g, off=g, E=3, M=32,
                  drows=g, lddr=8, dw=g):
    return fgg.load_library().fgg_moe_unpermute_rows_backward(dout, dtype, T, k, N, lddo, rows, ldr, w, s2r, r2s, off,
                                                              E, M, drows, lddr, dw, None)


@pytest.mark.parametrize("call", [permute, permute_bwd, unpermute, unpermute_bwd])
@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(N=0), INVALID), (dict(M=-1), INVALID),
    (dict(dtype=fgg.FGG_E4M3), UNSUPPORTED), (dict(s2r=None), INVALID), (dict(w=odd), INVALID),
    (dict(T=1 << 24), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED), (dict(M=1 << 28), UNSUPPORTED),
    (dict(T=1 << 26, k=64), UNSUPPORTED),
])
def test_rows_refuse(call, bad, status):
    assert call(**bad) == status


def test_rows_refuse_more():
    assert permute(ldx=7) == INVALID and permute(ldr=7) == INVALID and permute(x=None) == INVALID
    assert permute(rows=None) == INVALID and permute(r2s=None) == INVALID and permute(off=None) == INVALID
    assert permute(E=0) == INVALID and permute(E=1025) == INVALID and permute(x=odd, dtype=BF16) == INVALID
    assert permute_bwd(lddr=7) == INVALID and permute_bwd(lddx=7) == INVALID and permute_bwd(drows=None) == INVALID
    assert permute_bwd(x=None) == INVALID                       # dw needs the forward's input
    assert permute_bwd(ldx=7) == INVALID and permute_bwd(dx=None) == INVALID and permute_bwd(dw=odd) == INVALID
    assert unpermute(rows=None) == INVALID and unpermute(out=None) == INVALID and unpermute(ldo=7) == INVALID
    assert unpermute(ldr=7) == INVALID and unpermute(out=odd) == INVALID
    assert unpermute_bwd(rows=None) == INVALID and unpermute_bwd(ldr=7) == INVALID
    assert unpermute_bwd(dout=None) == INVALID and unpermute_bwd(drows=None) == INVALID
    assert unpermute_bwd(r2s=None) == INVALID and unpermute_bwd(off=None) == INVALID and unpermute_bwd(E=0) == INVALID
    # nothing to do
    assert permute(T=0, x=None) == 0 and permute(M=0, rows=None) == 0 and unpermute(T=0, out=None) == 0
    assert permute_bwd(T=0, dx=None) == 0 and unpermute_bwd(M=0, dw=None, drows=None) == 0


def gemv(G=3, T=4, k=2, N=32, K=128, x=g, xd=BF16, ldx=128, per=0, b=g, s=g, q=fgg.Q_E2M1_E8M0_1x32, ids=g, w=None,
         act=0, out=g, od=BF16, ldo=32):
    return fgg.load_library().fgg_moe_gemv_fp4(G, T, k, N, K, x, xd, ldx, per, b, s, fgg.QDesc(*q), ids, w, act, out,
                                               od, ldo, None)


@pytest.mark.parametrize("bad,status", [
    (dict(G=0), INVALID), (dict(G=1025), INVALID), (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID),
    (dict(N=-1), INVALID), (dict(K=-32), INVALID), (dict(ldx=127), INVALID), (dict(ldo=31), INVALID),
    (dict(act=2), INVALID), (dict(ids=None), INVALID), (dict(ids=None, G=1), INVALID),
    (dict(ids=None, G=1, k=1, w=g), INVALID), (dict(xd=fgg.FGG_E4M3), UNSUPPORTED), (dict(od=fgg.FGG_E8M0), UNSUPPORTED),
    (dict(w=g, act=1), UNSUPPORTED), (dict(q=fgg.Q_E2M1_1x16), UNSUPPORTED), (dict(q=fgg.Q_E4M3_128x128), UNSUPPORTED),
    (dict(K=0), UNSUPPORTED), (dict(K=112), UNSUPPORTED), (dict(K=96, q=fgg.Q_E2M1_E8M0_1x32_TILED), UNSUPPORTED),
    (dict(N=24, q=fgg.Q_E2M1_E8M0_1x32_TILED), UNSUPPORTED), (dict(T=1 << 21), UNSUPPORTED), (dict(x=None), INVALID),
    (dict(b=None), INVALID), (dict(s=None), INVALID), (dict(out=None), INVALID), (dict(x=odd), INVALID),
    (dict(b=ctypes.c_void_p(4104)), INVALID), (dict(out=odd), INVALID), (dict(ids=odd), INVALID), (dict(w=odd), INVALID),
    (dict(s=ctypes.c_void_p(4104), q=fgg.Q_E2M1_E8M0_1x32_TILED), INVALID),
])
def test_gemv_refuses(bad, status):
    assert gemv(**bad) == status


def test_gemv_nothing_to_do():
    assert gemv(T=0, x=None) == 0 and gemv(N=0, out=None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(AssertionError):
        fgg.moe_route(x, 2)
    with pytest.raises(AssertionError):
        fgg.moe_permute_rows(x, torch.zeros(8, dtype=torch.int32), torch.zeros(8, dtype=torch.int32),
                             torch.zeros(3, dtype=torch.int32))
    with pytest.raises(AssertionError):
        fgg.moe_gemv_fp4(x, torch.zeros(1, 4, 4, dtype=torch.uint8), torch.zeros(1, 4, 1, dtype=torch.uint8))
