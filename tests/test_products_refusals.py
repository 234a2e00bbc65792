"""The bf16 products and the adapters refuse bad arguments on the host, before any device work."""

import ctypes
import os

import pytest
import torch

import fp4_grouped_gemm_amd as fgg

pytestmark = pytest.mark.skipif(not os.path.exists(fgg.library_path()),
                                reason="libfgg.so not built (run __graft_entry__.build())")

g = ctypes.c_void_p(4096)
off16 = ctypes.c_void_p(4104)
odd = ctypes.c_void_p(4098)
F32, BF16, E4M3 = fgg.FGG_F32, fgg.FGG_BF16, fgg.FGG_E4M3
INVALID, UNSUPPORTED = 1, 2
WIDE = 1 << 22


def linear(G=3, M=40, N=32, K=16, x=g, ldx=16, w=g, off=g, cnt=None, y=g, dt=BF16, ldy=32):
    return fgg.load_library().fgg_grouped_linear(G, M, N, K, x, ldx, w, off, cnt, y, dt, ldy, None)


def dx(G=3, M=40, N=32, K=16, dy=g, lddy=32, w=g, off=g, cnt=None, out=g, dt=BF16, ldd=16):
    return fgg.load_library().fgg_grouped_linear_backward_input(G, M, N, K, dy, lddy, w, off, cnt, out, dt, ldd, None)


def dw(G=3, M=40, N=32, K=16, dy=g, lddy=32, x=g, ldx=16, off=g, cnt=None, out=g, dt=BF16, acc=0, ws=g, nb=1 << 30):
    return fgg.load_library().fgg_grouped_linear_backward_weight(G, M, N, K, dy, lddy, x, ldx, off, cnt, out, dt, acc,
                                                                 ws, nb, None)


def gated(G=3, M=40, N=32, K=16, x=g, ldx=16, w=g, off=g, cnt=None, a=g, lda=32, h=None, ldh=0):
    return fgg.load_library().fgg_grouped_gated(G, M, N, K, x, ldx, w, off, cnt, a, lda, h, ldh, None)


def gated_bwd(G=3, M=40, N=32, K=16, dy=g, lddy=16, wd=g, h=g, ldh=64, off=g, cnt=None, dh=g, lddh=64, a=None, lda=0):
    return fgg.load_library().fgg_grouped_gated_backward(G, M, N, K, dy, lddy, wd, h, ldh, off, cnt, dh, lddh, a, lda,
                                                         None)


@pytest.mark.parametrize("call", [linear, dx, dw, gated, gated_bwd])
@pytest.mark.parametrize("bad,status", [
    (dict(G=0), INVALID), (dict(G=1025), INVALID), (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=-8), INVALID),
    (dict(off=None), INVALID), (dict(off=None, G=1, cnt=g), INVALID), (dict(off=odd), INVALID), (dict(cnt=odd), INVALID),
    (dict(N=0), UNSUPPORTED), (dict(K=0), UNSUPPORTED), (dict(N=28), UNSUPPORTED), (dict(K=12), UNSUPPORTED),
    (dict(N=WIDE), UNSUPPORTED), (dict(K=WIDE), UNSUPPORTED), (dict(M=1 << 31), UNSUPPORTED),
])
def test_shapes(call, bad, status):
    assert call(**bad) == status


@pytest.mark.parametrize("call,pointers,strides", [
    (linear, ("x", "w", "y"), ("ldx", "ldy")), (dx, ("dy", "w", "out"), ("lddy", "ldd")),
    (dw, ("dy", "x", "out"), ("lddy", "ldx")), (gated, ("x", "w", "a"), ("ldx", "lda")),
    (gated_bwd, ("dy", "wd", "h", "dh"), ("lddy", "ldh", "lddh"))])
def test_pointers_and_strides(call, pointers, strides):
    for p in pointers:
        assert call(**{p: None}) == INVALID and call(**{p: off16}) == INVALID
    for ld in strides:
        assert call(**{ld: 8}) == INVALID                 # shorter than the row
        assert call(**{ld: 68}) == INVALID                # not whole 16-byte pieces
        assert call(**{ld: WIDE}) == UNSUPPORTED
    if call is not dw:                                    # (dw writes zeros without rows)
        assert call(M=0, **{pointers[0]: None}) == 0


def test_types_and_options():
    for call in (linear, dx, dw):
        assert call(dt=E4M3) == UNSUPPORTED
    assert gated(h=off16, ldh=64) == INVALID and gated(h=g, ldh=56) == INVALID
    assert gated_bwd(a=off16, lda=32) == INVALID and gated_bwd(a=g, lda=24) == INVALID
    assert linear(M=1 << 30, N=WIDE - 8, ldy=WIDE - 8) == UNSUPPORTED        # more tiles than a grid holds
    n = ctypes.c_size_t(0)
    ws = fgg.load_library().fgg_grouped_linear_backward_weight_workspace
    assert ws(1, 64, 32, 16, None) == INVALID and ws(0, 64, 32, 16, ctypes.byref(n)) == INVALID
    assert ws(1, 64, 32, 16, ctypes.byref(n)) == 0


def lora(T=5, L=3, r=16, N=32, K=48, x=g, ldx=48, ids=g, a=g, b=g, s=None, base=g, ldb=32, out=ctypes.c_void_p(8192),
         dt=BF16, ldo=32, ws=g, nb=1 << 30):
    return fgg.load_library().fgg_lora_add(T, L, r, N, K, x, ldx, ids, a, b, s, base, ldb, out, dt, ldo, ws, nb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(T=-1), INVALID), (dict(L=0), INVALID), (dict(r=0), INVALID), (dict(N=-8), INVALID), (dict(K=-8), INVALID),
    (dict(N=0), UNSUPPORTED), (dict(K=0), UNSUPPORTED), (dict(r=12), UNSUPPORTED), (dict(r=136), UNSUPPORTED),
    (dict(N=36), UNSUPPORTED), (dict(K=44), UNSUPPORTED), (dict(N=(1 << 20) + 8), UNSUPPORTED),
    (dict(K=(1 << 20) + 8), UNSUPPORTED), (dict(T=(1 << 26) + 1), UNSUPPORTED), (dict(dt=E4M3), UNSUPPORTED),
    (dict(ldx=40), INVALID), (dict(ldx=52), INVALID), (dict(ldb=24), INVALID), (dict(ldo=24), INVALID),
    (dict(ldo=36), INVALID), (dict(x=None), INVALID), (dict(ids=None), INVALID), (dict(a=None), INVALID),
    (dict(b=None), INVALID), (dict(base=None), INVALID), (dict(out=None), INVALID),
    (dict(x=off16), INVALID), (dict(a=off16), INVALID), (dict(b=off16), INVALID), (dict(base=off16), INVALID),
    (dict(out=off16), INVALID), (dict(ids=odd), INVALID), (dict(s=odd), INVALID), (dict(ws=off16), INVALID),
    (dict(out=g, ldo=40), INVALID),
])
def test_lora(bad, status):
    assert lora(**bad) == status


MANY = dict(T=2000, r=64, N=1024, K=4096, ldx=4096, ldb=1024, ldo=1024)


@pytest.mark.parametrize("bad", [dict(ws=None), dict(nb=0), dict(ws=off16), dict(nb=2000 * 64 * 4 - 1)])
def test_lora_of_many_tokens_needs_its_workspace(bad):
    assert lora(**MANY, **bad) == INVALID


def test_lora_nothing_to_do():
    assert lora(T=0, x=None, ws=None) == 0
    n = ctypes.c_size_t(1)
    ws = fgg.load_library().fgg_lora_workspace
    assert ws(0, 3, 16, 32, 48, ctypes.byref(n)) == 0 and n.value == 0
    assert ws(5, 3, 16, 32, 48, ctypes.byref(n)) == 0 and n.value == 0        # few tokens: one launch
    assert ws(2000, 3, 64, 1024, 4096, ctypes.byref(n)) == 0 and n.value >= 2000 * 64 * 4
    assert ws(5, 3, 16, 32, 48, None) == INVALID and ws(5, 3, 12, 32, 48, ctypes.byref(n)) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(1, 16, 8, dtype=torch.bfloat16)
    h = torch.zeros(4, 16, dtype=torch.bfloat16)
    for call in (lambda: fgg.grouped_linear(x, w), lambda: fgg.grouped_linear_backward_input(h, w),
                 lambda: fgg.grouped_linear_backward_weight(h, x, 1), lambda: fgg.grouped_gated(x, w),
                 lambda: fgg.grouped_gated_backward(h, w, h),
                 lambda: fgg.lora_add(h, x, torch.zeros(4, dtype=torch.int32), w, w)):
        with pytest.raises(AssertionError):
            call()
