"""The bf16 products and the adapters where elements lie past 2^31: weights, their gradients, rows and outputs."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, HALF, gated, product, within

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed + len(shape))
    t = torch.empty(*shape, dtype=BF16, device="cuda").normal_(generator=g)
    return t if scale == 1.0 else t.mul_(scale)


def test_weights_and_their_gradient():
    G, N, K = 34, 8192, 8200
    sizes = [70 + g % 5 for g in range(G)]
    offsets = torch.tensor([0] + sizes, device="cuda").cumsum(0).int()
    M = int(offsets[-1])
    assert G * N * K > 1 << 31
    x, dy, w = randn(M, K, seed=1), randn(M, N, seed=2), randn(G, N, K, seed=3)
    y = fgg.grouped_linear(x, w, offsets)
    dx = fgg.grouped_linear_backward_input(dy, w, offsets, out_dtype=F32)
    dw = fgg.grouped_linear_backward_weight(dy, x, G, offsets, out_dtype=BF16)
    for g in (0, 31, 32, G - 1):
        s, e = int(offsets[g]), int(offsets[g + 1])
        within(y[s:e], *product(x[s:e], w[g].t(), BF16), f"y {g}")
        within(dx[s:e], *product(dy[s:e], w[g], F32), f"dx {g}")
        within(dw[g], *product(dy[s:e].t(), x[s:e], BF16), f"dw {g}")


def test_rows_of_the_gated_block():
    M, I, K = 135000, 8192, 64
    at = [slice(0, 40), slice((1 << 31) // (2 * I) - 20, (1 << 31) // (2 * I) + 20), slice(M - 40, M)]
    assert M * 2 * I > 1 << 31
    x, w, wd = randn(M, K, seed=4), randn(1, 2 * I, K, seed=5, scale=0.125), randn(1, K, I, seed=6, scale=0.125)
    h = torch.empty(M, 2 * I, dtype=BF16, device="cuda")
    a, _ = fgg.grouped_gated(x, w, h=h)
    dh, _ = fgg.grouped_gated_backward(x, wd, h)
    for s in at:
        ref, bound = product(x[s], w[0].t(), BF16)
        within(h[s], ref, bound, "h")
        # a from the products before their rounding: |d silu| <= 1.1, the sigmoid's and products' roundings
        pre, off = product(x[s], w[0].t(), F32)
        (gate, up), (dg, du) = pre.chunk(2, dim=1), off.chunk(2, dim=1)
        want = gated(pre)
        slack = (gate.abs() + 4) * 2.0 ** -21 * want.abs() + 1.1 * dg * up.abs() + gate.abs() * du + 1.1 * dg * du
        within(a[s], want, HALF[BF16] * want.abs() + 1.01 * slack + 1e-37, "a")
        hs = h[s].double().requires_grad_()
        da, dda = product(x[s], wd[0], F32)
        gated(hs).backward(da)
        dgate, dup = h[s].double().chunk(2, dim=1)
        sig = torch.sigmoid(dgate)
        # the factors of da, and 2^-21 of the largest term for their own roundings
        f = torch.cat([dup.abs() * sig * (1 + dgate.abs()), dgate.abs() * sig], 1)
        both = torch.cat([da, da], 1).abs(), torch.cat([dda, dda], 1)
        big = torch.cat([dgate, dgate], 1).abs() + 4
        within(dh[s], hs.grad, HALF[BF16] * hs.grad.abs() + 1.01 * f * (both[1] + big * 2.0 ** -21 * both[0]) + 1e-37,
               "dh")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_the_adapters(dtype):
    T, L, r, N, K = 265000, 3, 8, 8192, 72
    assert T * N > 1 << 31
    base, x = torch.zeros(T, N, dtype=dtype, device="cuda"), randn(T, K, seed=7)
    a, b = randn(L, r, K, seed=8), randn(L, N, r, seed=9)
    ids = (torch.arange(T, device="cuda") * L // T).int()
    out = fgg.lora_add(base, x, ids, a, b, out=base)
    for s in (slice(0, 40), slice((1 << 31) // N - 20, (1 << 31) // N + 20), slice(T - 40, T)):
        e = int(ids[s][0])
        v, mag = x[s].double() @ a[e].double().t(), x[s].abs().double() @ a[e].abs().double().t()
        ref, B = v @ b[e].double().t(), b[e].abs().double().t()
        cut = 2.0 ** -17 if dtype == BF16 else 2.0 ** -24
        inner = (K + 2) * 2.0 ** -24 * mag + cut * v.abs()
        within(out[s], ref, HALF[dtype] * ref.abs() + 1.01 * inner @ B + (3 * r + 2) * 2.0 ** -24 * (v.abs() @ B) + 1e-37,
               "adapters")
