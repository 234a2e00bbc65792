"""Low-rank adapters per token against float64.

Bound: the inner sum's fp32 error (K 2^-24 of its magnitudes) and the parts' cut (2^-17 with bf16
outputs, 2^-24 with fp32) reach the result through |b|; the outer sum of up to 3 r products adds
(3 r + 2) 2^-24 of its magnitudes, and the result is rounded once."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, HALF, matrix, within

pytestmark = pytest.mark.gpu


def inputs(T, L, r, N, K, dtype, kind, seed=0, pad=8):
    g = torch.Generator(device="cuda").manual_seed(seed + T + r)
    x, base = matrix(g, T, K, K + pad), matrix(g, T, N, N + pad, dtype)
    a = (torch.randn(L, r, K, generator=g, device="cuda") * K ** -0.5).to(BF16)
    b = (torch.randn(L, N, r, generator=g, device="cuda") * r ** -0.5).to(BF16)
    scales = torch.rand(L, generator=g, device="cuda") + 0.5
    if kind == "runs":
        ids = torch.arange(T, device="cuda") * L // max(T, 1)
    elif kind == "one":
        ids = torch.full((T,), L - 1, device="cuda")
    else:
        ids = torch.randint(0, L, (T,), generator=g, device="cuda")
        ids[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
        if T > 2:
            ids[1], ids[2] = L, -2 ** 31           # neither is an adapter
    return base, x, ids.int(), a, b, scales


def check(got, base, x, ids, a, b, scales, dtype):
    T, K, r = x.shape[0], x.shape[1], a.shape[1]
    for e in range(a.shape[0]):
        t = torch.nonzero(ids == e)[:, 0]
        if not t.numel():
            continue
        X, A, B, s = x[t].double(), a[e].double(), b[e].double(), 1.0 if scales is None else scales[e].double()
        v, mag = X @ A.t(), X.abs() @ A.abs().t()
        ref = base[t].double() + s * (v @ B.t())
        cut = 2.0 ** -17 if dtype == BF16 else 2.0 ** -24
        inner = (K + 2) * 2.0 ** -24 * mag + cut * v.abs()
        outer = (3 * r + 2) * 2.0 ** -24 * (s * (v.abs() @ B.abs().t()) + base[t].double().abs())
        within(got[t], ref, HALF[dtype] * ref.abs() + 1.01 * s * (inner @ B.abs().t()) + outer + 1e-37, f"adapter {e}")
    none = (ids < 0) | (ids >= a.shape[0])
    assert torch.equal(got[none], base[none])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", ["runs", "any", "one"])
@pytest.mark.parametrize("T,L,r,N,K", [(1, 1, 8, 8, 8), (1, 3, 16, 264, 4104), (5, 4, 24, 40, 136), (16, 16, 16, 1000, 1992),
                                       (17, 40, 64, 96, 520), (70, 6, 128, 136, 72), (200, 300, 8, 64, 264),
                                       (513, 5, 16, 200, 328), (600, 3, 40, 1032, 136), (530, 9, 128, 72, 264),
                                       (1300, 64, 32, 72, 40), (2000, 2, 104, 264, 392), (300, 5, 16, 2056, 16392),
                                       (260, 3, 32, 4104, 8200), (300, 40, 64, 2048, 4104), (130, 4, 128, 4104, 4104),
                                       (3000, 4, 16, 2056, 1032), (2500, 3, 32, 4104, 520), (6000, 7, 64, 1032, 264),
                                       (1500, 2, 128, 2056, 2056), (4000, 5, 8, 3080, 136)])
def test_adapters(T, L, r, N, K, dtype, kind):
    base, x, ids, a, b, scales = inputs(T, L, r, N, K, dtype, kind)
    before = base.clone()
    got = fgg.lora_add(base, x, ids, a, b, scales)
    assert torch.equal(base, before)
    check(got, base, x, ids, a, b, scales, dtype)
    assert torch.equal(got, fgg.lora_add(base, x, ids, a, b, scales))
    held = base                                     # in place, rows strided
    assert fgg.lora_add(held, x, ids, a, b, scales, out=held) is held and torch.equal(held, got)


@pytest.mark.parametrize("T", [3, 40, 600])
def test_without_scales_and_without_tokens(T):
    base, x, ids, a, b, _ = inputs(T, 4, 16, 72, 136, F32, "any", 1)
    check(fgg.lora_add(base, x, ids, a, b), base, x, ids, a, b, None, F32)
    assert torch.equal(fgg.lora_add(base, x, torch.full_like(ids, -1), a, b), base)
    assert fgg.lora_add(base[:0], x[:0], ids[:0], a, b).shape == (0, 72)


@pytest.mark.parametrize("T", [20, 600])
def test_nan_stays_with_its_token_and_adapter(T):
    base, x, ids, a, b, scales = inputs(T, 4, 16, 72, 136, BF16, "any", 2)
    ids[:8] = torch.tensor([0, 1, 2, 3, 0, 1, 2, 3])
    clean = fgg.lora_add(base, x, ids, a, b, scales)
    a[1], b[2, :, 3] = float("nan"), float("inf")
    x[4] = float("nan")
    got = fgg.lora_add(base, x, ids, a, b, scales)
    apart = (ids != 1) & (ids != 2)
    apart[4] = False
    assert torch.equal(got[apart], clean[apart])
    assert got[ids == 1].isnan().all() and got[4].isnan().all()
    assert not got[ids == 2].isfinite().any()


@pytest.mark.parametrize("L,r,K", [(2100, 16, 32768), (2040, 16, 32768), (1030, 24, 65536)])
def test_factors_past_32_bit_offsets(L, r, K):
    # (2 GiB of factors and just less, read as one array, by tokens whose adapters lie anywhere in it)
    base, x, ids, a, b, scales = inputs(600, L, r, 40, K, F32, "any", 3)
    ids[-1], ids[-2] = L - 1, 0
    check(fgg.lora_add(base, x, ids, a, b, scales), base, x, ids, a, b, scales, F32)
