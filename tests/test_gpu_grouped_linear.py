"""The bf16 products of row segments (linear, its gradients) against float64, at ragged sizes:
one row to several tiles, widths that end inside a tile, sums that end inside a block, empty
segments, gaps of NaN between segments, strided rows."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, matrix, poison, product, segments, spans, within

pytestmark = pytest.mark.gpu

# rows, segments, N, K
SIZES = [(1, 1, 8, 8), (3, 2, 16, 24), (20, 5, 72, 136), (65, 1, 264, 64), (257, 3, 256, 72), (300, 1, 520, 1000),
         (700, 6, 1032, 200), (1000, 40, 136, 328), (1500, 2, 24, 2056), (600, 70, 64, 520)]


def case(M, G, N, K, padded, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + M + N)
    offsets, counts, rows = segments(G, M, seed + G, padded)
    if G == 1 and not padded:
        offsets = counts = None
    sp = [(0, M)] if offsets is None else spans(offsets, counts, rows)
    return g, offsets, counts, rows, sp


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,G,N,K", SIZES)
def test_linear(M, G, N, K, dtype, padded):
    g, offsets, counts, rows, sp = case(M, G, N, K, padded)
    x, w = matrix(g, rows, K, K + 8 * (M % 3)), (torch.randn(G, N, K, generator=g, device="cuda") * 0.1).to(BF16)
    live = poison(x, sp)
    out = matrix(g, rows, N, N + 8 * (M % 2), dtype)
    before = out.clone()
    got = fgg.grouped_linear(x, w, offsets, counts, out=out)
    assert got is out and torch.equal(got[~live], before[~live])
    for e, (s, t) in enumerate(sp):
        if t > s:
            within(got[s:t], *product(x[s:t], w[e].t(), dtype), f"segment {e}")


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,G,N,K", SIZES)
def test_backward_input(M, G, N, K, dtype, padded):
    g, offsets, counts, rows, sp = case(M, G, N, K, padded, 1)
    dy, w = matrix(g, rows, N, N + 8 * (M % 3)), (torch.randn(G, N, K, generator=g, device="cuda") * 0.1).to(BF16)
    live = poison(dy, sp)
    out = matrix(g, rows, K, K + 8 * (M % 2), dtype)
    before = out.clone()
    got = fgg.grouped_linear_backward_input(dy, w, offsets, counts, out=out)
    assert torch.equal(got[~live], before[~live])
    for e, (s, t) in enumerate(sp):
        if t > s:
            within(got[s:t], *product(dy[s:t], w[e], dtype), f"segment {e}")


@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,G,N,K", SIZES)
def test_backward_weight(M, G, N, K, dtype, padded):
    g, offsets, counts, rows, sp = case(M, G, N, K, padded, 2)
    dy, x = matrix(g, rows, N, N + 8 * (M % 3)), matrix(g, rows, K, K + 8 * (M % 2))
    poison(dy, sp), poison(x, sp)
    got = fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out_dtype=dtype)
    assert got.dtype == dtype and got.shape == (G, N, K)
    again = got.clone()
    fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out=again, accumulate=True)
    for e, (s, t) in enumerate(sp):
        if t == s:
            assert not got[e].any() and not again[e].any()
            continue
        ref, bound = product(dy[s:t].t(), x[s:t], dtype)
        within(got[e], ref, bound, f"segment {e}")
        # added in fp32 to what stands there and rounded once more
        within(again[e], 2 * ref, 3 * bound, f"segment {e}, twice")


def test_nothing_at_all():
    w = torch.randn(3, 16, 24, device="cuda").to(BF16)
    x, dy = torch.empty(0, 24, dtype=BF16, device="cuda"), torch.empty(0, 16, dtype=BF16, device="cuda")
    offsets = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert fgg.grouped_linear(x, w, offsets).shape == (0, 16)
    assert fgg.grouped_linear_backward_input(dy, w, offsets).shape == (0, 24)
    assert not fgg.grouped_linear_backward_weight(dy, x, 3, offsets).any()


def test_segments_stay_inside_the_rows():
    """offsets past M (a buffer too small for its rows): the rows that exist, and nothing else."""
    g = torch.Generator(device="cuda").manual_seed(5)
    M, N, K = 100, 72, 40
    x, w = matrix(g, M, K, K), matrix(g, 3 * N, K, K).view(3, N, K)
    offsets = torch.tensor([0, 60, 130, 400], dtype=torch.int32, device="cuda")
    got = fgg.grouped_linear(x, w, offsets, out_dtype=F32)
    for e, (s, t) in enumerate([(0, 60), (60, 100)]):
        within(got[s:t], *product(x[s:t], w[e].t(), F32), f"segment {e}")
    dy = matrix(g, M, N, N)
    dw = fgg.grouped_linear_backward_weight(dy, x, 3, offsets)
    within(dw[1], *product(dy[60:].t(), x[60:], F32), "the cut segment")
    assert not dw[2].any()


def test_same_bits_every_time():
    g = torch.Generator(device="cuda").manual_seed(6)
    dy, x, w = matrix(g, 3000, 264, 264), matrix(g, 3000, 136, 136), matrix(g, 264, 136, 136)[None].contiguous()
    for call in (lambda: fgg.grouped_linear(x, w), lambda: fgg.grouped_linear_backward_input(dy, w),
                 lambda: fgg.grouped_linear_backward_weight(dy, x, 1)):
        first = call()
        assert all(torch.equal(first, call()) for _ in range(3))
