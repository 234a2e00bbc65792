"""The bf16 products at the largest counts of rows that the calls take."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def sparse(M, cols, at, seed):
    """[M, cols] of zeros but for the rows `at`, which hold whole numbers of -4 to 4."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.zeros(M, cols, dtype=BF16, device="cuda")
    t[at] = torch.randint(-4, 5, (len(at), cols), generator=g, device="cuda").to(BF16)
    return t


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,first", [(MOST, None), (MOST, 3), (MOST - 62, None), (MOST - 63, None)])
def test_weight_gradient(M, first, dtype):
    """All terms but these are zero, and whole numbers this small have exact sums in any order."""
    at = torch.tensor([0, 1, 2, 3, 70, 2 ** 26 - 1, 2 ** 26, 2 ** 30 + 5, M - 66, M - 65, M - 64, M - 2, M - 1],
                      device="cuda")
    dy, x = sparse(M, 8, at, 1), sparse(M, 8, at, 2)
    offsets = None if first is None else torch.tensor([0, first, M], dtype=torch.int32, device="cuda")
    spans = [(0, M)] if first is None else [(0, first), (first, M)]
    got = fgg.grouped_linear_backward_weight(dy, x, len(spans), offsets, out_dtype=dtype)
    again = fgg.grouped_linear_backward_weight(dy, x, len(spans), offsets, out=got.clone(), accumulate=True)
    for g, (s, e) in enumerate(spans):
        rows = at[(at >= s) & (at < e)]
        want = dy[rows].double().t() @ x[rows].double()
        assert want.abs().max() > 0
        assert torch.equal(got[g].double(), want) and torch.equal(again[g].double(), 2 * want)
