"""Adapters with infinite factors: each launch form gives the definition's infinities, and only where they belong."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32
from test_gpu_lora import inputs

pytestmark = pytest.mark.gpu

INF = float("inf")
# tokens, ranks, columns, sum; whether a workspace is needed (two launches: tiles of 16 tokens, of 64)
FORMS = [(20, 16, 72, 136, False), (300, 16, 2056, 16392, True), (300, 64, 2048, 4104, True), (4000, 8, 3080, 136, True),
         (600, 40, 1032, 136, True), (530, 128, 72, 264, True)]


def form(T, r, N, K, two, dtype, kind, seed):
    assert (fgg.lora_workspace_bytes(T, 4, r, N, K) > 0) == two
    return inputs(T, 4, r, N, K, dtype, kind, seed)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,r,N,K,two", FORMS)
def test_infinite_rows_of_b(T, r, N, K, two, dtype):
    base, x, ids, a, b, scales = form(T, r, N, K, two, dtype, "any", 4)
    ids[:8] = torch.tensor([0, 1, 2, 3, 0, 1, 2, 3])
    clean = fgg.lora_add(base, x, ids, a, b, scales)
    # (in whole columns, in one column, and two of one column that meet with equal or with different signs)
    b[2, :, 3], b[1, 5, 0], b[1, 17, r - 1], b[0, 9, 1], b[0, 9, 6] = INF, -INF, INF, INF, -INF
    got = fgg.lora_add(base, x, ids, a, b, scales)
    touched = torch.zeros_like(got, dtype=torch.bool)
    touched[ids == 2] = True
    touched[ids == 1, 5] = touched[ids == 1, 17] = touched[ids == 0, 9] = True
    assert torch.equal(got[~touched], clean[~touched])
    for e in range(4):
        t = torch.nonzero(ids == e)[:, 0]
        X, A = x[t].double(), a[e].double()
        v, err = X @ A.t(), (K + 2) * 2.0 ** -24 * (X.abs() @ A.abs().t())
        sure = v.abs() > err                                         # (else the fp32 sum's sign is not fixed)
        for n, js in {2: [(n, [3]) for n in range(N)], 1: [(5, [0]), (17, [r - 1])], 0: [(9, [1, 6])]}.get(e, []):
            terms = v[:, js].sign() * b[e, n, js].double()
            ok = sure[:, js].all(1)
            assert ok.any()
            same = got[t[ok], n].double().nan_to_num(0, 1, -1) == terms.sum(1)[ok].nan_to_num(0, 1, -1)
            assert bool(same.all())
            assert not got[t, n].isfinite().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,r,N,K,two", FORMS)
def test_infinite_rows_of_x_and_a(T, r, N, K, two, dtype):
    """Positive factors: an infinite element makes its token's, or its adapter's, whole row infinite."""
    base, x, ids, a, b, scales = form(T, r, N, K, two, dtype, "runs", 5)
    x, a, b = x.abs() + 2.0 ** -10, a.abs() + 2.0 ** -10, b.abs() + 2.0 ** -10
    clean = fgg.lora_add(base, x, ids, a, b, scales)
    x[3, 7], x[T - 1, K - 1], a[1, 4, 0] = INF, -INF, INF
    got = fgg.lora_add(base, x, ids, a, b, scales)
    up, down = ids == 1, torch.zeros(T, dtype=torch.bool, device="cuda")
    up[3], down[T - 1] = True, True
    assert (got[up] == INF).all() and (got[down] == -INF).all()
    assert torch.equal(got[~up & ~down], clean[~up & ~down])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,r,N,K,two", FORMS)
def test_sums_past_the_largest_bf16_value(T, r, N, K, two, dtype):
    """Inner sums between the largest bf16 value and the largest fp32 value, scaled down by b: exact in 24 bits."""
    base, x, ids, a, b, _ = form(T, r, N, K, two, dtype, "runs", 6)
    top = 255 * 2.0 ** 120
    x[:], a[:], b[:], base[:] = 0, 0, 0, 0
    x[3, 0], x[3, 1] = top, 2.0 ** 119                   # the sum: top + 3/4 of the step that 2^127 has in bf16
    a[:, 0, 0], a[:, 0, 1] = 1, 1.5
    b[:, :, 0] = 2.0 ** -127
    got = fgg.lora_add(base, x, ids, a, b).double()
    want = (top + 1.5 * 2.0 ** 119) * 2.0 ** -127
    assert (got[3] == torch.tensor(want, dtype=torch.float64).to(dtype).double().item()).all()
    assert (got[:3] == 0).all() and (got[4:] == 0).all()
