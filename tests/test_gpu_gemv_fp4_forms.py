"""The few-token FP4 products in the forms that their launch rules choose between:
whatever the number of compute units they are told of, every output is written once
and right.

Tolerance: as in test_gpu_gemv_fp4.py's summed form, the chain of one wave counted
as the whole of K (K/32 instructions), 5 levels inside an instruction, 16 waves
joined and two roundings per slot, each 2^-23 (for sums that truncate) of the sum of
the products' magnitudes; a bf16 result adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

import fp4_grouped_gemm_amd as fgg
import oracle
import synth
from _util import cuda, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def all_cus():
    yield
    fgg.set_num_cus(0)


def _weights(seed, G, N, K, tiled):
    g = synth.rng(seed)
    codes = g.integers(0, 256, size=(G, N, K // 2), dtype=np.uint8)
    sc = g.integers(118, 130, size=(G, N, K // 32), dtype=np.uint8)
    b, s = cuda(codes), cuda(sc)
    if tiled:
        return oracle.fp4_weights(codes, sc), *fgg.pack_fp4_weights(b, s), fgg.Q_E2M1_E8M0_1x32_TILED
    return oracle.fp4_weights(codes, sc), b, s, fgg.Q_E2M1_E8M0_1x32


def _bound(mag, K, k):
    return (K / 32 + 5 + 16 + 2 * k) * 2.0 ** -23 * mag


@pytest.mark.parametrize("cus", [2, 3, 4, 6, 11, 40])
@pytest.mark.parametrize("tiled", [True, False])
def test_sum_writes_every_column(cus, tiled):
    """The summed form's tokens per workgroup and row tiles per wave are chosen apart: no pair of
    choices may leave columns out."""
    G, k, K = 5, 2, 256
    fgg.set_num_cus(cus)
    for N in (16, 32, 48, 64, 160):
        W, b, s, q = _weights(N, G, N, K, tiled)
        for T in (1, 3, 5, 6, 8, 9, 16, 21):
            g = synth.rng(T)
            ids = g.integers(0, G, size=(T, k)).astype(np.int32)
            w = g.random((T, k), dtype=np.float32)
            x = synth.to_bf16_values(g.standard_normal((T, K)).astype(np.float32))
            out = torch.full((T, N), float("nan"), device="cuda")
            fgg.moe_gemv_fp4(cuda(x, torch.bfloat16), b, s, cuda(ids), cuda(w), b_qdesc=q, n=N, out=out)
            ref, mag = oracle.moe_gemv_fp4(x, W, ids, w=w)
            assert np.all(np.abs(to_np(out) - ref) <= _bound(mag, K, k) + 2.0 ** -24 * np.abs(ref)), (N, T)
