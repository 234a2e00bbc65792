"""The few-token FP4 products in the forms that their launch rules choose between
(whatever the number of compute units they are told of, every output is written once
and right), and at the ends of the ranges of scales and activations.

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


@pytest.mark.parametrize("cus", [65535, 65536, 200000, 1 << 22, 1 << 29, 1 << 30, (1 << 31) - 1])
@pytest.mark.parametrize("T", [3, 70001])
def test_any_number_of_compute_units(cus, T):
    """The launch rules hold for every count that fgg_set_num_cus takes: no overflow, no grid past the limits."""
    G, N, K, k = 3, 16, 64, 1
    W, b, s, q = _weights(T, G, N, K, False)
    g = synth.rng(T)
    ids = g.integers(0, G, size=(T, k)).astype(np.int32)
    x = synth.to_bf16_values(g.standard_normal((T, K)).astype(np.float32))
    w = g.random((T, k), dtype=np.float32)
    fgg.set_num_cus(cus)
    args = (cuda(x, torch.bfloat16), b, s, cuda(ids))
    y = np.stack([x.astype(np.float64) @ W[e].T for e in range(G)])[ids[:, 0], np.arange(T)]
    mag = np.stack([np.abs(x.astype(np.float64)) @ np.abs(W[e].T) for e in range(G)])[ids[:, 0], np.arange(T)]
    got = to_np(fgg.moe_gemv_fp4(*args, out_dtype=torch.float32))[:, 0]
    assert np.all(np.abs(got - y) <= _bound(mag, K, k) + 2.0 ** -24 * np.abs(y))
    got = to_np(fgg.moe_gemv_fp4(*args, cuda(w), out_dtype=torch.float32))
    assert np.all(np.abs(got - y * w) <= _bound(mag * w, K, k) + 2.0 ** -24 * np.abs(y * w))


@pytest.mark.parametrize("tiled", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scale_bytes_at_the_ends(tiled, dtype):
    """One-hot activations and a row per code and scale byte: exact for every weight below 2^128 (0 to
    252 are all of the codes'), infinite or NaN from there on, NaN for byte 255, and each row by itself."""
    K, ends = 256, [0, 1, 2, 3, 126, 127, 252, 253, 254, 255]
    codes = np.repeat(np.tile(np.arange(16, dtype=np.uint8) * 17, len(ends))[:, None], K // 2, 1)[None]
    sc = np.repeat(np.repeat(np.array(ends, np.uint8), 16)[:, None], K // 32, 1)[None]
    N = codes.shape[1]
    W = oracle.fp4_weights(codes, sc)[0]
    b, s, q = cuda(codes), cuda(sc), fgg.Q_E2M1_E8M0_1x32
    if tiled:
        (b, s), q = fgg.pack_fp4_weights(b, s), fgg.Q_E2M1_E8M0_1x32_TILED
    for T in (1, 7, 16):
        for value in (1.0, -2.0 ** -20):
            x = np.zeros((T, K), np.float32)
            at = (np.arange(T) * 37 + 5) % K
            x[np.arange(T), at] = value
            got = to_np(fgg.moe_gemv_fp4(cuda(x, dtype), b, s, b_qdesc=q, n=N, out_dtype=torch.float32))
            want = W[:, at].T * value
            inside = np.abs(W[:, at].T) < 2.0 ** 128
            assert inside[:, :16 * 7].all() and not inside[:, 16 * 9:].any()
            np.testing.assert_array_equal(got[inside], want[inside].astype(np.float32))
            assert not np.isfinite(got[~inside]).any() and np.isnan(got[:, 16 * 9:]).all()


@pytest.mark.parametrize("byte", [127, 150, 220])
def test_the_smallest_activations(byte):
    """bf16 down to its smallest step is exact; of fp32 what lies below 2^-133 is dropped, nothing of a
    number of 2^-110 and more."""
    K, N = 96, 16
    codes = np.full((1, N, K // 2), 0x22, np.uint8)          # code 2: the value 1
    sc = np.full((1, N, K // 32), byte, np.uint8)
    b, s = cuda(codes), cuda(sc)
    scale = 2.0 ** (byte - 127)
    g = synth.rng(byte)

    def one_hot(v):
        x = np.zeros((len(v), K), np.float32)
        x[np.arange(len(v)), g.integers(0, K, len(v))] = v
        return x

    v = (np.arange(1, 128) * 2.0 ** -133).astype(np.float32) * np.where(np.arange(127) % 2, 1, -1).astype(np.float32)
    x = torch.from_numpy(one_hot(v)).to(torch.bfloat16).cuda()
    got = to_np(fgg.moe_gemv_fp4(x, b, s, out_dtype=torch.float32)).astype(np.float64)
    np.testing.assert_array_equal(got, np.repeat(v.astype(np.float64)[:, None] * scale, N, 1))
    e = np.arange(-149, -95)
    v = np.ldexp(1 + g.integers(0, 1 << 23, e.size) / 2.0 ** 23, e).astype(np.float32)
    got = to_np(fgg.moe_gemv_fp4(cuda(one_hot(v)), b, s, out_dtype=torch.float32)).astype(np.float64)
    err = np.abs(got - v.astype(np.float64)[:, None] * scale)
    assert np.all(err < 2.0 ** -133 * scale) and np.all(err[e >= -110] == 0)


@pytest.mark.parametrize("T,G,k,N,K", [(1, 1, 1, 64, 512), (16, 1, 1, 48, 512), (5, 1, 1, 32, 1024), (3, 2, 1, 9600, 256),
                                       (16, 2, 1, 9600, 512), (8, 2, 1, 9600, 1024), (2, 1, 1, 16, 4096)])
@pytest.mark.parametrize("tiled", [True, False])
@pytest.mark.parametrize("silu", [True, False])
def test_chain_of_a_waves_share(T, G, k, N, K, tiled, silu):
    """Nonnegative weights and activations, so that every sum only grows and no rounding is hidden by
    cancellation.  A wave takes spans of 512 of K, 16 instructions each, as many as its share of the
    tile's waves: from one wave a tile (K to 512 with many tiles) to eight, a chain of at most K/32
    instructions whatever the share, 5 levels inside one, 8 waves joined.  SiLU of g >= 0 has a slope of
    at most 1.1 and 16 roundings of its own."""
    g = synth.rng(N + K)
    rows = 2 * N if silu else N
    codes = (g.integers(0, 8, size=(G, rows, K // 2)) + 16 * g.integers(0, 8, size=(G, rows, K // 2))).astype(np.uint8)
    sc = g.integers(116, 120, size=(G, rows, K // 32), dtype=np.uint8)
    W = oracle.fp4_weights(codes, sc)
    b, s, q = cuda(codes), cuda(sc), fgg.Q_E2M1_E8M0_1x32
    if tiled:
        (b, s), q = fgg.pack_fp4_weights(b, s), fgg.Q_E2M1_E8M0_1x32_TILED
    ids = None if G == 1 else g.integers(0, G, size=(T, k)).astype(np.int32)
    x = synth.to_bf16_values(g.random((T, K), dtype=np.float32))
    got = to_np(fgg.moe_gemv_fp4(cuda(x, torch.bfloat16), b, s, None if ids is None else cuda(ids), b_qdesc=q, n=N,
                                 silu_mul=silu, out_dtype=torch.float32))
    levels = (K / 32 + 5 + 8) * 2.0 ** -23
    if silu:
        ref, mag, gate, up = oracle.moe_gemv_fp4(x, W, ids, silu_mul=True)
        eg, eu = levels * mag[..., 0, :], levels * mag[..., 1, :]
        tol = (up + eu) * 1.1 * eg + np.abs(gate) * eu + 17 * 2.0 ** -24 * np.abs(ref)
    else:
        ref, mag = oracle.moe_gemv_fp4(x, W, ids)
        tol = levels * mag + 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(got.reshape(ref.shape) - ref) <= tol)
