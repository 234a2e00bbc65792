"""GPU parity of the few-token FP4 products against the float64 oracle.

Tolerance: the products are exact; sums run in fp32, an instruction (32 of K)
counted as 5 levels of 32 products and one addition to the chain before it.  Where
K is split over 4 or 8 waves a chain has at most K/128 + 1 instructions and 8
partial sums are joined: depth = K/128 + 1 + 5 + 8.  In the summed form one wave
may take an expert's whole K, K/32 instructions, the experts are added with two
roundings each and 16 waves joined: depth = K/32 + 5 + 16 + 2k.  Each is 2^-23 (for
sums that truncate) of the sum of the products' magnitudes; fp32 activations take
three instructions a step.  SiLU is
|d silu| <= 1.1 |dg|, and 16 roundings of its own.  A bf16 result adds half a
step, 2^-8."""

import numpy as np
import pytest
import torch

import fp4_grouped_gemm_amd as fgg
import oracle
import synth
from _util import cuda, to_np

pytestmark = pytest.mark.gpu


def _weights(seed, G, N, K, tiled):
    g = synth.rng(seed)
    codes = g.integers(0, 256, size=(G, N, K // 2), dtype=np.uint8)
    sc = g.integers(118, 130, size=(G, N, K // 32), dtype=np.uint8)
    b, s = cuda(codes), cuda(sc)
    if tiled:
        return oracle.fp4_weights(codes, sc), *fgg.pack_fp4_weights(b, s), fgg.Q_E2M1_E8M0_1x32_TILED
    return oracle.fp4_weights(codes, sc), b, s, fgg.Q_E2M1_E8M0_1x32


def _x(seed, shape, dtype):
    x = synth.rng(seed).standard_normal(shape).astype(np.float32)
    return synth.to_bf16_values(x) if dtype == torch.bfloat16 else x


def _tol(mag, K, k, dtype, summed=False):
    chain = (K / 32 if summed else K / 128 + 1) * (3 if dtype == torch.float32 else 1)
    return (chain + 5 + (16 + 2 * k if summed else 8)) * 2.0 ** -23 * mag


def _half(dtype, ref):
    return 2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 2.0 ** -24 * np.abs(ref)


CASES = [  # T, G, k, N, K, tiled
    (1, 1, 1, 16, 128, True), (1, 1, 1, 4096, 7168, True), (1, 1, 1, 1, 32, False), (3, 1, 1, 45, 160, False),
    (16, 1, 1, 528, 1024, True), (17, 1, 1, 100, 2080, False), (40, 1, 1, 64, 256, True),
    (1, 32, 8, 256, 512, True), (2, 4, 3, 33, 96, False), (16, 8, 2, 160, 640, True), (13, 32, 8, 77, 1312, False),
    (5, 1024, 4, 16, 128, True), (16, 70, 64, 18, 64, False), (33, 6, 2, 48, 384, True),
    (12, 3, 3, 97, 2656, False), (10, 40, 5, 1040, 1152, True), (16, 2, 1, 31, 4096, False),
    (17, 32, 8, 2560, 256, True), (21, 20, 4, 1000, 288, False), (7, 24, 2, 500, 512, False), (6, 9, 4, 64, 1664, True),
]


@pytest.fixture(params=[0, 1], ids=["all CUs", "1 CU"], autouse=True)
def cus(request):
    """Also with the launch rules of a single compute unit: several tiles a workgroup, and two tiles
    a wave in the summed form whatever the number of columns."""
    fgg.set_num_cus(request.param)
    yield request.param
    fgg.set_num_cus(0)


def _ids(seed, T, G, k, drop=0.15):
    g = synth.rng(seed)
    ids = g.integers(0, G, size=(T, k)).astype(np.int32)     # an expert may stand twice in a token
    ids[g.random((T, k)) < drop] = -1
    ids[g.random((T, k)) < 0.03] = G + 3
    return ids


@pytest.mark.parametrize("T,G,k,N,K,tiled", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_plain(T, G, k, N, K, tiled, dtype):
    W, b, s, q = _weights(1, G, N, K, tiled)
    ids = None if G == 1 else _ids(2, T, G, k)
    for per_slot in (False, True) if ids is not None else (False,):
        x = _x(3, (T, k, K) if per_slot else (T, K), dtype)
        ref, mag = oracle.moe_gemv_fp4(x, W, ids)
        for od in (torch.float32, torch.bfloat16):
            got = to_np(fgg.moe_gemv_fp4(cuda(x, dtype), b, s, None if ids is None else cuda(ids), b_qdesc=q, n=N,
                                         out_dtype=od))
            err = np.abs(got - ref)
            assert np.all(err <= _tol(mag, K, k, dtype) * (1 + 2.0 ** -8) + _half(od, ref)), err.max()
            if ids is not None:
                assert (got[(ids < 0) | (ids >= G)] == 0).all()


@pytest.mark.parametrize("T,G,k,N,K,tiled", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_silu(T, G, k, N, K, tiled, dtype):
    W, b, s, q = _weights(4, G, 2 * N, K, tiled)
    ids = None if G == 1 else _ids(5, T, G, k)
    x = _x(6, (T, K), dtype) * np.float32(0.125)
    ref, mag, gate, up = oracle.moe_gemv_fp4(x, W, ids, silu_mul=True)
    eg, eu = _tol(mag[..., 0, :], K, 0, dtype), _tol(mag[..., 1, :], K, 0, dtype)
    with np.errstate(over="ignore"):
        silu = np.abs(gate / (1 + np.exp(-gate)))
    tol = (np.abs(up) + eu) * 1.1 * eg + silu * eu + 16 * 2.0 ** -24 * np.abs(ref)
    for od in (torch.float32, torch.bfloat16):
        got = to_np(fgg.moe_gemv_fp4(cuda(x, dtype), b, s, None if ids is None else cuda(ids), b_qdesc=q, n=N,
                                     silu_mul=True, out_dtype=od)).reshape(ref.shape)
        err = np.abs(got - ref)
        assert np.all(err <= tol * (1 + 2.0 ** -8) + _half(od, ref) + 2.0 ** -120), (err / (tol + 1e-30)).max()


@pytest.mark.parametrize("T,G,k,N,K,tiled", [c for c in CASES if c[1] > 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_sum(T, G, k, N, K, tiled, dtype):
    W, b, s, q = _weights(7, G, N, K, tiled)
    ids = _ids(8, T, G, k)
    w = synth.rng(9).random((T, k), dtype=np.float32)
    w[(ids < 0) | (ids >= G)] = np.nan                       # weights of absent experts are not read
    for per_slot in (True, False):
        x = _x(10, (T, k, K) if per_slot else (T, K), dtype)
        if per_slot:
            x[(ids < 0) | (ids >= G)] = np.nan               # nor their activations
        ref, mag = oracle.moe_gemv_fp4(np.nan_to_num(x), W, ids, w=w)
        for od in (torch.float32, torch.bfloat16):
            got = to_np(fgg.moe_gemv_fp4(cuda(x, dtype), b, s, cuda(ids), cuda(w), b_qdesc=q, n=N, out_dtype=od))
            err = np.abs(got - ref)
            assert np.all(err <= _tol(mag, K, k, dtype, True) * (1 + 2.0 ** -8) + _half(od, ref)), err.max()


@pytest.mark.parametrize("tiled", [True, False])
def test_every_code_and_scale(tiled):
    """One-hot activations: each output is one weight, exactly, for every code and the scale bytes 2 .. 252."""
    N, K = 256, 128
    codes = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, K // 2))[None]
    sc = np.stack([np.roll(np.arange(2, 253), 4 * i)[:4] for i in range(256)]).astype(np.uint8)[None]
    W = oracle.fp4_weights(codes, sc)[0]
    b, s = cuda(codes), cuda(sc)
    q = fgg.Q_E2M1_E8M0_1x32
    if tiled:
        b, s = fgg.pack_fp4_weights(b, s)
        q = fgg.Q_E2M1_E8M0_1x32_TILED
    for i in range(0, K, 16):
        x = np.zeros((16, K), np.float32)
        x[np.arange(16), i + np.arange(16)] = 1
        for dt in (torch.bfloat16, torch.float32):
            got = to_np(fgg.moe_gemv_fp4(cuda(x, dt), b, s, b_qdesc=q, n=N, out_dtype=torch.float32))
            np.testing.assert_array_equal(got, W[:, i:i + 16].T.astype(np.float32))


def test_fp32_activations_are_not_rounded():
    """x with all 24 significant bits, extremes included, times weights of one: exact."""
    vals = np.array([1 + 2.0 ** -23, 3.0000002, -1.7777777e30, 1.2345678e-30, 3.4028235e38, 16777215.0, 2.0 ** -100,
                     np.pi], np.float32)
    K = 32
    codes = np.full((1, 4, K // 2), 0x22, np.uint8)          # code 2: the value 1
    sc = np.full((1, 4, 1), 127, np.uint8)
    x = np.zeros((len(vals), K), np.float32)
    x[np.arange(len(vals)), 5] = vals
    got = to_np(fgg.moe_gemv_fp4(cuda(x), cuda(codes), cuda(sc), out_dtype=torch.float32))
    np.testing.assert_array_equal(got, np.tile(vals[:, None], (1, 4)))


def test_inf_and_nan_stay_in_their_token():
    W, b, s, q = _weights(11, 3, 40, 256, False)
    x = _x(12, (5, 256), torch.bfloat16)
    x[1, 7], x[3, 200] = np.nan, np.inf
    ids = np.array([[0, 1], [1, 2], [0, 2], [2, 1], [1, 0]], np.int32)
    for dt in (torch.bfloat16, torch.float32):
        got = to_np(fgg.moe_gemv_fp4(cuda(x, dt), b, s, cuda(ids), torch.ones(5, 2, device="cuda")))
        clean = to_np(fgg.moe_gemv_fp4(cuda(np.nan_to_num(x, posinf=0), dt), b, s, cuda(ids),
                                       torch.ones(5, 2, device="cuda")))
        assert np.isnan(got[1]).all() and not np.isfinite(got[3]).all()
        np.testing.assert_array_equal(got[[0, 2, 4]], clean[[0, 2, 4]])


def test_the_same_bits_every_time():
    G, N, K, T, k = 6, 96, 1024, 9, 3
    _, b, s, q = _weights(13, G, N, K, False)
    bt, st = fgg.pack_fp4_weights(b, s)
    x, ids = cuda(_x(14, (T, K), torch.bfloat16), torch.bfloat16), cuda(_ids(15, T, G, k))
    w = torch.rand(T, k, device="cuda")
    for kw in (dict(), dict(topk_w=w), dict(silu_mul=True)):
        n = N // 2 if "silu_mul" in kw else N
        for args, more in (((b, s), dict()), ((bt, st), dict(b_qdesc=fgg.Q_E2M1_E8M0_1x32_TILED, n=n))):
            a = fgg.moe_gemv_fp4(x, *args, ids, out_dtype=torch.float32, **more, **kw)
            for _ in range(3):
                assert torch.equal(a, fgg.moe_gemv_fp4(x, *args, ids, out_dtype=torch.float32, **more, **kw))


def test_strided_activations_and_output():
    W, b, s, q = _weights(16, 1, 50, 192, False)
    x = cuda(_x(17, (7, 192), torch.bfloat16), torch.bfloat16)
    want = fgg.moe_gemv_fp4(x, b, s)
    wide = torch.full((7, 205), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 3:195] = x
    out = torch.full((7, 61), 9.0, dtype=torch.bfloat16, device="cuda")
    fgg.moe_gemv_fp4(wide[:, 3:195], b, s, out=out[:, 5:55])
    assert torch.equal(out[:, 5:55], want) and (out[:, :5] == 9).all() and (out[:, 55:] == 9).all()


def test_no_tokens():
    _, b, s, q = _weights(18, 2, 16, 32, False)
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    assert fgg.moe_gemv_fp4(x, b, s, torch.empty(0, 2, dtype=torch.int32, device="cuda")).shape == (0, 2, 16)
