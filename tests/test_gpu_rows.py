"""GPU parity of the permuted rows in the activations' own type, the way back,
and their gradients, against the float64 oracle.

Tolerances (u = 2^-24): a weighted row is one fp32 product; a token's sum is k
fused multiply-adds, k u of the sum of magnitudes; a dot product is per-thread
chains of at most N/256 rounded up to whole passes (16 elements) joined by 8
additions, (N/128 + 32) u of the sum of magnitudes covers it; a bf16 result adds half
a step, 2^-8 of it.  Unweighted rows are copies, bit for bit."""

import numpy as np
import pytest
import torch

import fp4_grouped_gemm_amd as fgg
import oracle
import synth
from _util import cuda, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SHAPES = [(1, 1, 1, 1), (1, 8, 256, 2048), (5, 2, 3, 7), (33, 3, 5, 515), (64, 2, 4, 4096), (17, 64, 90, 129),
          (300, 4, 16, 1001), (9, 8, 64, 8200), (130, 6, 8, 1023), (3, 1, 2, 16384), (41, 5, 7, 8), (70, 2, 3, 12), (66, 8, 9, 500), (10, 3, 4, 513),
          (10, 3, 4, 1025)]


def _half(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 0.0


def _case(seed, T, k, E, N, dtype, drop=0.2):
    g = synth.rng(seed)
    ids = np.stack([g.permutation(max(E, k))[:k] for _ in range(T)]).astype(np.int32)
    ids[g.random((T, k)) < drop] = -1
    if T > 2:
        ids[T // 2] = -1                                    # a token without a row
    perm = fgg.moe_permute(cuda(ids), E)
    total = int(perm["offsets"][-1])
    x = g.standard_normal((T, N)).astype(np.float32)
    rows = g.standard_normal((perm["m_cap"], N)).astype(np.float32)
    if dtype == torch.bfloat16:
        x, rows = synth.to_bf16_values(x), synth.to_bf16_values(rows)
    w = g.random((T, k), dtype=np.float32)
    w[ids < 0] = np.nan                                     # weights of dropped pairs are not read
    return ids, perm, total, x, rows, w


def _poison(t, perm, total):
    """NaN in the rows that hold nothing: none of it may reach a token."""
    t = t.clone()
    r2s = perm["row_to_src"]
    t[(r2s < 0).nonzero()[:, 0]] = float("nan")
    return t


@pytest.mark.parametrize("T,k,E,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_permute_rows(T, k, E, N, dtype):
    ids, p, total, x, rows, w = _case(1, T, k, E, N, dtype)
    s2r, M = to_np(p["src_to_row"]), p["m_cap"]
    out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
    got = to_np(fgg.moe_permute_rows(cuda(x, dtype), p["src_to_row"], p["row_to_src"], p["offsets"], out=out))
    np.testing.assert_array_equal(got, oracle.rows_from_tokens(x, None, s2r, total, np.full((M, N), 3.0)))
    out.fill_(3.0)
    got = to_np(fgg.moe_permute_rows(cuda(x, dtype), p["src_to_row"], p["row_to_src"], p["offsets"], topk_w=cuda(w),
                                     out=out))
    ref = oracle.rows_from_tokens(x, w, s2r, total, np.full((M, N), 3.0))
    assert np.all(np.abs(got - ref) <= (U + _half(dtype)) * np.abs(ref) * (1 + U))


@pytest.mark.parametrize("T,k,E,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_unpermute_rows(T, k, E, N, dtype):
    ids, p, total, x, rows, w = _case(2, T, k, E, N, dtype)
    s2r = to_np(p["src_to_row"])
    d = _poison(cuda(rows, dtype), p, total)
    for wt in (None, w):
        got = to_np(fgg.moe_unpermute_rows(d, p["src_to_row"], T, topk_w=None if wt is None else cuda(wt)))
        ref = oracle.tokens_from_rows(rows, wt, s2r, T)
        mag = oracle.tokens_from_rows(np.abs(rows), None if wt is None else np.abs(wt), s2r, T)
        assert np.all(np.abs(got - ref) <= k * U * mag * (1 + _half(dtype)) + _half(dtype) * np.abs(ref))
        assert (got[(ids < 0).all(1)] == 0).all()


@pytest.mark.parametrize("T,k,E,N", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients(T, k, E, N, dtype):
    ids, p, total, x, rows, w = _case(3, T, k, E, N, dtype)
    s2r, M = to_np(p["src_to_row"]), p["m_cap"]
    xd, rd, wd = cuda(x, dtype), _poison(cuda(rows, dtype), p, total), cuda(w)
    dots = oracle.pair_dots(x, rows, s2r)
    tol = (N / 128 + 32) * U * oracle.pair_dots(np.abs(x), np.abs(rows), s2r)
    for wt, wg in ((None, None), (w, wd)):
        # permute: rows are the incoming gradient, x the forward's input
        dx, dw = fgg.moe_permute_rows_backward(rd, p["src_to_row"], T, topk_w=wg, x=xd)
        ref = oracle.tokens_from_rows(rows, wt, s2r, T)
        mag = oracle.tokens_from_rows(np.abs(rows), None if wt is None else np.abs(wt), s2r, T)
        assert np.all(np.abs(to_np(dx) - ref) <= k * U * mag * (1 + _half(dtype)) + _half(dtype) * np.abs(ref))
        assert np.all(np.abs(to_np(dw) - dots) <= tol)
        alone, none = fgg.moe_permute_rows_backward(rd, p["src_to_row"], T, topk_w=wg)
        assert none is None and torch.equal(alone, dx)
        # unpermute: x is the incoming gradient, rows the forward's input
        out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
        dr, dw = fgg.moe_unpermute_rows_backward(xd, p["src_to_row"], p["row_to_src"], p["offsets"], topk_w=wg,
                                                 rows=rd, out=out)
        ref = oracle.rows_from_tokens(x, wt, s2r, total, np.full((M, N), 3.0))
        assert np.all(np.abs(to_np(dr) - ref) <= (U + _half(dtype)) * np.abs(ref) * (1 + U))
        assert np.all(np.abs(to_np(dw) - dots) <= tol)
        out = torch.full((M, N), 3.0, dtype=dtype, device="cuda")
        alone, none = fgg.moe_unpermute_rows_backward(xd, p["src_to_row"], p["row_to_src"], p["offsets"], topk_w=wg,
                                                      out=out)
        assert none is None and torch.equal(alone, dr)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [1, 3, 5, 9, 13, 250, 500, 515, 1027, 2049])
def test_infinities_at_every_end_of_a_row(N, dtype):
    """One row holds an infinity in column c, the token a one everywhere: the product is that
    infinity, not a NaN, whichever columns are loaded twice; the other way round alike."""
    cols = sorted({c for c in [0, 1, 2] + list(range(N - 18, N)) if 0 <= c < N})
    T = len(cols)
    p = fgg.moe_permute(cuda(np.zeros((T, 1), np.int32)), 1)
    s2r = p["src_to_row"]
    x, rows = torch.ones(T, N, device="cuda"), torch.ones(p["m_cap"], N, device="cuda")
    w = torch.ones(T, 1, device="cuda")
    for inf_in_rows in (True, False):
        a, b = x.clone(), rows.clone()
        for t, c in enumerate(cols):
            if inf_in_rows:
                b[s2r[t].long(), c] = float("inf")
            else:
                a[t, c] = float("inf")
        a, b = a.to(dtype), b.to(dtype)
        _, dw = fgg.moe_permute_rows_backward(b, s2r, T, topk_w=w, x=a)
        assert (dw == float("inf")).all()
        _, dw = fgg.moe_unpermute_rows_backward(a, s2r, p["row_to_src"], p["offsets"], topk_w=w, rows=b)
        assert (dw == float("inf")).all()


def test_combine_bit_for_bit():
    ids, p, total, x, rows, w = _case(4, 200, 6, 32, 1000, torch.bfloat16)
    d = cuda(rows, torch.bfloat16)
    w = np.nan_to_num(w)
    assert torch.equal(fgg.moe_unpermute_rows(d, p["src_to_row"], 200, topk_w=cuda(w)),
                       fgg.moe_combine(d, p["src_to_row"], cuda(w)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N", [6, 264, 1005])
def test_strides_and_offsets(dtype, N):
    """Rows inside wider buffers, at every element offset: the columns beside them are neither read nor written."""
    T, k, E = 23, 3, 4
    ids, p, total, x, rows, w = _case(5, T, k, E, N, dtype)
    s2r, M = p["src_to_row"], p["m_cap"]
    dense = fgg.moe_permute_rows(cuda(x, dtype), s2r, p["row_to_src"], p["offsets"], topk_w=cuda(w))
    back = fgg.moe_unpermute_rows(cuda(rows, dtype), s2r, T, topk_w=cuda(w))
    for at in (0, 1, 3, 8):
        wide = torch.full((T, N + 11), float("nan"), dtype=dtype, device="cuda")
        wide[:, at:at + N] = cuda(x, dtype)
        out = torch.full((M, N + 13), 5.0, dtype=dtype, device="cuda")
        fgg.moe_permute_rows(wide[:, at:at + N], s2r, p["row_to_src"], p["offsets"], topk_w=cuda(w),
                             out=out[:, at:at + N])
        assert torch.equal(out[:total, at:at + N], dense[:total])
        assert (out[:, :at] == 5).all() and (out[:, at + N:] == 5).all() and (out[total:] == 5).all()
        wide = torch.full((M, N + 11), float("nan"), dtype=dtype, device="cuda")
        wide[:, at:at + N] = cuda(rows, dtype)
        out = torch.full((T, N + 9), 5.0, dtype=dtype, device="cuda")
        fgg.moe_unpermute_rows(wide[:, at:at + N], s2r, T, topk_w=cuda(w), out=out[:, at:at + N])
        assert torch.equal(out[:, at:at + N], back)
        assert (out[:, :at] == 5).all() and (out[:, at + N:] == 5).all()


def test_a_buffer_too_small_drops_rows():
    T, k, E, N = 40, 4, 3, 100
    g = synth.rng(6)
    ids = g.integers(0, E, size=(T, k)).astype(np.int32)    # an expert may stand twice in a token
    x = g.standard_normal((T, N)).astype(np.float32)
    p = fgg.moe_permute(cuda(ids), E, m_cap=200)
    assert int(p["offsets"][-1]) > 200
    s2r = to_np(p["src_to_row"])
    assert (s2r < 0).any()
    got = fgg.moe_permute_rows(cuda(x), p["src_to_row"], p["row_to_src"], p["offsets"])
    np.testing.assert_array_equal(to_np(got), oracle.rows_from_tokens(x, None, s2r, 200, np.zeros((200, N))))
    # a map made for a larger buffer: the pairs past this one are skipped
    full = fgg.moe_permute(cuda(ids), E)
    s2r = to_np(full["src_to_row"])
    rows = g.standard_normal((200, N)).astype(np.float32)
    got = to_np(fgg.moe_unpermute_rows(cuda(rows), full["src_to_row"], T))
    ref = oracle.tokens_from_rows(rows, None, s2r, T)
    assert np.abs(got - ref).max() <= k * U * np.abs(rows).max() * k


def test_no_tokens_and_no_rows():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    r2s = torch.full((6,), -1, dtype=torch.int32, device="cuda")
    out = torch.full((6, 16), 2.0, device="cuda")
    fgg.moe_permute_rows(x, e, r2s, off, out=out)
    assert (out == 2).all()
    assert fgg.moe_unpermute_rows(out, e, 0).shape == (0, 16)
    # tokens, but no room for any row
    none = torch.full((10,), -1, dtype=torch.int32, device="cuda")
    x = torch.randn(5, 16, device="cuda")
    assert fgg.moe_permute_rows(x, none, e, off).shape == (0, 16)
    assert (fgg.moe_unpermute_rows(torch.empty(0, 16, device="cuda"), none, 5) == 0).all()
    dr, dw = fgg.moe_unpermute_rows_backward(x, none, e, off, rows=torch.empty(0, 16, device="cuda"))
    assert dr.shape == (0, 16) and (dw == 0).all()
    dx, dw = fgg.moe_permute_rows_backward(torch.empty(0, 16, device="cuda"), none, 5, x=x)
    assert (dx == 0).all() and (dw == 0).all()


def test_rows_in_a_graph_and_twice_the_same():
    T, k, E, N = 70, 4, 8, 2056
    ids, p, total, x, rows, w = _case(7, T, k, E, N, torch.bfloat16)
    xd, rd, wd = cuda(x, torch.bfloat16), cuda(rows, torch.bfloat16), cuda(np.nan_to_num(w))

    def step():
        r = fgg.moe_permute_rows(xd, p["src_to_row"], p["row_to_src"], p["offsets"])
        y = fgg.moe_unpermute_rows(r, p["src_to_row"], T, topk_w=wd)
        dr, dw = fgg.moe_unpermute_rows_backward(xd, p["src_to_row"], p["row_to_src"], p["offsets"], topk_w=wd, rows=rd)
        dx, dv = fgg.moe_permute_rows_backward(rd, p["src_to_row"], T, topk_w=wd, x=xd)
        return r[:total], y, dr[:total], dw, dx, dv

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(3):
        xd.mul_(1.5 if i else 1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(held, step()):
            assert torch.equal(a, b)
