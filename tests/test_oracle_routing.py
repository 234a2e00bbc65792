"""Pins of the routing oracle: hand-worked selections, gradients against
differences of the oracle's own forward, the rows against the permute's maps,
the 4-bit products against a loop."""

import numpy as np
import pytest

import oracle
import synth


def test_route_by_hand():
    x = np.array([[1.0, 3.0, 3.0, 2.0], [-np.inf, 0.0, -np.inf, -np.inf], [-np.inf] * 4, [0.0, -0.0, 0.0, 0.0]])
    ids, w = oracle.moe_route(x, 2)
    assert ids.tolist() == [[1, 2], [1, -1], [-1, -1], [0, 1]]
    e = np.exp(x[0])
    np.testing.assert_allclose(w[0], e[[1, 2]] / e.sum(), rtol=1e-14)
    assert w[1].tolist() == [1.0, 0.0] and w[2].tolist() == [0.0, 0.0] and w[3].tolist() == [0.25, 0.25]
    ids, w = oracle.moe_route(x, 2, gate="sigmoid", bias=np.array([5.0, 0, 0, 0]), renormalize=True, scale=2.0)
    assert ids[0].tolist() == [0, 1]                      # the bias lifts expert 0 ...
    s = 1 / (1 + np.exp(-x[0]))
    np.testing.assert_allclose(w[0], 2 * s[[0, 1]] / s[[0, 1]].sum(), rtol=1e-14)   # ... and stays out of the weights


@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(gate, renorm):
    g = synth.rng(5)
    T, E, k = 4, 7, 3
    x = g.standard_normal((T, E))
    x[1, 2:] = -np.inf
    ids, _ = oracle.moe_route(x, k, gate)
    ids[3] = [4, 4, 1]                                    # a repeated id counts twice
    dw = g.standard_normal((T, k))
    got = oracle.moe_route_backward(x, ids, dw, gate, renorm, 1.5)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            if np.isneginf(x[t, e]):
                assert got[t, e] == 0
                continue
            hi, lo = x.copy(), x.copy()
            hi[t, e] += h
            lo[t, e] -= h
            d = ((oracle.gate_weights(hi, ids, gate, renorm, 1.5) - oracle.gate_weights(lo, ids, gate, renorm, 1.5))
                 * dw).sum() / (2 * h)
            assert abs(d - got[t, e]) < 1e-8, (t, e)


def test_rows_are_the_permute_and_its_transpose():
    g = synth.rng(6)
    T, k, E, N = 11, 3, 4, 5
    ids = g.integers(-1, E, size=(T, k))
    p = oracle.moe_permute(ids, E, 8)
    total = int(p["offsets"][-1])
    M = total + 3
    x, w = g.standard_normal((T, N)), g.standard_normal((T, k))
    rows = oracle.rows_from_tokens(x, w, p["src_to_row"], total, np.full((M, N), 7.0))
    for r in range(total):
        s = p["row_to_src"][r]
        want = np.zeros(N) if s < 0 else w.reshape(-1)[s] * x[s // k]
        np.testing.assert_array_equal(rows[r], want)
    assert (rows[total:] == 7).all()
    # <permute(x), d> = <x, unpermute(d)>: the backward is the transpose
    d = g.standard_normal((M, N))
    d[total:] = 0
    back = oracle.tokens_from_rows(d, w, p["src_to_row"], T)
    np.testing.assert_allclose((rows * d).sum(), (x * back).sum(), rtol=1e-12)
    # and the weights' gradient is the derivative of the same product
    dots = oracle.pair_dots(x, d, p["src_to_row"])
    np.testing.assert_allclose((rows * d).sum(), (w * dots).sum(), rtol=1e-12)


def test_gemv_against_a_loop():
    g = synth.rng(7)
    G, N, K, T, k = 3, 6, 64, 2, 2
    codes = g.integers(0, 256, size=(G, N, K // 2), dtype=np.uint8)
    sc = g.integers(120, 132, size=(G, N, K // 32), dtype=np.uint8)
    W = oracle.fp4_weights(codes, sc)
    table = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    for e in range(G):
        for n in range(N):
            for i in range(K):
                c = (codes[e, n, i // 2] >> (4 * (i % 2))) & 15
                assert W[e, n, i] == table[c] * 2.0 ** (int(sc[e, n, i // 32]) - 127)
    x = g.standard_normal((T, K))
    ids = np.array([[2, 0], [1, 5]], dtype=np.int32)
    w = np.array([[0.25, 0.5], [1.0, np.nan]])
    y, _ = oracle.moe_gemv_fp4(x, W, ids)
    np.testing.assert_allclose(y[0, 0], [sum(W[2, n, i] * x[0, i] for i in range(K)) for n in range(N)], rtol=1e-12)
    assert (y[1, 1] == 0).all()
    s, _ = oracle.moe_gemv_fp4(x, W, ids, w=w)
    np.testing.assert_allclose(s[0], 0.25 * y[0, 0] + 0.5 * y[0, 1], rtol=1e-12)
    np.testing.assert_allclose(s[1], y[1, 0], rtol=1e-12)
