"""GPU parity of the router and its gradient against the float64 oracle.

Tolerances (fp32, u = 2^-24): a score is one exponential of a difference (the
difference's rounding is worth |x - max| u relative, the exponential 2u), a sum
of at most 16 + 6 roundings, a division and the scale: (64 + R) u with R the
spread of the logits (at most 104, below which an fp32 exponential is 0).  The
gradient multiplies two such scores and subtracts: twice that, relative to the
sum of the magnitudes of its terms.  A bf16 result adds half a step, 2^-8."""

import numpy as np
import pytest
import torch

import fp4_grouped_gemm_amd as fgg
import oracle
import synth
from _util import cuda, to_np

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 2.0 ** -120


def _logits(seed, T, E, dtype, shut=0.05, spread=2.0):
    g = synth.rng(seed)
    x = (g.standard_normal((T, E)) * spread).astype(np.float32)
    if shut:
        x[g.random((T, E)) < shut] = -np.inf
        x[T // 2] = -np.inf                                # a token without any expert
    if dtype == torch.bfloat16:
        f = np.isfinite(x)
        x[f] = synth.to_bf16_values(x)[f]
    return x


def _spread(x):
    f = x[np.isfinite(x)]
    return min(104.0, float(f.max() - f.min())) if f.size else 0.0


def _check_weights(w, ref, x, what=""):
    tol = (64 + _spread(x)) * U
    assert np.all(np.abs(w - ref) <= tol * np.abs(ref) + TINY), (what, np.abs(w - ref).max())


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (3, 16, 16), (65, 17, 3), (9, 64, 64), (130, 33, 5),
                                   (31, 160, 6), (7, 256, 1), (515, 256, 8), (5, 1000, 64), (2, 1024, 10)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_route(T, E, k, dtype, gate):
    x = _logits(T + E, T, E, dtype)
    bias = (synth.rng(E).standard_normal(E) * 0.1).astype(np.float32)
    d = cuda(x, dtype)
    for b in (None, bias):
        for renorm, scale in ((False, 1.0), (True, 2.5)):
            ids, w = fgg.moe_route(d, k, gate, bias=None if b is None else cuda(b), renormalize=renorm, scale=scale)
            ref_ids, ref_w = oracle.moe_route(x, k, gate, b, renorm, scale)
            assert np.array_equal(to_np(ids), ref_ids), (b is not None, renorm)
            _check_weights(to_np(w), ref_w, x, (b is not None, renorm))


def test_ties_go_to_the_lower_expert():
    x = np.zeros((6, 200), np.float32)
    x[1, ::2] = -0.0
    x[2, 150:] = 1.0
    x[3, [7, 71, 135, 199]] = 3.0                           # the same lane of four registers
    x[4, [64, 1]] = 2.0
    x[5] = -np.inf
    x[5, [190, 5]] = -np.inf
    for b in (None, np.zeros(200, np.float32)):
        ids, _ = fgg.moe_route(cuda(x), 5, bias=None if b is None else cuda(b))
        got = to_np(ids)
        assert got[0].tolist() == got[1].tolist() == [0, 1, 2, 3, 4]
        assert got[2].tolist() == [150, 151, 152, 153, 154]
        assert got[3].tolist() == [7, 71, 135, 199, 0]
        assert got[4].tolist() == [1, 64, 0, 2, 3]
        assert got[5].tolist() == [-1] * 5


@pytest.mark.parametrize("E", [3, 16, 30, 61, 100, 250, 500, 1000])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_keys_that_differ_in_their_low_bits(E, gate):
    """Equal scores, biases 2^-24 apart in [0.5, 1): 32 bits would hold them, the keys' upper halves (20 bits of
    fraction) do not; every third bias repeats the one before, a tie for the lower expert."""
    g = synth.rng(E)
    step = g.permutation(E)
    step[2::3] = step[1::3][:len(step[2::3])]
    bias = (0.5 + step * 2.0 ** -24).astype(np.float32)
    x = np.full((5, E), -1.5, np.float32)
    x[1, E // 2] = 4.0
    x[2, ::2] = -np.inf
    k = min(E, 20)
    ids, w = fgg.moe_route(cuda(x), k, gate, bias=cuda(bias), renormalize=True)
    ref_ids, ref_w = oracle.moe_route(x, k, gate, bias, True, 1.0)
    assert np.array_equal(to_np(ids), ref_ids)
    _check_weights(to_np(w), ref_w, x, gate)


def test_saturated_scores_with_a_bias():
    """Scores that round to 0 or 1, or lie far apart: the bias orders them."""
    x = np.array([[100.0, 50.0, -800.0, -1000.0, 3e38, -3e38, 0.0, 1.0]], np.float32)
    bias = np.array([0.1, 0.2, 0.05, 0.06, 0.15, 0.07, -0.6, -0.7], np.float32)
    for gate in ("softmax", "sigmoid"):
        ids, w = fgg.moe_route(cuda(x), 8, gate, bias=cuda(bias))
        ref_ids, ref_w = oracle.moe_route(x, 8, gate, bias, False, 1.0)
        assert np.array_equal(to_np(ids), ref_ids)
        _check_weights(to_np(w), ref_w, np.array([0.0, 104.0]), gate)


def test_extreme_logits():
    low, top = np.float32(-3e38), np.float32(3e38)
    x = np.array([[low, low, 0, 0], [top, low, 0, 0], [-200, -201, -300, -250], [low, -np.inf, -np.inf, -np.inf],
                  [90, 88, -90, 0]], np.float32)
    for gate in ("softmax", "sigmoid"):
        for renorm in (False, True):
            ids, w = fgg.moe_route(cuda(x), 3, gate, renormalize=renorm)
            ref_ids, ref_w = oracle.moe_route(x, 3, gate, None, renorm)
            assert np.array_equal(to_np(ids), ref_ids)
            _check_weights(to_np(w), ref_w, np.array([0.0, 104.0]), (gate, renorm))


def test_nan_and_inf_logits():
    x = np.array([[1, np.nan, 2, 0], [np.inf, 1, 2, 0], [np.nan] * 4, [1, 2, 3, 4]], np.float32)
    for gate in ("softmax", "sigmoid"):
        for bias in (None, cuda(np.array([0, 0, 0, 0.5], np.float32))):
            ids, w = fgg.moe_route(cuda(x), 2, gate, bias=bias, renormalize=True)
            ids, w = to_np(ids), to_np(w)
            assert 1 not in ids[0] and (ids[0] >= 0).all() and np.isnan(w[0]).all()
            assert ids[2].tolist() == [-1, -1] and (w[2] == 0).all()
            assert ids[3].tolist() == [3, 2] and np.isfinite(w[3]).all()
            assert ids[1, 0] == 0 or (gate == "softmax" and bias is not None)
    # a closed or NaN bias closes the expert
    b = np.array([0, -np.inf, np.nan, 0], np.float32)
    ids, _ = fgg.moe_route(cuda(x[3:]), 4, "sigmoid", bias=cuda(b))
    assert to_np(ids)[0].tolist() == [3, 0, -1, -1]


def test_strided_logits_and_outputs_in_place():
    x = _logits(3, 40, 60, torch.float32, shut=0)
    big = torch.full((40, 77), float("nan"), device="cuda")
    big[:, 5:65] = cuda(x)
    ids = torch.full((40, 4), 99, dtype=torch.int32, device="cuda")
    w = torch.full((40, 4), 99.0, device="cuda")
    fgg.moe_route(big[:, 5:65], 4, ids=ids, weights=w)
    ref_ids, ref_w = oracle.moe_route(x, 4)
    assert np.array_equal(to_np(ids), ref_ids)
    _check_weights(to_np(w), ref_w, x)
    out = torch.full((40, 80), 7.0, device="cuda")
    dw = torch.randn(40, 4, device="cuda")
    fgg.moe_route_backward(big[:, 5:65], ids, dw, out=out[:, 3:63])
    assert torch.equal(out[:, 3:63], fgg.moe_route_backward(cuda(x), ids, dw))
    assert (out[:, :3] == 7).all() and (out[:, 63:] == 7).all()


def _gradient_scale(x, ids, dw, gate, renorm, scale):
    """Sum of the magnitudes of the gradient's terms."""
    s = oracle.gate_weights(x, np.tile(np.arange(x.shape[1]), (x.shape[0], 1)), gate, False)
    w = oracle.gate_weights(x, ids, gate, renorm)
    u = np.abs(scale * dw) * (ids >= 0)
    mean = (u * w).sum(1, keepdims=True)
    out = np.zeros(x.shape)
    for t in range(x.shape[0]):
        for j, e in enumerate(ids[t]):
            if e >= 0:
                out[t, e] += (w[t, j] if renorm else s[t, e]) * (u[t, j] + (mean[t, 0] if renorm else 0))
    return out + (s * mean if gate == "softmax" and not renorm else 0)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 256, 8), (65, 17, 3), (9, 64, 64), (31, 160, 6), (70, 30, 4),
                                   (257, 256, 8), (5, 1000, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward(T, E, k, dtype, gate, renorm):
    x = _logits(T + 2 * E, T, E, dtype)
    ids, _ = oracle.moe_route(x, k, gate)
    if T > 3 and k > 1:
        ids[0, 1] = ids[0, 0]                               # a repeated id
        ids[1, 0] = E + 5                                   # and ids that are no expert's
        ids[2, :] = -1
    dw = synth.rng(T).standard_normal((T, k)).astype(np.float32)
    got = to_np(fgg.moe_route_backward(cuda(x, dtype), cuda(ids), cuda(dw), gate, renorm, 1.5))
    ids = np.where(ids >= E, -1, ids)
    ref = oracle.moe_route_backward(x, ids, dw, gate, renorm, 1.5)
    tol = 2 * (64 + _spread(x)) * U * _gradient_scale(x, ids, dw, gate, renorm, 1.5) + TINY
    if dtype == torch.bfloat16:
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
    assert np.all(got[np.isneginf(x)] == 0)


def test_route_in_a_graph_and_on_another_stream():
    x = cuda(_logits(9, 300, 128, torch.float32))
    bias = torch.randn(128, device="cuda") * 0.1
    want = fgg.moe_route(x, 6, "sigmoid", bias=bias, renormalize=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = fgg.moe_route(x, 6, "sigmoid", bias=bias, renormalize=True)
        grad = fgg.moe_route_backward(x, got[0], got[1], "sigmoid", True)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    held = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ids, w = fgg.moe_route(held, 6, "sigmoid", bias=bias, renormalize=True)
        d = fgg.moe_route_backward(held, ids, w, "sigmoid", True)
    for seed in range(3):
        held.copy_(cuda(_logits(20 + seed, 300, 128, torch.float32)) if seed else x)
        graph.replay()
        torch.cuda.synchronize()
        a, b = fgg.moe_route(held, 6, "sigmoid", bias=bias, renormalize=True)
        assert torch.equal(a, ids) and torch.equal(b, w)
        assert torch.equal(d, fgg.moe_route_backward(held, a, b, "sigmoid", True))
        if seed == 0:
            assert torch.equal(d, grad)


def _by_key(key, k):
    """The k largest keys that are numbers above -inf, ties to the lower expert."""
    key = np.where(np.isnan(key), -np.inf, key)
    ids = np.argsort(-key, kind="stable")[:k]
    return np.where(np.isneginf(key[ids]), -1, ids)


@pytest.mark.parametrize("E", [6, 29, 60, 100, 200, 400, 1000])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_order_of_rows_with_nan_and_inf_and_a_bias(E, gate):
    """Under a softmax a NaN or +inf leaves no score: the other experts are ranked by the bias alone, here
    against the logits' order.  A sigmoid's scores do not depend on one another: the NaN is left out, the
    rest are ranked by score + bias."""
    g = synth.rng(E)
    rise = np.sort(g.standard_normal(E)).astype(np.float32)
    x = np.tile(rise, (6, 1))
    x[0, E // 2] = np.nan
    x[1, E // 3] = np.inf
    x[2, 1], x[2, E - 1] = np.nan, np.inf
    x[3, 0], x[3, 2], x[3, 4] = np.nan, -np.inf, np.nan
    x[4, :E - 2] = np.nan
    bias = np.linspace(0.02, -0.02, E).astype(np.float32)    # (less than the spread of the scores)
    bias[3] = -np.inf
    k = min(E, 12)
    ids, w = fgg.moe_route(cuda(x), k, gate, bias=cuda(bias), renormalize=True)
    ids, w = to_np(ids), to_np(w)
    for t in range(6):
        row = x[t].astype(np.float64)
        if gate == "sigmoid":
            score = oracle.routing.scores(row[None], gate)[0]
        elif np.isnan(row).any() or np.isposinf(row).any():
            score = np.zeros(E)
        else:
            score = oracle.routing.scores(row[None], gate)[0]
        key = np.where(np.isnan(row) | np.isneginf(row), -np.inf, score + bias.astype(np.float64))
        want = _by_key(key, k)
        assert ids[t].tolist() == want.tolist(), t
        nan = np.isnan(row).any() or (gate == "softmax" and np.isposinf(row).any())
        assert (np.isnan(w[t]) if nan else np.isfinite(w[t]))[want >= 0].all() and (w[t][want < 0] == 0).all(), t


@pytest.mark.parametrize("E,k", [(6, 3), (29, 4), (60, 5), (100, 8), (400, 8)])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient_of_a_nan_that_was_chosen(E, k, gate, renorm):
    """Ids that name a NaN logit (the router gives none, a caller may): its weight is a NaN, and so is
    every gradient that the weight enters, all of the token's chosen experts where their weights share a sum."""
    g = synth.rng(E + k)
    x = g.standard_normal((3, E)).astype(np.float32)
    ids = np.stack([g.permutation(E)[:k] for _ in range(3)]).astype(np.int32)
    x[1, ids[1, 1]] = np.nan
    dw = g.standard_normal((3, k)).astype(np.float32)
    got = to_np(fgg.moe_route_backward(cuda(x), cuda(ids), cuda(dw), gate, renorm))
    nan = np.zeros(x.shape, bool)
    if renorm:
        nan[1, ids[1]] = True
    elif gate == "softmax":
        nan[1] = True
    else:
        nan[1, ids[1, 1]] = True
    assert np.array_equal(np.isnan(got), nan)
    clean = x.copy()
    clean[1] = 0
    rest = to_np(fgg.moe_route_backward(cuda(clean), cuda(ids), cuda(dw), gate, renorm))
    assert np.array_equal(got[[0, 2]], rest[[0, 2]])


def _open_case(seed, T, E, k, dtype):
    """Random logits, no row and few experts closed: nearly every slot holds an expert."""
    g = synth.rng(seed)
    x = (g.standard_normal((T, E)) * 2.0).astype(np.float32)
    if dtype == torch.bfloat16:
        x = synth.to_bf16_values(x).astype(np.float32)
    if E > 2 * k:
        x[g.random((T, E)) < 0.05] = -np.inf
    return x


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (1, 40, 4), (1, 64, 6), (1, 100, 8), (1, 256, 8), (1, 384, 8),
                                   (1, 1024, 16),
                                   (7, 65, 4), (33, 100, 6), (130, 128, 8), (5, 127, 60),
                                   (9, 257, 8), (70, 300, 6), (65, 384, 8), (31, 500, 10), (6, 512, 64)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gate", ["softmax", "sigmoid"])
def test_expert_counts(T, E, k, dtype, gate):
    """One token with real logits, and two and eight experts a lane (E 65 to 128, 257 to 512), forward with and
    without a bias and backward, against the oracle."""
    x = _open_case(7 * T + E, T, E, k, dtype)
    bias = (synth.rng(E + 1).standard_normal(E) * 0.1).astype(np.float32)
    d = cuda(x, dtype)
    dw = synth.rng(T + 3).standard_normal((T, k)).astype(np.float32)
    for renorm in (False, True):
        for b in (None, bias):
            ids, w = fgg.moe_route(d, k, gate, bias=None if b is None else cuda(b), renormalize=renorm, scale=1.5)
            ref_ids, ref_w = oracle.moe_route(x, k, gate, b, renorm, 1.5)
            assert (ref_ids >= 0).all()
            assert np.array_equal(to_np(ids), ref_ids)
            _check_weights(to_np(w), ref_w, x, (b is not None, renorm))
        got = to_np(fgg.moe_route_backward(d, cuda(ref_ids), cuda(dw), gate, renorm, 1.5))
        ref = oracle.moe_route_backward(x, ref_ids, dw, gate, renorm, 1.5)
        tol = 2 * (64 + _spread(x)) * U * _gradient_scale(x, ref_ids, dw, gate, renorm, 1.5) + TINY
        if dtype == torch.bfloat16:
            tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref)
        assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
        assert E == 1 or k == E or renorm and k == 1 or np.count_nonzero(ref) >= k
