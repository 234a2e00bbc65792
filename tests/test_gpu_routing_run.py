"""The routing operators used together: a training step of an expert layer whose
gradients are compared with float64 automatic differentiation of the same layer,
and the generation step's layer (router, gate-up with SiLU, down with the
gate-weighted sum) against the float64 oracle.

Tolerances: the training step runs in fp32 throughout; its gradients pass three
matrix products of at most 64 terms, and four of the operators (each within
about (64 + R) 2^-24 of the magnitude of its terms): 1e-4 of the largest
element of each gradient is over five times the sum of those.  The
generation step keeps h in bf16 (half a step, 2^-8 relative to each element, and
the fp32 sums' share, far below it: twice that is allowed); the error of a sum of K
such products is at most that part of the sum of their magnitudes, the
oracle's second result."""

import numpy as np
import pytest
import torch

import fp4_grouped_gemm_amd as fgg
import oracle
import synth
from _util import cuda, to_np

pytestmark = pytest.mark.gpu


def _experts(rows, offsets, w1):
    out = torch.zeros(rows.shape[0], w1.shape[2], dtype=rows.dtype, device=rows.device)
    for e in range(w1.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        out[a:b] = rows[a:b] @ w1[e]
    return out


@pytest.mark.parametrize("gate,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
@pytest.mark.parametrize("T,k", [(1, 1), (37, 2), (150, 4)])
def test_training_step(gate, renorm, T, k):
    E, N, H = 6, 64, 56
    g = torch.Generator().manual_seed(T + k)
    x = torch.randn(T, N, generator=g)
    wr = torch.randn(N, E, generator=g) * 0.2
    w1 = torch.randn(E, N, H, generator=g) * 0.1
    bias = torch.randn(E, generator=g) * 0.1
    dout = torch.randn(T, H, generator=g)

    # forward and backward by the framework's calls
    xd, wrd, w1d, dd = x.cuda(), wr.cuda(), w1.cuda(), dout.cuda()
    logits = xd @ wrd
    ids, tw = fgg.moe_route(logits, k, gate, bias=bias.cuda(), renormalize=renorm, scale=1.25)
    p = fgg.moe_permute(ids, E)
    maps = (p["src_to_row"], p["row_to_src"], p["offsets"])
    rows = fgg.moe_permute_rows(xd, *maps, out=torch.zeros(p["m_cap"], N, device="cuda"))
    y = _experts(rows, p["offsets"], w1d)
    out = fgg.moe_unpermute_rows(y, p["src_to_row"], T, topk_w=tw)
    dy, dtw = fgg.moe_unpermute_rows_backward(dd, *maps, topk_w=tw, rows=y, out=torch.zeros_like(y))
    drows = _experts(dy, p["offsets"], w1d.transpose(1, 2))
    off = p["offsets"].tolist()
    dw1 = torch.stack([rows[off[e]:off[e + 1]].t() @ dy[off[e]:off[e + 1]] for e in range(E)])
    dx, _ = fgg.moe_permute_rows_backward(drows, p["src_to_row"], T)
    dlogits = fgg.moe_route_backward(logits, ids, dtw, gate, renorm, 1.25)
    dx = dx + dlogits @ wrd.t()
    dwr = xd.t() @ dlogits

    # the layer from its definition, in float64
    X, WR, W1 = (t.double().requires_grad_() for t in (x, wr, w1))
    L = X @ WR
    s = torch.softmax(L, 1) if gate == "softmax" else torch.sigmoid(L)
    at = ids.cpu().long()
    w = torch.gather(s, 1, at)
    w = 1.25 * (w / w.sum(1, keepdim=True) if renorm else w)
    want = sum(w[:, j:j + 1] * torch.bmm(X[:, None], W1[at[:, j]])[:, 0] for j in range(k))
    want.backward(dout.double())
    key = s + bias.double()
    assert torch.equal(at, torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k])
    for got, ref in ((out, want), (dx, X.grad), (dw1, W1.grad), (dwr, WR.grad)):
        ref = ref.detach().numpy()
        assert np.abs(to_np(got) - ref).max() <= 1e-4 * max(np.abs(ref).max(), 1e-3)


def test_permuted_order_is_bypassed_the_same_way():
    """permute_rows then unpermute_rows with unit weights: k times the token, exactly, for small integers."""
    T, k, E, N = 90, 4, 12, 130
    ids = torch.stack([torch.randperm(E)[:k] for _ in range(T)]).int().cuda()
    x = torch.randint(-8, 9, (T, N), device="cuda").bfloat16()
    p = fgg.moe_permute(ids, E)
    rows = fgg.moe_permute_rows(x, p["src_to_row"], p["row_to_src"], p["offsets"])
    assert torch.equal(fgg.moe_unpermute_rows(rows, p["src_to_row"], T), x * k)


@pytest.mark.parametrize("T,tiled", [(1, True), (3, False), (16, True)])
def test_generation_step(T, tiled):
    E, k, K, I = 12, 3, 256, 128
    g = synth.rng(T)
    x = synth.to_bf16_values(g.standard_normal((T, K)).astype(np.float32))
    wr = (g.standard_normal((K, E)) * 0.1).astype(np.float32)
    up = (g.standard_normal((E, 2 * I, K)) * 0.1).astype(np.float32)
    down = (g.standard_normal((E, K, I)) * 0.1).astype(np.float32)

    def weights(w):
        q = [fgg.quantize_blockwise(cuda(w[e]), fgg.Q_E2M1_E8M0_1x32) for e in range(E)]
        b, s = torch.stack([c for c, _ in q]), torch.stack([c for _, c in q])
        vals = oracle.fp4_weights(to_np(b), to_np(s))
        if tiled:
            return vals, (*fgg.pack_fp4_weights(b, s),), dict(b_qdesc=fgg.Q_E2M1_E8M0_1x32_TILED)
        return vals, (b, s), {}

    uv, ub, uq = weights(up)
    dv, db, dq = weights(down)
    xd, wrd = cuda(x, torch.bfloat16), cuda(wr)

    def step(xd):
        logits = xd.float() @ wrd
        ids, w = fgg.moe_route(logits, k, renormalize=True)
        h = fgg.moe_gemv_fp4(xd, *ub, topk_ids=ids, n=I, silu_mul=True, **uq)
        return ids, w, h, fgg.moe_gemv_fp4(h, *db, topk_ids=ids, topk_w=w, n=K, out_dtype=torch.float32, **dq)

    ids, w, h, out = step(xd)
    ref_h = oracle.moe_gemv_fp4(x, uv, to_np(ids), silu_mul=True)[0]
    assert np.abs(to_np(h) - ref_h).max() <= 2.0 ** -7 * np.abs(ref_h).max()
    ref, mag = oracle.moe_gemv_fp4(ref_h, dv, to_np(ids), w=to_np(w))
    assert np.all(np.abs(to_np(out) - ref) <= 2.0 ** -7 * mag)

    # the same step captured once and replayed on other tokens, eager work in between
    held = xd.clone()
    step(held)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(held)
    for seed in range(3):
        held.copy_(cuda(synth.rng(50 + seed).standard_normal((T, K)).astype(np.float32)))
        graph.replay()
        eager = step(held)
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


def test_two_calls_at_once():
    """Two streams run the calls side by side: nothing is shared between them."""
    T, G, k, K, N = 16, 16, 4, 512, 256
    g = synth.rng(3)
    b = cuda(g.integers(0, 256, size=(G, N, K // 2), dtype=np.uint8))
    s = cuda(g.integers(120, 128, size=(G, N, K // 32), dtype=np.uint8))
    cases = []
    for i in range(2):
        x = torch.randn(T, K, device="cuda").bfloat16()
        logits = torch.randn(T, G, device="cuda")
        ids, w = fgg.moe_route(logits, k)
        cases.append((x, logits, ids, w, fgg.moe_gemv_fp4(x, b, s, ids, w)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(20):
        for i, (x, logits, ids, w, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                a, c = fgg.moe_route(logits, k)
                got[i].append((a, c, fgg.moe_gemv_fp4(x, b, s, a, c)))
    torch.cuda.synchronize()
    for i, (x, logits, ids, w, out) in enumerate(cases):
        for a, c, o in got[i]:
            assert torch.equal(a, ids) and torch.equal(c, w) and torch.equal(o, out)
