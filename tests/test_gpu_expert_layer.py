"""The operators of a feed-forward layer used together: a training step of an expert layer in bf16
(router, rows in expert order, gated block, down projection, weighted sum, and every gradient)
against float64 automatic differentiation; a dense layer whose projections carry adapters; the same
captured in a graph and replayed; calls on two streams at once and on another stream than the
current one.

Tolerance of the training step: every tensor that passes from call to call is rounded to bf16
(half a step, 2^-8 relative to each element).  A gradient passes at most six such roundings (x rows, h,
a, dy, dh, dx); each moves a product's sum by at most 2^-8 of the norm of its terms, so six of them
stay within 6 * 2^-8 = 2.4 % of the gradient's norm; rounding errors are independent, so the norm of
the difference is far below that bound, which is what is asserted (Frobenius norms)."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32

pytestmark = pytest.mark.gpu
BOUND = 6 * 2.0 ** -8


def near(got, ref, what, bound=BOUND):
    got, ref = got.double(), ref.detach().double().to(got.device)
    assert torch.isfinite(got).all(), what
    off = float((got - ref).norm() / ref.norm().clamp_min(1e-30))
    assert off <= bound, f"{what}: {off:.3g}"


@pytest.mark.parametrize("T,k,E,D,I,align", [(1, 2, 4, 64, 40, 128), (37, 2, 6, 72, 136, 1), (300, 3, 8, 264, 200, 128),
                                             (700, 2, 5, 520, 392, 8)])
def test_training_step(T, k, E, D, I, align):
    g = torch.Generator().manual_seed(T)
    x = torch.randn(T, D, generator=g).to(BF16)
    wr = (torch.randn(D, E, generator=g) * 0.2)
    w1 = (torch.randn(E, 2 * I, D, generator=g) * D ** -0.5).to(BF16)
    w2 = (torch.randn(E, D, I, generator=g) * I ** -0.5).to(BF16)
    dout = torch.randn(T, D, generator=g).to(BF16)
    xd, wrd, w1d, w2d, dd = (t.cuda() for t in (x, wr, w1, w2, dout))

    logits = xd.float() @ wrd
    ids, tw = fgg.moe_route(logits, k, renormalize=True)
    p = fgg.moe_permute(ids, E, align)
    maps = (p["src_to_row"], p["row_to_src"], p["offsets"])
    seg = dict(offsets=p["offsets"], counts=p["counts"])
    M = p["m_cap"]
    # what no call writes holds NaN: nothing may read it
    empty = (lambda n: torch.full((M, n), float("nan"), dtype=BF16, device="cuda"))
    rows = fgg.moe_permute_rows(xd, *maps, out=empty(D))
    a, h = fgg.grouped_gated(rows, w1d, **seg, out=empty(I), h=empty(2 * I))
    y = fgg.grouped_linear(a, w2d, **seg, out=empty(D))
    out = fgg.moe_unpermute_rows(y, p["src_to_row"], T, topk_w=tw)

    dy, dtw = fgg.moe_unpermute_rows_backward(dd, *maps, topk_w=tw, rows=y, out=empty(D))
    dh, again = fgg.grouped_gated_backward(dy, w2d, h, **seg, out=empty(2 * I), a=empty(I))
    dw2 = fgg.grouped_linear_backward_weight(dy, again, E, **seg)
    dw1 = fgg.grouped_linear_backward_weight(dh, rows, E, **seg)
    drows = fgg.grouped_linear_backward_input(dh, w1d, **seg, out=empty(D))
    dx, _ = fgg.moe_permute_rows_backward(drows, p["src_to_row"], T)
    dlogits = fgg.moe_route_backward(logits, ids, dtw, renormalize=True)
    dwr = xd.float().t() @ dlogits

    X, WR, W1, W2 = (t.double().requires_grad_() for t in (x, wr, w1, w2))
    at = ids.cpu().long()
    # (the router's path into x is left out here: its gradient is checked by dwr)
    w_x = torch.softmax(torch.gather(x.double() @ WR, 1, at), 1)
    want = 0
    for j in range(k):
        hh = torch.bmm(W1[at[:, j]], X[:, :, None])[:, :, 0]
        aa = hh[:, :I] * torch.sigmoid(hh[:, :I]) * hh[:, I:]
        want = want + w_x[:, j:j + 1] * torch.bmm(W2[at[:, j]], aa[:, :, None])[:, :, 0]
    want.backward(dout.double())
    near(out, want, "out")
    near(dx, X.grad, "dx")
    near(dw1, W1.grad, "dw1")
    near(dw2, W2.grad, "dw2")
    # (dlogits passes the dot products of y's rounded rows, whose shares cancel in the softmax's gradient)
    near(dwr, WR.grad, "dwr", 2 * BOUND)


def layer(x, w1, w2, ids, up, down, h=None):
    """A dense gated block whose output projection and pre-activations carry each token's adapter."""
    h = fgg.grouped_linear(x, w1)
    h = fgg.lora_add(h, x, ids, *up, out=h)
    gate, u = h.chunk(2, 1)
    a = (gate.float() * torch.sigmoid(gate.float()) * u.float()).to(BF16)
    y = fgg.grouped_linear(a, w2, out_dtype=F32)
    return fgg.lora_add(y, a, ids, *down)


def dense_case(T, seed=0, D=264, I=200, L=5, r=16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = (lambda *s, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(BF16))
    x, w1, w2 = n(T, D), n(1, 2 * I, D, scale=D ** -0.5), n(1, D, I, scale=I ** -0.5)
    ids = torch.randint(-1, L, (T,), generator=g, device="cuda").int()
    up = (n(L, r, D, scale=D ** -0.5), n(L, 2 * I, r, scale=0.3), torch.rand(L, generator=g, device="cuda"))
    down = (n(L, r, I, scale=I ** -0.5), n(L, D, r, scale=0.3), None)
    return x, w1, w2, ids, up, down


@pytest.mark.parametrize("T", [1, 16, 130, 700])
def test_adapters_beside_the_products(T):
    x, w1, w2, ids, up, down = dense_case(T)
    got = layer(x, w1, w2, ids, up, down)
    d = (lambda t: t.double())
    pick = (lambda t: torch.where((ids >= 0)[(...,) + (None,) * (t.dim() - 1)], d(t)[ids.clamp_min(0).long()], 0.0))
    h = d(x) @ d(w1[0]).t() + pick(up[2])[:, None] * torch.bmm(pick(up[1]), torch.bmm(pick(up[0]), d(x)[:, :, None]))[:, :, 0]
    gate, u = h.chunk(2, 1)
    a = gate * torch.sigmoid(gate) * u
    want = a @ d(w2[0]).t() + torch.bmm(pick(down[1]), torch.bmm(pick(down[0]), a[:, :, None]))[:, :, 0]
    near(got, want, "layer")


@pytest.mark.parametrize("T", [1, 40, 700])
def test_captured_and_replayed(T):
    """One graph of the dense layer and of a training pass, replayed on other inputs with eager work in between."""
    x, w1, w2, ids, up, down = dense_case(T, 1)
    dy = torch.randn(T, w2.shape[1], device="cuda").to(BF16)

    def step():
        out = layer(x, w1, w2, ids, up, down)
        h = torch.empty(T, w1.shape[1], dtype=BF16, device="cuda")
        a, _ = fgg.grouped_gated(x, w1, h=h)
        dh, again = fgg.grouped_gated_backward(dy, w2, h, a=torch.empty_like(a))
        return (out, a, dh, again, fgg.grouped_linear_backward_input(dh, w1),
                fgg.grouped_linear_backward_weight(dh, x, 1), fgg.grouped_linear_backward_weight(dy, again, 1, out_dtype=BF16))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in range(4):
        new = dense_case(T, 10 + seed)
        x.copy_(new[0]), ids.copy_(new[3])
        dy.copy_(torch.randn(T, dy.shape[1], device="cuda"))
        graph.replay()
        eager = step()
        torch.cuda.synchronize()
        for got, want in zip(captured, eager):
            assert torch.equal(got, want)


def test_two_streams_at_once():
    cases = [dense_case(T, T) for T in (24, 600)]
    want = [layer(*c) for c in cases]
    dys = [torch.randn(c[0].shape[0], c[2].shape[1], device="cuda").to(BF16) for c in cases]
    dws = [fgg.grouped_linear_backward_weight(dy, c[0], 1) for dy, c in zip(dys, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(10):
        for i, c in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append((layer(*c), fgg.grouped_linear_backward_weight(dys[i], c[0], 1)))
    torch.cuda.synchronize()
    for i in range(2):
        for out, dw in got[i]:
            assert torch.equal(out, want[i]) and torch.equal(dw, dws[i])


def test_fewer_workgroups():
    """The persistent shape with another number of compute units set: the same results."""
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(4200, 520, generator=g, device="cuda").to(BF16)
    w = torch.randn(1, 4112, 520, generator=g, device="cuda").to(BF16)
    want = fgg.grouped_linear(x, w)
    try:
        for n in (5, 40, 200, 300):
            fgg.set_num_cus(n)
            assert torch.equal(fgg.grouped_linear(x, w), want), n
    finally:
        fgg.set_num_cus(0)
