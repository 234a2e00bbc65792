"""The bf16 products at the largest counts of rows that the calls take."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


@pytest.fixture(autouse=True)
def room():
    """These tests hold up to 90 GB at a time: what the allocator keeps is given back on both sides."""
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


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


def nonzeros(t):
    return sum(int(torch.count_nonzero(part)) for part in t.split(2 ** 26))


@pytest.mark.parametrize("call", [fgg.grouped_linear, fgg.grouped_linear_backward_input])
@pytest.mark.parametrize("bounds", [None, (5, MOST - 300)])
def test_rows(call, bounds):
    """2^31 - 1 rows of 8 columns: 2^25 of the smallest tiles."""
    M = MOST
    at = torch.tensor([0, 4, 5, 2 ** 28 + 1, 2 ** 30, M - 301, M - 300, M - 256, M - 255, M - 1], device="cuda")
    x = sparse(M, 8, at, 3)
    spans = [(0, M)] if bounds is None else [(0, bounds[0]), bounds, (bounds[1], M)]
    g = torch.Generator(device="cuda").manual_seed(4)
    w = torch.randint(-4, 5, (len(spans), 8, 8), generator=g, device="cuda").to(BF16)
    offsets = None if bounds is None else torch.tensor([0, *bounds, M], dtype=torch.int32, device="cuda")
    y = call(x, w, offsets)
    which = [next(i for i, (s, e) in enumerate(spans) if s <= r < e) for r in at.tolist()]
    ww = w.double() if call is fgg.grouped_linear_backward_input else w.double().transpose(1, 2)
    want = torch.stack([x[r].double() @ ww[i] for r, i in zip(at.tolist(), which)])
    assert torch.equal(y[at].double(), want) and nonzeros(y) == nonzeros(want)


def test_gated_rows():
    M = 2 ** 30 - 5
    at = torch.tensor([0, 77, 2 ** 29 - 1, 2 ** 29, M - 257, M - 1], device="cuda")
    x = sparse(M, 8, at, 5)
    w = torch.zeros(1, 16, 8, dtype=BF16, device="cuda")
    w[0, :8], w[0, 8:] = torch.eye(8, device="cuda"), torch.eye(8, device="cuda").flip(0)
    a, _ = fgg.grouped_gated(x, w)
    gate = x[at].double()
    want = gate * torch.sigmoid(gate) * gate.flip(1)
    assert ((a[at].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -18) * want.abs()).all()
    assert nonzeros(a) == nonzeros(want)
    del a
    h = torch.zeros(M, 16, dtype=BF16, device="cuda")
    h[at] = torch.cat([x[at], x[at].flip(1)], 1)
    dh, _ = fgg.grouped_gated_backward(x, w[:, :8], h)           # (da = x)
    hs = h[at].double().requires_grad_()
    (hs[:, :8] * torch.sigmoid(hs[:, :8]) * hs[:, 8:]).backward(gate)
    # the gate's derivative has two terms that can cancel: for |gate| up to 4 they are below 5 |up| each
    assert ((dh[at].double() - hs.grad).abs() <= 2.0 ** -8 * hs.grad.abs() + 2.0 ** -18 * 10 * 16).all()
    assert nonzeros(dh) <= 16 * len(at)


def test_wide_output():
    """2^35 outputs, 2^23 of the smallest tiles."""
    M, N, K = 2 ** 23, 4096, 64
    g = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda", dtype=torch.int8).to(BF16)
    w = torch.randint(-2, 3, (1, N, K), generator=g, device="cuda").to(BF16)
    y = fgg.grouped_linear(x, w)
    for s in (0, 2 ** 19 - 50, 2 ** 22 - 3, M - 300):
        rows = slice(s, s + 300)
        assert torch.equal(y[rows].double(), x[rows].double() @ w[0].double().t())


def test_many_weight_gradients():
    """600 gradients of 8192 x 8192: 2^23 and more of the smallest tiles, one segment empty."""
    G, N, K = 600, 8192, 8192
    offsets = torch.arange(G + 1, device="cuda", dtype=torch.int32) * 8
    offsets[300] = offsets[301]
    M = 8 * G
    g = torch.Generator(device="cuda").manual_seed(7)
    dy = torch.randint(-2, 3, (M, N), generator=g, device="cuda").to(BF16)
    x = torch.randint(-2, 3, (M, K), generator=g, device="cuda").to(BF16)
    dw = fgg.grouped_linear_backward_weight(dy, x, G, offsets, out_dtype=BF16)
    for e in (0, 299, 300, 301, G - 1):
        s, t = int(offsets[e]), int(offsets[e + 1])
        assert torch.equal(dw[e], (dy[s:t].float().t() @ x[s:t].float()).to(BF16))
        assert bool((dw[e] == 0).all()) == (e == 300)
