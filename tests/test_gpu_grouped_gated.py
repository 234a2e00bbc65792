"""The gated block (both projections, SiLU and the product) and its gradient against float64."""

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, HALF, gated, matrix, poison, product, segments, spans, within

pytestmark = pytest.mark.gpu

# rows, segments, I, K
SIZES = [(1, 1, 8, 8), (3, 2, 24, 40), (16, 6, 136, 264), (130, 1, 128, 64), (259, 3, 200, 72), (700, 5, 392, 520),
         (900, 40, 72, 328), (513, 1, 1000, 136)]
# silu and its derivative are within |g| 2^-23 (exponential), a few 2^-24 otherwise: 2^-18 for |g| to 32
ACT = 2.0 ** -18


def case(M, G, padded, seed):
    g = torch.Generator(device="cuda").manual_seed(seed + M)
    offsets, counts, rows = segments(G, M, seed + G, padded)
    if G == 1 and not padded:
        offsets = counts = None
    return g, offsets, counts, rows, [(0, M)] if offsets is None else spans(offsets, counts, rows)


@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("M,G,I,K", SIZES)
def test_forward(M, G, I, K, padded, keep):
    g, offsets, counts, rows, sp = case(M, G, padded, 3)
    x = matrix(g, rows, K, K + 8)
    w = (torch.randn(G, 2 * I, K, generator=g, device="cuda") * (2.0 / K ** 0.5)).to(BF16)
    live = poison(x, sp)
    out = matrix(g, rows, I, I + 8 * (M % 2))
    h = matrix(g, rows, 2 * I, 2 * I + 8) if keep else None
    a0, h0 = out.clone(), None if h is None else h.clone()
    a, hh = fgg.grouped_gated(x, w, offsets, counts, out=out, h=h)
    assert a is out and hh is h and torch.equal(a[~live], a0[~live])
    if keep:
        assert torch.equal(h[~live], h0[~live])
    for e, (s, t) in enumerate(sp):
        if t == s:
            continue
        ref, bound = product(x[s:t], w[e].t(), BF16)
        if keep:
            within(h[s:t], ref, bound, f"pre-activations of segment {e}")
        off = bound - HALF[BF16] * ref.abs()                   # the fp32 sums' share: a is formed from them
        gate, up = ref.chunk(2, dim=1)
        silu = gate * torch.sigmoid(gate)
        ref_a = silu * up
        moved = 1.1 * up.abs() * off[:, :I] + silu.abs() * off[:, I:] + 1.1 * off[:, :I] * off[:, I:]
        within(a[s:t], ref_a, (HALF[BF16] + ACT) * ref_a.abs() + 1.01 * moved + 1e-38, f"segment {e}")


@pytest.mark.parametrize("with_a", [False, True])
@pytest.mark.parametrize("padded", [False, True])
@pytest.mark.parametrize("M,G,I,N", SIZES)
def test_backward(M, G, I, N, padded, with_a):
    g, offsets, counts, rows, sp = case(M, G, padded, 4)
    dy, h = matrix(g, rows, N, N + 8), matrix(g, rows, 2 * I, 2 * I + 8, scale=3.0)
    wd = (torch.randn(G, N, I, generator=g, device="cuda") * 0.1).to(BF16)
    live = poison(dy, sp)
    poison(h, sp)
    out = matrix(g, rows, 2 * I, 2 * I + 8 * (M % 2))
    a = matrix(g, rows, I, I + 8) if with_a else None
    d0, a0 = out.clone(), None if a is None else a.clone()
    dh, aa = fgg.grouped_gated_backward(dy, wd, h, offsets, counts, out=out, a=a)
    assert dh is out and aa is a and torch.equal(dh[~live], d0[~live])
    if with_a:
        assert torch.equal(a[~live], a0[~live])
    for e, (s, t) in enumerate(sp):
        if t == s:
            continue
        hd = h[s:t].double().requires_grad_()
        act = gated(hd)
        da, bound = product(dy[s:t], wd[e], BF16)
        off = bound - HALF[BF16] * da.abs()
        act.backward(da)
        one = torch.autograd.grad(gated(hd), hd, torch.ones_like(da))[0].abs()     # |d a / d h|
        # the derivative's two terms can cancel: their own magnitudes bound its rounding
        gate, up = h[s:t].double().chunk(2, dim=1)
        sg = torch.sigmoid(gate)
        terms = torch.cat([up.abs() * sg * (1 + gate.abs() * (1 - sg)), (gate * sg).abs()], 1)
        two = torch.cat([da, da], 1).abs()
        within(dh[s:t], hd.grad, HALF[BF16] * hd.grad.abs() + one * 1.01 * torch.cat([off, off], 1)
               + ACT * terms * two + 1e-38, f"segment {e}")
        if with_a:
            ref = act.detach()
            within(a[s:t], ref, (HALF[BF16] + ACT) * ref.abs() + 1e-38, f"activation of segment {e}")


def test_large_pre_activations():
    """Gates far out: silu(g) is g above and 0 below, the derivative 1 and 0; no NaN comes of e^-g overflowing."""
    I = 8
    gate = torch.tensor([-3e38, -1e30, -200.0, -89.0, 0.0, 89.0, 1e30, 3e38], device="cuda")
    h = torch.cat([gate, torch.full((I,), 0.5, device="cuda")])[None].to(BF16)
    eye = torch.eye(I, device="cuda").to(BF16)[None]
    dy = torch.ones(1, I, dtype=BF16, device="cuda")
    a = torch.empty(1, I, dtype=BF16, device="cuda")
    dh, _ = fgg.grouped_gated_backward(dy, eye, h, a=a)
    gd = h[0, :I].double()
    step = (gd > 0).double() + 0.5 * (gd == 0)
    assert torch.allclose(a[0].double(), 0.5 * gd * step, rtol=2.0 ** -8, atol=1e-30)
    assert torch.allclose(dh[0, :I].double(), 0.5 * step, rtol=2.0 ** -8, atol=1e-30)
    assert torch.allclose(dh[0, I:].double(), gd * step, rtol=2.0 ** -8, atol=1e-30)
    x = torch.full((1, 8), 1.0, dtype=BF16, device="cuda")
    w = torch.zeros(1, 16, 8, dtype=BF16, device="cuda")
    w[0, :8, 0], w[0, 8:, 0] = h[0, :8], 0.5
    a, _ = fgg.grouped_gated(x, w)
    assert torch.allclose(a[0].double(), 0.5 * gd * step, rtol=2.0 ** -8, atol=1e-30)


def test_nan_stays_in_its_row():
    g = torch.Generator(device="cuda").manual_seed(9)
    x, w = matrix(g, 40, 64, 64), matrix(g, 48, 64, 64)[None].contiguous()
    clean, _ = fgg.grouped_gated(x, w)
    x[7] = float("nan")
    a, _ = fgg.grouped_gated(x, w)
    assert a[7].isnan().all() and torch.equal(a[:7], clean[:7]) and torch.equal(a[8:], clean[8:])
