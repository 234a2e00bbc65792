"""The products at the sizes that take the larger tile shapes (with a last round in quarters), that
cut the weights' gradient's sum, and that go to the few-row kernel; each against float64."""

import os
import subprocess
import sys

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, HALF, gated, matrix, poison, product, segments, spans, within

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# outputs' rows and columns, segments, sum: Large (289 and more tiles of 256 x 256: one round and quarters), Medium
SIZES = [(4200, 4112, 1, 520), (4300, 4112, 3, 584), (2100, 1040, 1, 1096), (2000, 1168, 4, 2056)]


def rows_case(M, G, padded, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    offsets, counts, rows = segments(G, M, seed, padded, empty=False)
    if G == 1:
        offsets, counts, rows = None, None, M
    return g, offsets, counts, rows, [(0, M)] if offsets is None else spans(offsets, counts, rows)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,W,G,S", SIZES)
def test_linear_and_input_gradient(M, W, G, S, dtype):
    g, offsets, counts, rows, sp = rows_case(M, G, True, 1)
    x, w = matrix(g, rows, S, S + 8), (torch.randn(G, W, S, generator=g, device="cuda") * 0.1).to(BF16)
    live = poison(x, sp)
    for weights, call in ((w, fgg.grouped_linear), (w.transpose(1, 2).contiguous(), fgg.grouped_linear_backward_input)):
        out = matrix(g, rows, W, W + 8, dtype)
        before = out.clone()
        call(x, weights, offsets, counts, out=out)
        assert torch.equal(out[~live], before[~live])
        for e, (s, t) in enumerate(sp):
            within(out[s:t], *product(x[s:t], w[e].t(), dtype), f"{call.__name__}, segment {e}")


@pytest.mark.parametrize("M,W,G,S", SIZES)
def test_gated_and_gradient(M, W, G, S):
    g, offsets, counts, rows, sp = rows_case(M, G, True, 2)
    x, w = matrix(g, rows, S, S), (torch.randn(G, W, S, generator=g, device="cuda") * S ** -0.5).to(BF16)
    I = W // 2
    live = poison(x, sp)
    out, h = matrix(g, rows, I, I + 8), matrix(g, rows, W, W)
    a0, h0 = out.clone(), h.clone()
    fgg.grouped_gated(x, w, offsets, counts, out=out, h=h)
    assert torch.equal(out[~live], a0[~live]) and torch.equal(h[~live], h0[~live])
    for e, (s, t) in enumerate(sp):
        ref, bound = product(x[s:t], w[e].t(), BF16)
        within(h[s:t], ref, bound, f"pre-activations, segment {e}")
        # |d silu| <= 1.1: the fp32 sums' error, then the activation's and the result's rounding
        off = bound - HALF[BF16] * ref.abs()
        gate, up = ref.chunk(2, dim=1)
        act = gated(ref)
        within(out[s:t], act, (HALF[BF16] + 2.0 ** -18) * act.abs() + 1.2 * (up.abs() * off[:, :I] + gate.abs() * off[:, I:])
               + off[:, :I] * off[:, I:] + 1e-30, f"segment {e}")
    # back, with W columns of pre-activations' halves each
    wd = (torch.randn(G, S, W, generator=g, device="cuda") * 0.1).to(BF16)
    h2 = matrix(g, rows, 2 * W, 2 * W + 8, scale=2.0)
    dh, a = matrix(g, rows, 2 * W, 2 * W), matrix(g, rows, W, W)
    d0 = dh.clone()
    fgg.grouped_gated_backward(x, wd, h2, offsets, counts, out=dh, a=a)
    assert torch.equal(dh[~live], d0[~live])
    for e, (s, t) in enumerate(sp):
        da, bound = product(x[s:t], wd[e], BF16)
        off = bound - HALF[BF16] * da.abs()
        gate, up = h2[s:t].double().chunk(2, dim=1)
        sg = torch.sigmoid(gate)
        one = torch.cat([up * sg * (1 + gate * (1 - sg)), gate * sg], 1)
        terms = torch.cat([up.abs() * sg * (1 + gate.abs() * (1 - sg)), (gate * sg).abs()], 1)
        two, off = torch.cat([da, da], 1), torch.cat([off, off], 1)
        within(dh[s:t], two * one, HALF[BF16] * (two * one).abs() + 1.01 * one.abs() * off + 2.0 ** -18 * terms * two.abs()
               + 1e-30, f"gradient, segment {e}")
        act = gated(h2[s:t].double())
        within(a[s:t], act, (HALF[BF16] + 2.0 ** -18) * act.abs() + 1e-30, f"activation again, segment {e}")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K,G", [(1100, 4104, 4104, 1), (3000, 2312, 2056, 4), (1400, 1032, 2056, 1),
                                     (20000, 520, 264, 1), (9000, 72, 136, 3), (30000, 1024, 1160, 1), (70000, 8, 16, 1)])
def test_weight_gradient(M, N, K, G, dtype):
    g, offsets, counts, rows, sp = rows_case(M, G, True, 3)
    dy, x = matrix(g, rows, N, N + 8), matrix(g, rows, K, K)
    poison(dy, sp), poison(x, sp)
    got = fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out_dtype=dtype)
    again = got.clone()
    fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out=again, accumulate=True)
    for e, (s, t) in enumerate(sp):
        ref, bound = product(dy[s:t].t(), x[s:t], dtype)
        within(got[e], ref, bound, f"segment {e}")
        within(again[e], 2 * ref, 3 * bound, f"segment {e}, twice")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("M,N,K,G", [(1, 4096, 7168, 1), (7, 1000, 2056, 1), (17, 520, 1992, 1), (32, 264, 72, 1),
                                     (20, 200, 4104, 4), (40, 136, 776, 2), (50, 64, 7000, 40), (1, 8, 8, 1)])
def test_few_rows(M, N, K, G, dtype):
    g, offsets, counts, rows, sp = rows_case(M, G, False, 4)
    x, w = matrix(g, rows, K, K + 8), (torch.randn(G, N, K, generator=g, device="cuda") * 0.1).to(BF16)
    got = fgg.grouped_linear(x, w, offsets, counts, out_dtype=dtype)
    for e, (s, t) in enumerate(sp):
        if t > s:
            within(got[s:t], *product(x[s:t], w[e].t(), dtype), f"segment {e}")
    if N % 16 == 0:
        h = torch.empty(rows, N, dtype=BF16, device="cuda")
        a, _ = fgg.grouped_gated(x, w, offsets, counts, h=h)
        plain, _ = fgg.grouped_gated(x, w, offsets, counts)
        assert torch.equal(a, plain)
        for e, (s, t) in enumerate(sp):
            if t > s:
                within(h[s:t], *product(x[s:t], w[e].t(), BF16), f"pre-activations, segment {e}")


def test_more_rows_in_one_segment_than_in_the_others():
    """Few rows per segment on average, all of them in one: several passes over its weights."""
    g = torch.Generator(device="cuda").manual_seed(8)
    M, N, K, G = 100, 24, 520, 4
    x, w = matrix(g, M, K, K), matrix(g, G * N, K, K).view(G, N, K)
    offsets = torch.tensor([0, 0, 97, 100, 100], dtype=torch.int32, device="cuda")
    got = fgg.grouped_linear(x, w, offsets)
    within(got[:97], *product(x[:97], w[1].t(), BF16), "the long one")
    within(got[97:], *product(x[97:], w[2].t(), BF16), "the short one")


def test_the_sizes_reach_every_kernel():
    """Which kernels the sizes above take, by the library's launch trace."""
    code = """
import torch, fp4_grouped_gemm_amd as fgg
z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
for M, W, S in ((4200, 4112, 520), (2100, 1040, 1096), (300, 528, 1000), (7, 1008, 2056)):
    x, w, wt = z(M, S), z(1, W, S), z(1, S, W)
    fgg.grouped_linear(x, w)
    fgg.grouped_gated(x, w)
    fgg.grouped_linear_backward_input(x, wt)
    fgg.grouped_gated_backward(x, wt, z(M, 2 * W))
for M, N, K in ((1100, 4104, 4104), (1400, 1032, 2056), (300, 520, 520)):
    fgg.grouped_linear_backward_weight(z(M, N), z(M, K), 1)
for acc in (False, True):
    for t in (torch.float32, torch.bfloat16):
        fgg.grouped_linear_backward_weight(z(20000, 520), z(20000, 264), 1, accumulate=acc,
                                           out=torch.zeros(1, 520, 264, dtype=t, device="cuda"))
for T, N, K in ((4, 64, 72), (300, 2048, 16384), (5000, 2048, 1032)):
    for r in (8, 16, 32, 64, 128):
        for t in (torch.float32, torch.bfloat16):
            fgg.lora_add(torch.zeros(T, N, dtype=t, device="cuda"), z(T, K), torch.zeros(T, dtype=torch.int32, device="cuda"),
                         z(2, r, K), z(2, N, r))
torch.cuda.synchronize()
"""
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, FGG_DEBUG="1"), capture_output=True, text=True,
                       cwd=ROOT, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = {line.split("[fgg] ")[1].split(":")[0] for line in r.stderr.splitlines() if "[fgg] " in line}
    new = [k["kernel"] for k in fgg.kernel_table()
           if k["kernel"].startswith(("gemm_bf16", "rows_bf16", "dw_join", "lora_"))]
    assert len(new) == 15 + 2 + 4 + 27
    assert not set(new) - seen, sorted(set(new) - seen)
