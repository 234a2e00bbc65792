"""The few-row form of the linear layer and the gated block where segments are uneven: passes of 64 rows of one
segment side by side, and which calls take the form."""

import os
import subprocess
import sys

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, HALF, gated, matrix, poison, product, within

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("sizes,N,K", [
    ((0, 64, 0, 0), 512, 264), ((65, 0, 0, 1, 0), 264, 520), ((0,) * 9 + (256,) + (0,) * 6, 504, 200),
    ((1, 129, 0, 2, 0, 0, 63, 61), 72, 1032), ((0, 0, 200, 17, 0, 33, 6, 0, 0, 0, 0, 0, 0, 0, 0, 0), 136, 72),
    ((16,) * 16, 512, 136), ((32, 31, 1, 64), 1000, 2056),
])
def test_uneven_segments(sizes, N, K, dtype):
    g = torch.Generator(device="cuda").manual_seed(21)
    G, gap = len(sizes), 2
    firsts = [sum(sizes[:e]) + gap * e for e in range(G)]
    M = sum(sizes)                                     # (with rows of no segment: behind the last one's too)
    rows = M + gap * G
    offsets = torch.tensor(firsts + [rows], dtype=torch.int32, device="cuda")
    counts = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    sp = [(s, s + n) for s, n in zip(firsts, sizes)]
    x, w = matrix(g, rows, K, K + 8), (torch.randn(G, N, K, generator=g, device="cuda") * 0.1).to(BF16)
    live = poison(x, sp)
    y = matrix(g, rows, N, N, dtype)
    y0 = y.clone()
    fgg.grouped_linear(x, w, offsets, counts, out=y)
    assert torch.equal(y[~live], y0[~live])
    I = N // 2 // 8 * 8
    w2 = w[:, :2 * I].contiguous()
    a, h = matrix(g, rows, I, I), matrix(g, rows, 2 * I, 2 * I)
    a0 = a.clone()
    fgg.grouped_gated(x, w2, offsets, counts, out=a, h=h)
    assert torch.equal(a[~live], a0[~live])
    for e, (s, t) in enumerate(sp):
        if s == t:
            continue
        within(y[s:t], *product(x[s:t], w[e].t(), dtype), f"segment {e}")
        ref, bound = product(x[s:t], w2[e].t(), BF16)
        within(h[s:t], ref, bound, f"pre-activations of segment {e}")
        # |d silu| <= 1.1: the fp32 sums' error, then the activation's and the result's rounding
        off = bound - HALF[BF16] * ref.abs()
        gate, up = ref.abs().chunk(2, dim=1)
        act = gated(ref)
        moved = 1.2 * (up * off[:, :I] + gate * off[:, I:]) + off[:, :I] * off[:, I:]
        within(a[s:t], act, (HALF[BF16] + 2.0 ** -18) * act.abs() + moved + 1e-30, f"segment {e}")


def test_which_calls_take_the_form():
    """By the launch trace: few rows of few tiles do, however they are spread; 24 rows a segment on 128 tiles, more than
    32 a segment, and more than 256 in all do not."""
    calls = [(1, 1, 4096, True), (1, 32, 4096, True), (1, 33, 4096, False), (1, 16, 8192, True), (1, 17, 8192, False),
             (16, 256, 512, True), (16, 257, 512, False), (16, 512, 512, False), (4, 96, 2048, False),
             (64, 256, 128, True), (64, 512, 128, False)]
    code = f"""
import torch, fp4_grouped_gemm_amd as fgg
for G, M, N, _ in {calls!r}:
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")
    o = torch.tensor([0] * G + [M], dtype=torch.int32, device="cuda")
    fgg.grouped_linear(z(M, 72), z(G, N, 72), o)
    fgg.grouped_gated(z(M, 72), z(G, N, 72), o)
torch.cuda.synchronize()
"""
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, FGG_DEBUG="1"), capture_output=True, text=True,
                       cwd=ROOT, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = [line.split("[fgg] ")[1].split(":")[0] for line in r.stderr.splitlines() if "[fgg] " in line]
    assert [s.startswith("rows_bf16") for s in seen] == [few for *_, few in calls for _ in range(2)], seen
