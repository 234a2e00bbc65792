"""Empty segments in launches of Large tiles taken one after the other: a tile without a sum between full ones, first,
last, and among the tiles that go in quarters; and NaN beside the adapters' tiles of 16 tokens."""

import os
import subprocess
import sys

import pytest
import torch

import fp4_grouped_gemm_amd as fgg
from _products import BF16, F32, matrix, poison, product, within
from test_gpu_lora import inputs

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

N = K = 4104                  # 17 x 17 tiles of 256 x 256 a segment; 3 and 8 of them leave a last round of 99 and of 8
# rows of each segment (the last round in quarters lies in the last one)
ROWS = [(0, 6100, 0), (0, 2300, 4001), (2500, 0, 3700), (3600, 2700, 0), (0, 0, 5000),
        (0, 2000, 65, 0, 0, 4800, 3001, 0), (3000, 0, 1, 4000, 64, 0, 2900, 2200)]


@pytest.mark.parametrize("gap", [0, 3])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows", ROWS)
def test_weight_gradient(rows, dtype, gap):
    g = torch.Generator(device="cuda").manual_seed(11)
    G = len(rows)
    firsts = [gap + sum(rows[:e]) + gap * e for e in range(G)]
    M = firsts[-1] + rows[-1] + gap
    offsets = torch.tensor(firsts + [M], dtype=torch.int32, device="cuda")
    counts = torch.tensor(rows, dtype=torch.int32, device="cuda")
    sp = [(s, s + n) for s, n in zip(firsts, rows)]
    dy, x = matrix(g, M, N, N + 8), matrix(g, M, K, K)
    poison(dy, sp), poison(x, sp)
    got = torch.full((G, N, K), float("nan"), dtype=dtype, device="cuda")
    fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out=got)
    again = got.clone()
    held = [e for e in range(G) if rows[e] == 0]
    again[held] = 3.0
    fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out=again, accumulate=True)
    for e, (s, t) in enumerate(sp):
        if s == t:
            assert (got[e] == 0).all() and (again[e] == 3).all()
            continue
        ref, bound = product(dy[s:t].t(), x[s:t], dtype)
        within(got[e], ref, bound, f"segment {e}")
        within(again[e], 2 * ref, 3 * bound, f"segment {e}, twice")
    assert torch.equal(got, fgg.grouped_linear_backward_weight(dy, x, G, offsets, counts, out_dtype=dtype))


def test_these_are_large_tiles():
    code = f"""
import torch, fp4_grouped_gemm_amd as fgg
for rows in {ROWS!r}:
    o = torch.tensor((0,) + rows, device="cuda").cumsum(0).int()
    t = torch.zeros(sum(rows), {N}, dtype=torch.bfloat16, device="cuda")
    fgg.grouped_linear_backward_weight(t, t, len(rows), o)
torch.cuda.synchronize()
"""
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, FGG_DEBUG="1"), capture_output=True, text=True,
                       cwd=ROOT, timeout=100)
    assert r.returncode == 0, r.stderr[-2000:]
    seen = [line.split("[fgg] ")[1].split(":")[0] for line in r.stderr.splitlines() if "[fgg] " in line]
    assert seen == ["gemm_bf16_kernel<dw,Large>"] * len(ROWS), seen


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,r,N,K", [(300, 16, 2056, 16392), (300, 32, 2048, 8200), (130, 64, 4104, 4104),
                                     (300, 128, 2048, 4104)])
def test_nan_beside_tiles_of_16_tokens(T, r, N, K, dtype):
    """NaN in an adapter, a token and a column of B stay there (two launches, fewer than 512 tokens)."""
    base, x, ids, a, b, scales = inputs(T, 4, r, N, K, dtype, "any", 12)
    assert fgg.lora_workspace_bytes(T, 4, r, N, K) > 0
    ids[:8] = torch.tensor([0, 1, 2, 3, 0, 1, 2, 3])
    clean = fgg.lora_add(base, x, ids, a, b, scales)
    a[1], b[2, 5], x[4], base[7, 3] = float("nan"), float("nan"), float("nan"), float("nan")
    got = fgg.lora_add(base, x, ids, a, b, scales)
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[ids == 1] = hit[4] = True
    hit[ids == 2, 5] = hit[7, 3] = True
    assert got[hit].isnan().all() and torch.equal(got[~hit], clean[~hit])
