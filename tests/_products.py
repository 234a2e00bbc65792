"""Segments, inputs and 64-bit references for the tests of the bf16 products (plain torch in
float64, on whatever device the inputs are)."""

import torch

BF16, F32 = torch.bfloat16, torch.float32
HALF = {BF16: 2.0 ** -8, F32: 2.0 ** -24}        # half a step, relative


def segments(G, M, seed, padded, empty=True):
    """(offsets, counts or None, total rows): G segments of M rows in all, some of them empty; padded: each
    begins at a multiple of 8 rows past a gap, and counts says how many rows are real."""
    g = torch.Generator().manual_seed(seed)
    p = torch.rand(G, generator=g) + 0.05
    if empty and G > 2:
        p[torch.randperm(G, generator=g)[:max(1, G // 4)]] = 0
    sizes = torch.bincount(torch.multinomial(p, M, True, generator=g), minlength=G) if M else torch.zeros(G).long()
    taken = (sizes + 15) // 8 * 8 if padded else sizes
    offsets = torch.zeros(G + 1, dtype=torch.long)
    offsets[1:] = torch.cumsum(taken, 0)
    return offsets.int().cuda(), sizes.int().cuda() if padded else None, int(offsets[-1])


def spans(offsets, counts, M):
    """[(first, end)] of every segment as host numbers, inside [0, M)."""
    off = offsets.tolist()
    out = []
    for g in range(len(off) - 1):
        s, e = min(max(off[g], 0), M), min(off[g + 1], M)
        if counts is not None:
            e = min(e, off[g] + int(counts[g]))
        out.append((s, max(s, e)))
    return out


def matrix(g, rows, cols, ld, dtype=BF16, scale=1.0, junk=None):
    """A [rows, cols] view of row stride ld; what lies between rows is junk (NaN where given)."""
    whole = torch.full((max(rows, 1), ld), float("nan") if junk is None else junk, dtype=dtype, device="cuda")
    view = whole[:rows, :cols]
    view.copy_(torch.randn(rows, cols, generator=g, device="cuda") * scale)
    return view


def poison(t, spans):
    """NaN in every row of no segment."""
    live = torch.zeros(t.shape[0], dtype=torch.bool, device=t.device)
    for s, e in spans:
        live[s:e] = True
    t[~live] = float("nan")
    return live


def within(got, ref, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    err = (got - ref).abs()
    bad = err > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst "
                           f"{float((err / bound.clamp_min(1e-300)).max()):.3g} times the bound")


def product(a, b, dtype):
    """a @ b in float64 and how far a kernel may be from it: products of bf16 numbers are exact in fp32, a sum of
    n of them in any order is within n 2^-24 of the sum of their magnitudes, and is rounded once."""
    a, b = a.double(), b.double()
    ref, mag = a @ b, a.abs() @ b.abs()
    return ref, HALF[dtype] * ref.abs() + a.shape[1] * 2.0 ** -24 * mag + 1e-38


def gated(h):
    """silu(gate) up of float64 pre-activations."""
    gate, up = h.chunk(2, dim=1)
    return gate * torch.sigmoid(gate) * up
