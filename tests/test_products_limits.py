"""Sizes past what the bf16 products take are refused on the host; those at the limits run in
test_gpu_products_longest.py."""

import ctypes
import os

import pytest

import fp4_grouped_gemm_amd as fgg
from test_products_refusals import UNSUPPORTED, WIDE, dw, dx, gated, gated_bwd, linear

pytestmark = pytest.mark.skipif(not os.path.exists(fgg.library_path()),
                                reason="libfgg.so not built (run __graft_entry__.build())")

MOST = WIDE - 8


def up(a, b):
    return -(-a // b)


HALF_WIDE = MOST // 2 // 8 * 8


@pytest.mark.parametrize("call,tiles,sizes", [
    (linear, up(1 << 19, 256) * up(MOST, 256), dict(G=1, off=None, M=1 << 19, N=MOST, ldy=MOST)),
    (linear, (up((1 << 19) - 512, 256) + 2) * up(MOST, 256), dict(G=2, M=(1 << 19) - 512, N=MOST, ldy=MOST)),
    (dx, up(1 << 19, 256) * up(MOST, 256), dict(G=1, off=None, M=1 << 19, K=MOST, ldd=MOST)),
    (gated, up(1 << 18, 256) * up(MOST, 128), dict(G=1, off=None, M=1 << 18, N=MOST, lda=MOST)),
    (gated_bwd, up(1 << 20, 256) * up(HALF_WIDE, 256),
     dict(G=1, off=None, M=1 << 20, N=HALF_WIDE, ldh=MOST, lddh=MOST)),
    (dw, 1024 * up(MOST, 256) * up(520, 256), dict(G=1024, N=MOST, K=520, lddy=MOST, ldx=520)),
])
def test_more_tiles_than_a_call_has(call, tiles, sizes):
    """2^25 tiles of 256 x 256 (gated: 256 x 128), a segment's partial one counted."""
    assert tiles >= 1 << 25                     # (these pointers must reach no device)
    assert call(**sizes) == UNSUPPORTED


def test_workspace_of_sizes_past_the_limits():
    n = ctypes.c_size_t(0)
    ws = fgg.load_library().fgg_grouped_linear_backward_weight_workspace
    for sizes in ((1, 64, WIDE, 16), (1, 64, 16, WIDE), (1, 1 << 31, 16, 16), (1, 64, 1 << 60, 1 << 60)):
        assert ws(*sizes, ctypes.byref(n)) == UNSUPPORTED
    assert ws(1, (1 << 31) - 1, 8, 8, ctypes.byref(n)) == 0 and n.value % (8 * 8 * 4) == 0
