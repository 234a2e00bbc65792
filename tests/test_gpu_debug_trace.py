"""FGG_DEBUG: every launch prints one line naming its kernel, problem, grid and
LDS budget (run in a child process, since the flag is read once per process)."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = r"""
import sys, torch
sys.path.insert(0, %r)
import fp4_grouped_gemm_amd as fgg
dev = "cuda"
x = torch.randn(256, 512, device=dev)
xq, xs = fgg.quantize_blockwise(x, fgg.Q_E4M3_1x128)
w = torch.randn(2, 256, 512, device=dev) * 0.02
bq = torch.stack([fgg.quantize_blockwise(w[e], fgg.Q_E4M3_128x128)[0] for e in range(2)])
sb = torch.stack([fgg.quantize_blockwise(w[e], fgg.Q_E4M3_128x128)[1] for e in range(2)])
ids = torch.randint(0, 2, (256, 1), dtype=torch.int32, device=dev)
p = fgg.moe_permute(ids, 2, 128, x=x)
q, s = fgg.grouped_gemm_silu_quantize(p["a"], p["sa"], bq, sb, p["offsets"])
h = fgg.grouped_gemm_scaled(p["a"], p["sa"], bq, sb, offsets=p["offsets"], masked_m=p["counts"])
out = fgg.moe_combine(h, p["src_to_row"], torch.ones(256, 1, device=dev))
y = fgg.scaled_gemm(xq, xs, bq[0], sb[0])
xq4, xs4 = fgg.quantize_blockwise(x, fgg.Q_E2M1_1x16)
y4 = fgg.scaled_gemm(xq4, xs4, xq4[:128], xs4[:128], qdesc="w4a4")
xq5, xe5 = fgg.quantize_blockwise(x, fgg.Q_E2M1_E8M0_1x32)
ld = (torch.randn(512, 32, device=dev) * 0.01).to(torch.bfloat16)
lu = (torch.randn(32, 128, device=dev) * 0.01).to(torch.bfloat16)
y5 = fgg.scaled_gemm(xq5, xe5, xq5[:128], xe5[:128], qdesc="mxfp4", x_bf16=x.to(torch.bfloat16), l_down=ld, l_up=lu)
torch.cuda.synchronize()
print("script done")
""" % ROOT


def test_debug_trace_names_every_launch():
    env = dict(os.environ, FGG_DEBUG="1")
    r = subprocess.run([sys.executable, "-c", SCRIPT], env=env, capture_output=True, text=True, timeout=180)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = [l for l in r.stderr.splitlines() if l.startswith("[fgg] ")]
    for kernel in ("quant_e4m3_1x128_kernel", "quant_e4m3_128x128_kernel", "permute_hist_kernel",
                   "permute_scatter_kernel", "permute_quantize_kernel", "gemm_fp8_contig_kernel<silu>",
                   "gemm_fp8_contig_kernel<plain>", "combine_kernel", "gemm_fp8_dense_kernel",
                   "quant_e2m1_1x16_kernel", "w4a4_prep_kernel", "w4a4_gemm_kernel",
                   "quant_e2m1_e8m0_1x32_kernel", "w4a4_lowrank_kernel", "gemm_mxfp4_kernel"):
        hits = [l for l in lines if l.startswith(f"[fgg] {kernel}:")]
        assert hits, f"no trace line for {kernel}"
        assert "grid=" in hits[0] and "lds=" in hits[0]
    assert any("counts" in l for l in lines if "contig_kernel<plain>" in l)


ROUTING_SCRIPT = r"""
import sys, torch
sys.path.insert(0, %r)
import fp4_grouped_gemm_amd as fgg
dev = "cuda"
fgg.set_num_cus(256)

def gemv(T, G, k, N, K, form, tiled, dtype=torch.bfloat16):
    rows = 2 * N if form == "silu" else N
    b = torch.zeros(G, rows, K // 2, dtype=torch.uint8, device=dev)
    s = torch.full((G, rows, K // 32), 127, dtype=torch.uint8, device=dev)
    q = fgg.Q_E2M1_E8M0_1x32
    if tiled:
        (b, s), q = fgg.pack_fp4_weights(b, s), fgg.Q_E2M1_E8M0_1x32_TILED
    ids = None if G == 1 else torch.arange(T * k, device=dev, dtype=torch.int32).view(T, k) %% G
    w = torch.ones(T, k, device=dev) if form == "sum" else None
    x = torch.ones(T, K, device=dev, dtype=dtype)
    torch.cuda.synchronize()
    fgg.moe_gemv_fp4(x, b, s, ids, w, b_qdesc=q, n=N, silu_mul=form == "silu")

def back(E):
    x = torch.zeros(5, E, device=dev)
    fgg.moe_route_backward(x, torch.zeros(5, 2, dtype=torch.int32, device=dev), torch.ones(5, 2, device=dev))

for call in sys.argv[1:]:
    print("[call]", call, file=sys.stderr, flush=True)
    eval(call)
    torch.cuda.synchronize()
for i, k in enumerate(fgg.kernel_table()):
    print("[table]", k["kernel"], k["threads"], k["lds_bytes"], fgg.kernel_compiled_lds(i), sep="|", file=sys.stderr)
""" % ROOT

LISTS = 4096 + 4096 + 2048 + 1024 + 64 + 512 + 4096      # pairs, experts, visits, columns, gate weights


def _gemv_lds(waves, tiles, scratch):
    """The lists, a 1 KB tile of partial sums per wave and row tile, 4 KB a wave to turn activations."""
    return LISTS + waves * tiles * 1024 + (waves * 4096 if scratch else 0)


ROUTING_CALLS = {   # call: threads, LDS bytes, rows of weights (or pairs of rows) a workgroup takes
    "gemv(1, 1, 1, 64, 2048, 'plain', True)": (256, _gemv_lds(4, 1, False), 16),
    "gemv(9, 1, 1, 64, 2048, 'plain', False)": (256, _gemv_lds(4, 1, True), 16),
    "gemv(3, 1, 1, 32, 8192, 'plain', True)": (512, _gemv_lds(8, 1, False), 16),
    "gemv(5, 1, 1, 32, 8192, 'plain', True)": (512, _gemv_lds(8, 1, True), 16),
    "gemv(2, 2, 1, 9600, 256, 'plain', False)": (256, _gemv_lds(4, 1, False), 64),
    "gemv(8, 2, 1, 9600, 256, 'silu', True)": (256, _gemv_lds(4, 2, True), 64),
    "gemv(2, 2, 1, 9600, 1024, 'silu', True)": (256, _gemv_lds(4, 2, False), 32),
    "gemv(7, 1, 1, 48, 4096, 'silu', True)": (512, _gemv_lds(8, 2, True), 16),
    "gemv(7, 1, 1, 48, 4096, 'silu', True, torch.float32)": (512, _gemv_lds(8, 2, False), 16),
    "gemv(16, 32, 8, 512, 256, 'sum', True)": (1024, _gemv_lds(16, 1, False), 16),
    "gemv(16, 8, 8, 512, 256, 'sum', False)": (1024, _gemv_lds(16, 1, False), 16),
    "gemv(16, 8, 2, 4096, 256, 'sum', False)": (1024, _gemv_lds(16, 1, True), 16),
    "gemv(16, 8, 2, 4096, 256, 'sum', False, torch.float32)": (1024, _gemv_lds(16, 1, False), 16),
    "gemv(16, 2, 1, 8192, 128, 'sum', False)": (512, _gemv_lds(8, 1, True), 16),
    "gemv(3, 2, 1, 8192, 128, 'sum', True)": (512, _gemv_lds(8, 1, False), 16),
    "gemv(16, 2, 1, 8192, 128, 'sum', True)": (1024, _gemv_lds(16, 2, True), 32),
    "back(8)": (256, 0, 0), "back(30)": (256, 0, 0), "back(64)": (256, 1024, 0), "back(100)": (256, 2048, 0),
    "back(200)": (256, 4096, 0), "back(500)": (256, 8192, 0), "back(1000)": (256, 16384, 0),
}


def test_routing_launches_state_their_workgroup():
    """The few-token products and the router's gradient have several forms: the line of a launch, the table's
    entry of that name and the compiled kernel agree, and with the form that the sizes call for."""
    env = dict(os.environ, FGG_DEBUG="1")
    r = subprocess.run([sys.executable, "-c", ROUTING_SCRIPT, *ROUTING_CALLS], env=env, capture_output=True, text=True,
                       timeout=180)
    assert r.returncode == 0, r.stderr[-2000:]
    table, lines, call = {}, {}, None
    for l in r.stderr.splitlines():
        if l.startswith("[call] "):
            call = l[7:]
        elif l.startswith(("[fgg] gemv_fp4_kernel", "[fgg] route_backward_kernel")):
            assert call not in lines, l
            lines[call] = l
        elif l.startswith("[table]|"):
            name, threads, lds, compiled = l.split("|")[1:]
            table[name] = (int(threads), int(lds), int(compiled))
    for call, (threads, lds, rows) in ROUTING_CALLS.items():
        l = lines[call]
        assert f" threads={threads} " in l and f" tile={rows}x" in l and f" lds={lds} B " in l, (call, l)
        name = l[len("[fgg] "):l.index(": ")]
        assert table[name] == (threads, lds, lds), (call, l, table[name])
