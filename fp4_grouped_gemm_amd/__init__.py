"""Python binding of libfgg.so (block-scaled FP8/FP4 MoE grouped GEMM for MI355X).

Argument marshalling only: torch supplies device memory and the current HIP
stream; every step of the computation runs in the library's HIP kernels.  The
names follow the C ABI in ``include/fgg.h``, which documents layouts, formats
and error behaviour.  There is no fallback path: if the library is missing or
the device is not gfx950, calls raise.  No call records an autograd node: results are
detached whatever their inputs require, and the gradients are the ``_backward`` calls.
"""

import ctypes
import os

import torch

__all__ = [
    "FggError", "load_library", "library_path",
    "Q_E4M3_1x128", "Q_E4M3_128x128", "Q_E2M1_1x16", "Q_E2M1_E8M0_1x32", "Q_E2M1_E8M0_1x32_TILED",
    "quantize_blockwise", "moe_permute", "moe_permute_outputs", "moe_permute_workspace_bytes",
    "moe_permute_quantize_noalloc", "grouped_gemm_scaled", "grouped_gemm_silu_quantize", "pack_fp4_weights",
    "scaled_gemm", "moe_combine", "set_num_cus", "kernel_table", "kernel_compiled_lds",
    "moe_route", "moe_route_backward", "moe_permute_rows", "moe_permute_rows_backward", "moe_unpermute_rows",
    "moe_unpermute_rows_backward", "moe_gemv_fp4", "grouped_linear", "grouped_linear_backward_input",
    "grouped_linear_backward_weight", "grouped_linear_backward_weight_workspace_bytes", "grouped_gated",
    "grouped_gated_backward", "lora_add", "lora_workspace_bytes",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libfgg.so")

FGG_F32, FGG_BF16, FGG_E4M3, FGG_E2M1X2, FGG_E8M0, FGG_E2M1X2_TILED = 0, 1, 2, 3, 4, 5
FGG_ACT_NONE, FGG_ACT_SILU_MUL = 0, 1
FGG_LAYOUT_CONTIGUOUS, FGG_LAYOUT_MASKED = 0, 1
FGG_GATE_SOFTMAX, FGG_GATE_SIGMOID = 0, 1
_STATUS = {0: "FGG_OK", 1: "FGG_ERR_INVALID_VALUE", 2: "FGG_ERR_UNSUPPORTED", 3: "FGG_ERR_HIP"}


class FggError(RuntimeError):
    def __init__(self, fn, status, hip_error=0):
        self.status = status
        self.hip_error = hip_error
        extra = f" (hipError {hip_error})" if status == 3 else ""
        super().__init__(f"{fn}: {_STATUS.get(status, status)}{extra}")


class QDesc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_int32), ("scale", ctypes.c_int32),
                ("block_rows", ctypes.c_int32), ("block_k", ctypes.c_int32)]


class KernelInfo(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_char_p), ("entry", ctypes.c_char_p), ("tile_m", ctypes.c_int32),
                ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32), ("threads", ctypes.c_int32),
                ("stages", ctypes.c_int32), ("stage_bytes", ctypes.c_int32), ("other_bytes", ctypes.c_int32),
                ("lds_bytes", ctypes.c_int32)]


class Epilogue(ctypes.Structure):
    _fields_ = [("x_bf16", ctypes.c_void_p), ("l_down", ctypes.c_void_p), ("l_up", ctypes.c_void_p),
                ("rank", ctypes.c_int32), ("bias", ctypes.c_void_p)]


Q_E4M3_1x128 = (FGG_E4M3, FGG_F32, 1, 128)
Q_E4M3_128x128 = (FGG_E4M3, FGG_F32, 128, 128)
Q_E2M1_1x16 = (FGG_E2M1X2, FGG_F32, 1, 16)
Q_E2M1_E8M0_1x32 = (FGG_E2M1X2, FGG_E8M0, 1, 32)
Q_E2M1_E8M0_1x32_TILED = (FGG_E2M1X2_TILED, FGG_E8M0, 1, 32)   # masked-GEMM weights from pack_fp4_weights

_lib = None


def library_path() -> str:
    return _LIB_PATH


def load_library():
    """Load libfgg.so once and declare its signatures.  Raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"{_LIB_PATH} is missing: build it with `python -m fp4_grouped_gemm_amd.build`")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I32, I64, SZ, F32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "fgg_status_string": ([I32], ctypes.c_char_p),
        "fgg_last_hip_error": ([], I32),
        "fgg_set_num_cus": ([ctypes.c_int], I32),
        "fgg_kernel_count": ([], I32),
        "fgg_kernel_info_get": ([I32, ctypes.POINTER(KernelInfo)], I32),
        "fgg_kernel_compiled_lds": ([I32, ctypes.POINTER(I64)], I32),
        "fgg_quantize_blockwise": ([P, I32, I64, I64, I64, I32, QDesc, P, P, P, P], I32),
        "fgg_moe_permute_workspace": ([I64, I32, I32, ctypes.POINTER(SZ)], I32),
        "fgg_moe_permute": ([P, I64, I32, I32, I32, P, P, I64, P, P, P, P, P, P, I64, P, SZ, P], I32),
        "fgg_moe_permute_quantize": ([P, I64, I32, I32, I32, P, I32, I64, I64, P, P, P, P, P, P, I64, P, SZ, P], I32),
        "fgg_moe_permute_quantize_noalloc": ([P, I64, I32, I32, I32, P, I32, I64, I64, P, P, P, P, P, P, I64, P], I32),
        "fgg_grouped_gemm_scaled": ([I32, I32, I64, I64, I64, P, P, QDesc, P, P, QDesc, P, P, P, I64, P], I32),
        "fgg_grouped_gemm_silu_quantize": ([I32, I64, I64, I64, P, P, QDesc, P, P, QDesc, P, P, P, P, P], I32),
        "fgg_scaled_gemm_workspace": ([I64, I64, I64, QDesc, QDesc, ctypes.POINTER(Epilogue), ctypes.POINTER(SZ)], I32),
        "fgg_scaled_gemm": ([I64, I64, I64, P, P, QDesc, P, P, QDesc, ctypes.POINTER(Epilogue), P, I64, P, SZ, P], I32),
        "fgg_moe_combine": ([P, I64, P, P, I64, I32, I64, P, I64, P], I32),
        "fgg_moe_down_combine_workspace": ([I64, ctypes.POINTER(SZ)], I32),
        "fgg_moe_down_combine": ([I32, I64, I64, I64, P, P, QDesc, P, P, QDesc, P, P, P, P, P, I64, I32, P, I64, P, SZ,
                                  P, I64, P], I32),
        "fgg_pack_fp4_weights_bytes": ([I32, I64, I64, ctypes.POINTER(SZ), ctypes.POINTER(SZ)], I32),
        "fgg_pack_fp4_weights": ([P, P, I32, I64, I64, P, P, P], I32),
        "fgg_moe_route": ([P, I32, I64, I32, I64, I32, I32, P, I32, F32, P, P, P], I32),
        "fgg_moe_route_backward": ([P, I32, I64, I32, I64, I32, I32, I32, F32, P, P, P, I64, P], I32),
        "fgg_moe_permute_rows": ([P, I32, I64, I32, I64, I64, P, P, P, P, I32, I64, P, I64, P], I32),
        "fgg_moe_permute_rows_backward": ([P, I32, I64, I64, P, I64, P, P, I64, I32, I64, P, I64, P, P], I32),
        "fgg_moe_unpermute_rows": ([P, I32, I64, I64, P, P, I64, I32, I64, P, I64, P], I32),
        "fgg_moe_unpermute_rows_backward": ([P, I32, I64, I32, I64, I64, P, I64, P, P, P, P, I32, I64, P, I64, P, P],
                                            I32),
        "fgg_moe_gemv_fp4": ([I32, I64, I32, I64, I64, P, I32, I64, I32, P, P, QDesc, P, P, I32, P, I32, I64, P], I32),
        "fgg_grouped_linear": ([I32, I64, I64, I64, P, I64, P, P, P, P, I32, I64, P], I32),
        "fgg_grouped_linear_backward_input": ([I32, I64, I64, I64, P, I64, P, P, P, P, I32, I64, P], I32),
        "fgg_grouped_linear_backward_weight_workspace": ([I32, I64, I64, I64, ctypes.POINTER(SZ)], I32),
        "fgg_grouped_linear_backward_weight": ([I32, I64, I64, I64, P, I64, P, I64, P, P, P, I32, I32, P, SZ, P], I32),
        "fgg_grouped_gated": ([I32, I64, I64, I64, P, I64, P, P, P, P, I64, P, I64, P], I32),
        "fgg_grouped_gated_backward": ([I32, I64, I64, I64, P, I64, P, P, I64, P, P, P, I64, P, I64, P], I32),
        "fgg_lora_workspace": ([I64, I32, I32, I64, I64, ctypes.POINTER(SZ)], I32),
        "fgg_lora_add": ([I64, I32, I32, I64, I64, P, I64, P, P, P, P, P, I64, P, I32, I64, P, SZ, P], I32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(fn_name, status):
    if status != 0:
        lib = load_library()
        raise FggError(fn_name, status, lib.fgg_last_hip_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _q(desc):
    return QDesc(*desc)


def set_num_cus(n: int) -> None:
    _check("fgg_set_num_cus", load_library().fgg_set_num_cus(int(n)))


def kernel_table():
    """Every kernel of the library with its tile and LDS budget (fgg_kernel_info_get)."""
    lib = load_library()
    out = []
    for i in range(lib.fgg_kernel_count()):
        ki = KernelInfo()
        _check("fgg_kernel_info_get", lib.fgg_kernel_info_get(i, ctypes.byref(ki)))
        d = {f: getattr(ki, f) for f, _ in KernelInfo._fields_}
        d["kernel"] = d["kernel"].decode()
        d["entry"] = d["entry"].decode()
        out.append(d)
    return out


def kernel_compiled_lds(i: int) -> int:
    """Static LDS bytes of kernel i as compiled (asks the HIP runtime; needs the GPU)."""
    n = ctypes.c_int64(0)
    _check("fgg_kernel_compiled_lds", load_library().fgg_kernel_compiled_lds(int(i), ctypes.byref(n)))
    return n.value


# ------------------------------------------------------------------ quantize

def quantize_blockwise(x: torch.Tensor, qdesc=Q_E4M3_1x128, silu_mul: bool = False, out=None, scales=None,
                       rows_dev=None):
    """Quantize a [rows, cols] fp32/bf16 tensor (rows may have a larger stride).

    With silu_mul=True the input has 2·cols columns laid out [gate | up].
    rows_dev (int32 device tensor, one element) limits the rows processed to
    min(rows, rows_dev[0]) without a host synchronization.
    Returns (codes, scales) in the layouts of include/fgg.h:
      Q_E4M3_1x128:     codes uint8 [rows, cols],   scales f32 [cols/128, rows]
      Q_E4M3_128x128:   codes uint8 [rows, cols],   scales f32 [rows/128, cols/128]
      Q_E2M1_1x16:      codes uint8 [rows, cols/2], scales f32 [rows, cols/16]
      Q_E2M1_E8M0_1x32: codes uint8 [rows, cols/2], scales u8  [rows, cols/32]
    """
    assert x.dim() == 2 and x.dtype in (torch.float32, torch.bfloat16) and x.stride(1) == 1
    rows, width = x.shape
    cols = width // 2 if silu_mul else width
    data, sdt, br, bk = qdesc
    dev = x.device
    if out is None:
        out = torch.empty((rows, cols if data == FGG_E4M3 else cols // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        if qdesc == Q_E4M3_1x128:
            shape = (cols // 128, rows)
        elif qdesc == Q_E4M3_128x128:
            shape = (rows // 128, cols // 128)
        else:
            shape = (rows, cols // bk)
        scales = torch.empty(shape, dtype=torch.uint8 if sdt == FGG_E8M0 else torch.float32, device=dev)
    xdt = FGG_F32 if x.dtype == torch.float32 else FGG_BF16
    st = load_library().fgg_quantize_blockwise(
        _ptr(x), xdt, rows, cols, x.stride(0), FGG_ACT_SILU_MUL if silu_mul else FGG_ACT_NONE,
        _q(qdesc), _ptr(rows_dev), _ptr(out), _ptr(scales), _stream(dev))
    _check("fgg_quantize_blockwise", st)
    return out, scales


# ------------------------------------------------------------------- permute

def moe_permute_workspace_bytes(T: int, k: int, E: int) -> int:
    n = ctypes.c_size_t(0)
    _check("fgg_moe_permute_workspace", load_library().fgg_moe_permute_workspace(T, k, E, ctypes.byref(n)))
    return n.value


def moe_permute_outputs(T: int, k: int, E: int, align: int = 128, K: int = 0, m_cap=None, device="cuda"):
    """Allocate the output buffers of moe_permute (for reuse across calls)."""
    if m_cap is None:
        m_cap = T * k + E * (align - 1)
    out = dict(
        offsets=torch.empty(E + 1, dtype=torch.int32, device=device),
        counts=torch.empty(E, dtype=torch.int32, device=device),
        src_to_row=torch.empty(max(T * k, 1), dtype=torch.int32, device=device),
        row_to_src=torch.empty(max(m_cap, 1), dtype=torch.int32, device=device),
        a=None, sa=None, m_cap=m_cap,
        workspace=torch.empty(max(moe_permute_workspace_bytes(T, k, E), 1), dtype=torch.uint8, device=device))
    if K:
        out["a"] = torch.empty((max(m_cap, 1), K), dtype=torch.uint8, device=device)
        out["sa"] = torch.empty((K // 128, max(m_cap, 1)), dtype=torch.float32, device=device)
    return out


def moe_permute(topk_ids: torch.Tensor, num_experts: int, align: int = 128, xq=None, xs=None,
                m_cap=None, workspace=None, out=None, x=None):
    """Stable padded permute.  topk_ids int32 [T, k] on the device.  With xq
    (uint8 [T, K]) and xs (f32 [K/128, T]) the permuted codes/scales are
    gathered too.  With x (bf16 or f32 [T, K], unit column stride) instead,
    the 1x128 e4m3 quantization is fused into the gather
    (fgg_moe_permute_quantize; same outputs as quantizing first).  Returns a
    dict of device tensors (see include/fgg.h); ``out`` (from
    moe_permute_outputs) is filled instead of allocating."""
    assert topk_ids.dtype == torch.int32 and topk_ids.dim() == 2 and topk_ids.is_contiguous()
    T, k = topk_ids.shape
    E = int(num_experts)
    dev = topk_ids.device
    if x is not None:
        assert xq is None and x.dim() == 2 and x.shape[0] == T and x.stride(1) == 1
        assert x.dtype in (torch.bfloat16, torch.float32)
        K = x.shape[1]
        if out is None:
            out = moe_permute_outputs(T, k, E, align, K, m_cap, dev)
        assert out["a"] is not None and out["a"].shape[1] == K
        if workspace is None:
            workspace = out["workspace"]
        st = load_library().fgg_moe_permute_quantize(
            _ptr(topk_ids), T, k, E, align, _ptr(x), FGG_BF16 if x.dtype == torch.bfloat16 else FGG_F32, K,
            x.stride(0), _ptr(out["offsets"]), _ptr(out["counts"]), _ptr(out["src_to_row"]),
            _ptr(out["row_to_src"]), _ptr(out["a"]), _ptr(out["sa"]), out["m_cap"], _ptr(workspace),
            workspace.numel(), _stream(dev))
        _check("fgg_moe_permute_quantize", st)
        m = out["m_cap"]
        return dict(offsets=out["offsets"], counts=out["counts"], src_to_row=out["src_to_row"][:T * k],
                    row_to_src=out["row_to_src"][:m], a=out["a"], sa=out["sa"], m_cap=m)
    K = 0 if xq is None else xq.shape[1]
    if out is None:
        out = moe_permute_outputs(T, k, E, align, K, m_cap, dev)
    m_cap = out["m_cap"]
    offsets, counts, s2r, r2s = out["offsets"], out["counts"], out["src_to_row"], out["row_to_src"]
    a_out, sa_out = out["a"], out["sa"]
    if xq is not None:
        assert xq.dtype == torch.uint8 and xq.is_contiguous() and xs.is_contiguous()
        assert a_out is not None and a_out.shape[1] == K
    if workspace is None:
        workspace = out["workspace"]
    st = load_library().fgg_moe_permute(
        _ptr(topk_ids), T, k, E, align, _ptr(xq), _ptr(xs), K, _ptr(offsets), _ptr(counts), _ptr(s2r),
        _ptr(r2s), _ptr(a_out), _ptr(sa_out), m_cap, _ptr(workspace), workspace.numel(), _stream(dev))
    _check("fgg_moe_permute", st)
    return dict(offsets=offsets, counts=counts, src_to_row=s2r[:T * k], row_to_src=r2s[:m_cap], a=a_out,
                sa=sa_out, m_cap=m_cap)


def moe_permute_quantize_noalloc(topk_ids: torch.Tensor, num_experts: int, x: torch.Tensor, out, align: int = 128):
    """fgg_moe_permute_quantize_noalloc: the fused permute-quantize with the library's
    static device scratch instead of a workspace (for callers that cannot allocate).
    ``out`` (from moe_permute_outputs) receives every output; its workspace is unused."""
    assert topk_ids.dtype == torch.int32 and topk_ids.dim() == 2 and topk_ids.is_contiguous()
    assert x.dim() == 2 and x.stride(1) == 1 and x.dtype in (torch.bfloat16, torch.float32)
    T, k = topk_ids.shape
    K = x.shape[1]
    assert out["a"] is not None and out["a"].shape[1] == K
    st = load_library().fgg_moe_permute_quantize_noalloc(
        _ptr(topk_ids), T, k, int(num_experts), align, _ptr(x), FGG_BF16 if x.dtype == torch.bfloat16 else FGG_F32,
        K, x.stride(0), _ptr(out["offsets"]), _ptr(out["counts"]), _ptr(out["src_to_row"]), _ptr(out["row_to_src"]),
        _ptr(out["a"]), _ptr(out["sa"]), out["m_cap"], _stream(topk_ids.device))
    _check("fgg_moe_permute_quantize_noalloc", st)
    m = out["m_cap"]
    return dict(offsets=out["offsets"], counts=out["counts"], src_to_row=out["src_to_row"][:T * k],
                row_to_src=out["row_to_src"][:m], a=out["a"], sa=out["sa"], m_cap=m)


# --------------------------------------------------------------------- GEMMs

def grouped_gemm_scaled(a, a_scales, b, b_scales, offsets=None, masked_m=None,
                        b_qdesc=Q_E4M3_128x128, out=None, n=None):
    """Contiguous layout when ``offsets`` is given (a [M, K], a_scales [K/128, M],
    b [G, N, K], b_scales [G, N/128, K/128]); masked layout when ``masked_m``
    is given (a [G, M, K], a_scales [G, K/128, M], b [G, N, K/2] with E8M0
    scales [G, N, K/32] for Q_E2M1_E8M0_1x32, or e4m3 as above).  With
    ``offsets``, an optional ``masked_m`` gives each group's real row count
    (the permute's counts): the padding rows past it are not written.
    With Q_E2M1_E8M0_1x32_TILED (weights from pack_fp4_weights) ``n`` gives N.
    Returns bf16 [M, N] or [G, M, N]."""
    G = b.shape[0]
    N = int(n) if n is not None else b.shape[1]
    dev = a.device
    if offsets is not None:
        M, K = a.shape
        layout = FGG_LAYOUT_CONTIGUOUS
        if out is None:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    else:
        _, M, K = a.shape
        layout = FGG_LAYOUT_MASKED
        if out is None:
            out = torch.empty((G, M, N), dtype=torch.bfloat16, device=dev)
    for t in (a, a_scales, b, b_scales):
        assert t.is_contiguous()
    st = load_library().fgg_grouped_gemm_scaled(
        layout, G, M, N, K, _ptr(a), _ptr(a_scales), _q(Q_E4M3_1x128), _ptr(b), _ptr(b_scales), _q(b_qdesc),
        _ptr(offsets), _ptr(masked_m), _ptr(out), out.stride(-2), _stream(dev))
    _check("fgg_grouped_gemm_scaled", st)
    return out


def grouped_gemm_silu_quantize(a, a_scales, b, b_scales, offsets, counts=None, out=None, scales=None):
    """Gate-up grouped GEMM with SiLU(gate)*up and the 1x128 e4m3 requantization
    fused (fgg_grouped_gemm_silu_quantize): a [M, K] e4m3 with [K/128, M]
    scales, b [G, 2I, K] ([gate | up] rows) with [G, 2I/128, K/128] scales.
    ``counts`` (optional, [G] int32): real rows per group; padding rows past
    them are not written.  Returns (codes uint8 [M, I], scales f32 [I/128, M])."""
    G, N2, K = b.shape
    I = N2 // 2
    M = a.shape[0]
    dev = a.device
    for t in (a, a_scales, b, b_scales, offsets):
        assert t.is_contiguous()
    if out is None:
        out = torch.empty((M, I), dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty((I // 128, M), dtype=torch.float32, device=dev)
    st = load_library().fgg_grouped_gemm_silu_quantize(
        G, M, I, K, _ptr(a), _ptr(a_scales), _q(Q_E4M3_1x128), _ptr(b), _ptr(b_scales), _q(Q_E4M3_128x128),
        _ptr(offsets), _ptr(counts), _ptr(out), _ptr(scales), _stream(dev))
    _check("fgg_grouped_gemm_silu_quantize", st)
    return out, scales


def pack_fp4_weights(b, b_scales, out=None, scales_out=None):
    """Re-lay out FP4 expert weights for the masked GEMM (fgg_pack_fp4_weights):
    b [G, N, K/2] uint8 E2M1 pairs and b_scales [G, N, K/32] uint8 E8M0 ->
    (b_tiled uint8 [G, N*K/2], s_tiled uint8 [G, (N/16)*ceil(K/512)*256]), used with
    b_qdesc=Q_E2M1_E8M0_1x32_TILED."""
    G, N, Kh = b.shape
    K = 2 * Kh
    for t in (b, b_scales):
        assert t.is_contiguous()
    lib = load_library()
    nb, ns = ctypes.c_size_t(0), ctypes.c_size_t(0)
    _check("fgg_pack_fp4_weights_bytes", lib.fgg_pack_fp4_weights_bytes(G, N, K, ctypes.byref(nb), ctypes.byref(ns)))
    dev = b.device
    if out is None:
        out = torch.empty((G, nb.value // max(G, 1)), dtype=torch.uint8, device=dev)
    if scales_out is None:
        scales_out = torch.empty((G, ns.value // max(G, 1)), dtype=torch.uint8, device=dev)
    assert out.numel() >= nb.value and scales_out.numel() >= ns.value
    st = lib.fgg_pack_fp4_weights(_ptr(b), _ptr(b_scales), G, N, K, _ptr(out), _ptr(scales_out), _stream(dev))
    _check("fgg_pack_fp4_weights", st)
    return out, scales_out


def _scaled_qdescs(qdesc):
    return {"fp8": (Q_E4M3_1x128, Q_E4M3_128x128), "w4a4": (Q_E2M1_1x16, Q_E2M1_1x16),
            "mxfp4": (Q_E2M1_E8M0_1x32, Q_E2M1_E8M0_1x32)}[qdesc]


def scaled_gemm_workspace_bytes(M: int, N: int, K: int, qdesc: str = "fp8", rank: int = 0) -> int:
    """Workspace bytes scaled_gemm needs (fgg_scaled_gemm_workspace)."""
    aq, bq = _scaled_qdescs(qdesc)
    epi = Epilogue(None, None, None, int(rank), None)
    n = ctypes.c_size_t(0)
    _check("fgg_scaled_gemm_workspace", load_library().fgg_scaled_gemm_workspace(
        M, N, K, _q(aq), _q(bq), ctypes.byref(epi), ctypes.byref(n)))
    return n.value


def scaled_gemm(a, a_scales, b, b_scales, qdesc="fp8", x_bf16=None, l_down=None, l_up=None, bias=None,
                out=None, workspace=None):
    """Dense case.  qdesc "fp8": a [M, K] e4m3 with [K/128, M] scales, b [N, K]
    with [N/128, K/128] scales.  qdesc "w4a4": a [M, K/2], b [N, K/2] packed
    E2M1 with [rows, K/16] fp32 scales; qdesc "mxfp4": the same codes with
    [rows, K/32] E8M0 scale bytes.  Both FP4 forms take an optional low-rank
    branch (x_bf16 [M, K], l_down [K, r], l_up [r, N], r = 32) and bias [N] (bf16)."""
    dev = a.device
    M = a.shape[0]
    N = b.shape[0]
    aq, bq = _scaled_qdescs(qdesc)
    K = a.shape[1] if qdesc == "fp8" else a.shape[1] * 2
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    epi = None
    if qdesc != "fp8" and (l_down is not None or bias is not None):
        rank = 0 if l_down is None else int(l_down.shape[1])
        epi = Epilogue(None if x_bf16 is None else x_bf16.data_ptr(),
                       None if l_down is None else l_down.data_ptr(),
                       None if l_up is None else l_up.data_ptr(), rank,
                       None if bias is None else bias.data_ptr())
    lib = load_library()
    nbytes = ctypes.c_size_t(0)
    _check("fgg_scaled_gemm_workspace", lib.fgg_scaled_gemm_workspace(
        M, N, K, _q(aq), _q(bq), ctypes.byref(epi) if epi is not None else None, ctypes.byref(nbytes)))
    if workspace is None and nbytes.value > 0:
        workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=dev)
    st = lib.fgg_scaled_gemm(M, N, K, _ptr(a), _ptr(a_scales), _q(aq), _ptr(b), _ptr(b_scales), _q(bq),
                             ctypes.byref(epi) if epi is not None else None, _ptr(out), out.stride(0),
                             _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev))
    _check("fgg_scaled_gemm", st)
    return out


def moe_combine(y, src_to_row, topk_w, out=None):
    """out[t] = Σ_j w[t, j] · y[src_to_row[t·k + j]] (bf16 [T, N])."""
    T, k = topk_w.shape
    N = y.shape[1]
    dev = y.device
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    st = load_library().fgg_moe_combine(_ptr(y), y.stride(0), _ptr(src_to_row), _ptr(topk_w), T, k, N,
                                         _ptr(out), out.stride(0), _stream(dev))
    _check("fgg_moe_combine", st)
    return out


def moe_down_combine_workspace_bytes(M: int) -> int:
    n = ctypes.c_size_t(0)
    _check("fgg_moe_down_combine_workspace", load_library().fgg_moe_down_combine_workspace(M, ctypes.byref(n)))
    return n.value


def moe_down_combine(a, a_scales, b, b_scales, offsets, counts, src_to_row, row_to_src, topk_w, y, out=None,
                     workspace=None):
    """Down GEMM and combine in one call (fgg_moe_down_combine): ``out`` equals
    ``moe_combine(grouped_gemm_scaled(a, ..., offsets, masked_m=counts), src_to_row, topk_w)``
    bit for bit.  ``y`` (bf16 [M, N]) receives the rows of tokens with two or more
    routed slots; rows of single-slot tokens go straight to ``out`` (bf16 [T, N])."""
    G, N, K = b.shape
    M = a.shape[0]
    T, k = topk_w.shape
    dev = a.device
    for t in (a, a_scales, b, b_scales, offsets, counts, src_to_row, row_to_src, topk_w):
        assert t.is_contiguous()
    if out is None:
        out = torch.empty((T, N), dtype=torch.bfloat16, device=dev)
    if workspace is None:
        workspace = torch.empty(moe_down_combine_workspace_bytes(M), dtype=torch.uint8, device=dev)
    st = load_library().fgg_moe_down_combine(
        G, M, N, K, _ptr(a), _ptr(a_scales), _q(Q_E4M3_1x128), _ptr(b), _ptr(b_scales), _q(Q_E4M3_128x128),
        _ptr(offsets), _ptr(counts), _ptr(src_to_row), _ptr(row_to_src), _ptr(topk_w), T, k, _ptr(y), y.stride(0),
        _ptr(workspace), workspace.numel(), _ptr(out), out.stride(0), _stream(dev))
    _check("fgg_moe_down_combine", st)
    return out


# ---------------------------------------------- router, rows in bf16/fp32, few tokens

_FLOAT = {torch.float32: FGG_F32, torch.bfloat16: FGG_BF16}
_GATES = {"softmax": FGG_GATE_SOFTMAX, "sigmoid": FGG_GATE_SIGMOID}


# These calls are small enough for the host's share to count (a launch is 3.2 us): the current
# stream's handle is asked for directly where torch offers that (0.1 us; the Stream object
# costs 1.9), and outputs made here are not checked.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_QDESC = {}


def _call(name, dev, *args):
    """Call the entry point on dev's current stream, with dev as the current device."""
    fn = getattr(_lib or load_library(), name)
    index = dev.index
    if index == _current_device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(index))
    if status != 0:
        _check(name, status)


def _addr(t):
    return None if t is None else t.data_ptr()


def _float_rows(t, name, dtype=None):
    """A 2-D fp32/bf16 CUDA tensor with unit column stride and rows that do not overlap; returns its row stride."""
    shape, dt = t.shape, t.dtype
    assert t.is_cuda and len(shape) == 2 and dt in _FLOAT and (dtype is None or dt == dtype), name
    ld, unit = t.stride()
    n = shape[1]
    assert unit == 1 or n <= 1, name
    if shape[0] <= 1 and ld < n:
        ld = n
    assert ld >= n, name
    return ld


def _dense(t, name, dev, dtype, shape=None, numel=None):
    """A contiguous tensor of the given type and shape (or number of elements) on dev, or None."""
    if t is None:
        return
    assert t.dtype == dtype and t.is_contiguous() and t.device == dev, name
    assert (shape is None or t.shape == shape) and (numel is None or t.numel() == numel), name


def moe_route(logits, k, gate="softmax", bias=None, renormalize=False, scale=1.0, ids=None, weights=None):
    """The router (fgg_moe_route): logits [T, E] (fp32 or bf16, rows may be strided) to
    (topk_ids int32 [T, k], topk_w fp32 [T, k]) in decreasing order, ties to the lower
    expert.  gate "softmax" or "sigmoid"; bias (fp32 [E]) enters the selection only;
    renormalize divides the weights by their sum over the k; scale multiplies them.
    Experts at -inf are never chosen; slots left over have id -1 and weight 0."""
    ld = _float_rows(logits, "logits")
    T, E = logits.shape
    k, dev = int(k), logits.device
    _dense(bias, "bias", dev, torch.float32, (E,))
    _dense(ids, "ids", dev, torch.int32, (T, k))
    _dense(weights, "weights", dev, torch.float32, (T, k))
    if ids is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if weights is None:
        weights = torch.empty((T, k), dtype=torch.float32, device=dev)
    _call("fgg_moe_route", dev, logits.data_ptr(), _FLOAT[logits.dtype], T, E, ld, k, _GATES[gate], _addr(bias),
          1 if renormalize else 0, float(scale), ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_route_backward(logits, topk_ids, dtopk_w, gate="softmax", renormalize=False, scale=1.0, out=None):
    """Gradient of moe_route's logits ([T, E], the logits' type) from that of its weights
    (fp32 [T, k]) at the ids it chose (fgg_moe_route_backward)."""
    ld = _float_rows(logits, "logits")
    T, E = logits.shape
    k, dev = topk_ids.shape[1], logits.device
    out, ldo = _rows_out(out, (T, E), logits, "out")
    _dense(topk_ids, "topk_ids", dev, torch.int32, (T, k))
    _dense(dtopk_w, "dtopk_w", dev, torch.float32, (T, k))
    _call("fgg_moe_route_backward", dev, logits.data_ptr(), _FLOAT[logits.dtype], T, E, ld, k, _GATES[gate],
          1 if renormalize else 0, float(scale), topk_ids.data_ptr(), dtopk_w.data_ptr(), out.data_ptr(), ldo)
    return out


def _slots(src_to_row, T, topk_w, dev):
    """k, from the T * k entries of the map (of no token: from the weights, or 1)."""
    _dense(src_to_row, "src_to_row", dev, torch.int32)
    if T == 0:
        return 1 if topk_w is None else topk_w.shape[1]
    assert src_to_row.numel() % T == 0, "src_to_row holds T * k pairs"
    return src_to_row.numel() // T


def _rows_out(out, shape, like, name):
    if out is None:
        return like.new_empty(shape), shape[1]
    ld = _float_rows(out, name, like.dtype)
    assert out.shape == shape and out.device == like.device, name
    return out, ld


def moe_permute_rows(x, src_to_row, row_to_src, offsets, topk_w=None, out=None):
    """Token rows (fp32 or bf16 [T, N]) in the order of moe_permute's maps, optionally scaled
    by topk_w (fp32 [T, k]): out [M, N] with M = row_to_src's length (fgg_moe_permute_rows).
    Padding rows are zeroed; rows past offsets[E] are left as they were."""
    ldx = _float_rows(x, "x")
    T, N = x.shape
    dev, M = x.device, row_to_src.numel()
    k = _slots(src_to_row, T, topk_w, dev)
    out, ldr = _rows_out(out, (M, N), x, "out")
    _dense(row_to_src, "row_to_src", dev, torch.int32)
    _dense(offsets, "offsets", dev, torch.int32)
    _dense(topk_w, "topk_w", dev, torch.float32, (T, k))
    _call("fgg_moe_permute_rows", dev, x.data_ptr(), _FLOAT[x.dtype], T, k, N, ldx, _addr(topk_w),
          src_to_row.data_ptr(), row_to_src.data_ptr(), offsets.data_ptr(), offsets.numel() - 1, M, out.data_ptr(),
          ldr)
    return out


def moe_permute_rows_backward(drows, src_to_row, T, topk_w=None, x=None, out=None):
    """Gradients of moe_permute_rows: (dx [T, N], dtopk_w fp32 [T, k] or None).  dtopk_w is
    computed when the forward's input x is given (fgg_moe_permute_rows_backward)."""
    lddr = _float_rows(drows, "drows")
    M, N = drows.shape
    dev = drows.device
    k = _slots(src_to_row, T, topk_w, dev)
    dx, lddx = _rows_out(out, (T, N), drows, "out")
    _dense(topk_w, "topk_w", dev, torch.float32, (T, k))
    dw, ldx = None, 0
    if x is not None:
        ldx = _float_rows(x, "x", drows.dtype)
        assert x.device == dev and x.shape == (T, N), "x"
        dw = torch.empty((T, k), dtype=torch.float32, device=dev)
    _call("fgg_moe_permute_rows_backward", dev, drows.data_ptr(), _FLOAT[drows.dtype], M, lddr, _addr(x), ldx,
          _addr(topk_w), src_to_row.data_ptr(), T, k, N, dx.data_ptr(), lddx, _addr(dw))
    return dx, dw


def moe_unpermute_rows(rows, src_to_row, T, topk_w=None, out=None):
    """out[t] = sum_j w[t, j] * rows[src_to_row[t k + j]] in the rows' type (fp32 or bf16,
    [M, N] -> [T, N]; weights of 1 without topk_w) (fgg_moe_unpermute_rows)."""
    ldr = _float_rows(rows, "rows")
    M, N = rows.shape
    dev = rows.device
    k = _slots(src_to_row, T, topk_w, dev)
    out, ldo = _rows_out(out, (T, N), rows, "out")
    _dense(topk_w, "topk_w", dev, torch.float32, (T, k))
    _call("fgg_moe_unpermute_rows", dev, rows.data_ptr(), _FLOAT[rows.dtype], M, ldr, _addr(topk_w),
          src_to_row.data_ptr(), T, k, N, out.data_ptr(), ldo)
    return out


def moe_unpermute_rows_backward(dout, src_to_row, row_to_src, offsets, topk_w=None, rows=None, out=None):
    """Gradients of moe_unpermute_rows: (drows [M, N], dtopk_w fp32 [T, k] or None).  dtopk_w
    is computed when the forward's rows are given (fgg_moe_unpermute_rows_backward)."""
    lddo = _float_rows(dout, "dout")
    T, N = dout.shape
    dev, M = dout.device, row_to_src.numel()
    k = _slots(src_to_row, T, topk_w, dev)
    drows, lddr = _rows_out(out, (M, N), dout, "out")
    _dense(row_to_src, "row_to_src", dev, torch.int32)
    _dense(offsets, "offsets", dev, torch.int32)
    _dense(topk_w, "topk_w", dev, torch.float32, (T, k))
    dw, ldr = None, 0
    if rows is not None:
        ldr = _float_rows(rows, "rows", dout.dtype)
        assert rows.device == dev and rows.shape == (M, N), "rows"
        dw = torch.empty((T, k), dtype=torch.float32, device=dev)
    _call("fgg_moe_unpermute_rows_backward", dev, dout.data_ptr(), _FLOAT[dout.dtype], T, k, N, lddo, _addr(rows), ldr,
          _addr(topk_w), src_to_row.data_ptr(), row_to_src.data_ptr(), offsets.data_ptr(), offsets.numel() - 1, M,
          drows.data_ptr(), lddr, _addr(dw))
    return drows, dw


def moe_gemv_fp4(x, b, b_scales, topk_ids=None, topk_w=None, b_qdesc=Q_E2M1_E8M0_1x32, n=None, silu_mul=False,
                 out=None, out_dtype=torch.bfloat16):
    """Few tokens times FP4 expert weights, activations unquantized (fgg_moe_gemv_fp4).

    x: fp32/bf16 [T, K] (every slot of a token reads its row) or [T, k, K] (a row per slot).
    b, b_scales: [G, N, K/2], [G, N, K/32] (with silu_mul 2N rows, [gate | up]), or their
    tiled form (Q_E2M1_E8M0_1x32_TILED, from pack_fp4_weights; ``n`` gives N, the output columns).
    topk_ids int32 [T, k]: the result is [T, k, N]; with topk_w (fp32 [T, k]) the
    gate-weighted sum over the slots, [T, N].  Without topk_ids (G = 1): [T, N]."""
    per_slot = x.dim() == 3
    assert x.is_cuda and (per_slot or x.dim() == 2) and x.dtype in _FLOAT and out_dtype in _FLOAT, "x"
    T, K = x.shape[0], x.shape[-1]
    dev, G = x.device, b.shape[0]
    k = 1 if topk_ids is None else topk_ids.shape[1]
    if per_slot:
        assert x.shape[1] == k and x.is_contiguous(), "x"
        ldx = K
    else:
        ldx = _float_rows(x, "x")
    rows = 2 if silu_mul else 1
    if b_qdesc == Q_E2M1_E8M0_1x32_TILED:
        assert n is not None, "n"
        N = int(n)
        _dense(b, "b", dev, torch.uint8, numel=G * rows * N * K // 2)
        _dense(b_scales, "b_scales", dev, torch.uint8, numel=G * (rows * N // 16) * ((K + 511) // 512) * 256)
    else:
        assert b.shape[1] % rows == 0 and (n is None or int(n) * rows == b.shape[1]), "n"
        N = b.shape[1] // rows
        _dense(b, "b", dev, torch.uint8, (G, rows * N, K // 2))
        _dense(b_scales, "b_scales", dev, torch.uint8, (G, rows * N, K // 32))
    _dense(topk_ids, "topk_ids", dev, torch.int32, (T, k))
    _dense(topk_w, "topk_w", dev, torch.float32, (T, k))
    shape = (T, N) if topk_ids is None or topk_w is not None else (T, k, N)
    ldo = N
    if out is None:
        out = torch.empty(shape, dtype=out_dtype, device=dev)
    else:
        assert out.device == dev and out.dtype in _FLOAT and out.shape == shape, "out"
        assert out.is_contiguous() or out.dim() == 2, "out"
        if out.dim() == 2:
            ldo = _float_rows(out, "out")
    desc = _QDESC.get(b_qdesc)
    if desc is None:
        desc = _QDESC[b_qdesc] = QDesc(*b_qdesc)
    _call("fgg_moe_gemv_fp4", dev, G, T, k, N, K, x.data_ptr(), _FLOAT[x.dtype], ldx, 1 if per_slot else 0,
          b.data_ptr(), b_scales.data_ptr(), desc, _addr(topk_ids), _addr(topk_w),
          FGG_ACT_SILU_MUL if silu_mul else FGG_ACT_NONE, out.data_ptr(), _FLOAT[out.dtype], ldo)
    return out


# ------------------------------------------ bf16 rows times their segment's weights

def _segments(offsets, counts, G, dev):
    _dense(offsets, "offsets", dev, torch.int32, (G + 1,))
    _dense(counts, "counts", dev, torch.int32, (G,))
    assert offsets is not None or G == 1, "offsets"


def _rows_of(t, name, dtype=None):
    """_float_rows, with a single row's stride taken as its width (whatever matrix it is a row of)."""
    ld = _float_rows(t, name, dtype)
    return ld if t.shape[0] > 1 else t.shape[1]


def _bf16_out(out, shape, dtype, dev, name):
    """The given output (checked) or a new one, and its row stride."""
    if out is None:
        assert dtype in _FLOAT, name
        return torch.empty(shape, dtype=dtype, device=dev), shape[1]
    ld = _rows_of(out, name)
    assert out.shape == shape and out.device == dev, name
    return out, ld


def grouped_linear(x, w, offsets=None, counts=None, out=None, out_dtype=torch.bfloat16):
    """Rows times their segment's weights (fgg_grouped_linear): x bf16 [M, K] (rows may be strided), w bf16
    [G, N, K], segment g the rows [offsets[g], offsets[g + 1]) (of which the first counts[g]); without
    offsets one segment (G = 1).  Returns [M, N], bf16 or fp32; rows of no segment are left as ``out`` had them."""
    ldx = _rows_of(x, "x", torch.bfloat16)
    (M, K), dev = x.shape, x.device
    G, N = w.shape[0], w.shape[1]
    _dense(w, "w", dev, torch.bfloat16, (G, N, K))
    _segments(offsets, counts, G, dev)
    out, ldo = _bf16_out(out, (M, N), out_dtype, dev, "out")
    _call("fgg_grouped_linear", dev, G, M, N, K, x.data_ptr(), ldx, w.data_ptr(), _addr(offsets), _addr(counts),
          out.data_ptr(), _FLOAT[out.dtype], ldo)
    return out


def grouped_linear_backward_input(dy, w, offsets=None, counts=None, out=None, out_dtype=torch.bfloat16):
    """Gradient of grouped_linear's rows (fgg_grouped_linear_backward_input): dy bf16 [M, N], w bf16 [G, N, K];
    returns [M, K], bf16 or fp32, rows of no segment left as ``out`` had them."""
    lddy = _rows_of(dy, "dy", torch.bfloat16)
    (M, N), dev = dy.shape, dy.device
    G, K = w.shape[0], w.shape[2]
    _dense(w, "w", dev, torch.bfloat16, (G, N, K))
    _segments(offsets, counts, G, dev)
    out, ldo = _bf16_out(out, (M, K), out_dtype, dev, "out")
    _call("fgg_grouped_linear_backward_input", dev, G, M, N, K, dy.data_ptr(), lddy, w.data_ptr(), _addr(offsets),
          _addr(counts), out.data_ptr(), _FLOAT[out.dtype], ldo)
    return out


def grouped_linear_backward_weight_workspace_bytes(G: int, M: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check("fgg_grouped_linear_backward_weight_workspace",
           load_library().fgg_grouped_linear_backward_weight_workspace(G, M, N, K, ctypes.byref(n)))
    return n.value


def grouped_linear_backward_weight(dy, x, num_groups, offsets=None, counts=None, out=None, out_dtype=torch.float32,
                                   accumulate=False, workspace=None):
    """Gradient of grouped_linear's weights (fgg_grouped_linear_backward_weight): dy bf16 [M, N], x bf16 [M, K];
    returns [G, N, K], fp32 or bf16 (0 for an empty segment); accumulate adds to ``out``."""
    lddy, ldx = _rows_of(dy, "dy", torch.bfloat16), _rows_of(x, "x", torch.bfloat16)
    (M, N), K, dev, G = dy.shape, x.shape[1], dy.device, int(num_groups)
    assert x.shape[0] == M and x.device == dev, "x"
    _segments(offsets, counts, G, dev)
    if out is None:
        assert not accumulate and out_dtype in _FLOAT, "accumulate adds to out"
        out = torch.empty((G, N, K), dtype=out_dtype, device=dev)
    else:
        assert out.dtype in _FLOAT, "out"
        _dense(out, "out", dev, out.dtype, (G, N, K))
    nbytes = grouped_linear_backward_weight_workspace_bytes(G, M, N, K)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _dense(workspace, "workspace", dev, torch.uint8)
    _call("fgg_grouped_linear_backward_weight", dev, G, M, N, K, dy.data_ptr(), lddy, x.data_ptr(), ldx,
          _addr(offsets), _addr(counts), out.data_ptr(), _FLOAT[out.dtype], 1 if accumulate else 0, _addr(workspace),
          0 if workspace is None else workspace.numel())
    return out


def grouped_gated(x, w, offsets=None, counts=None, out=None, h=None):
    """The gated block's first half (fgg_grouped_gated): x bf16 [M, K], w bf16 [G, 2I, K] ([gate | up] rows);
    a = silu(gate) * up, bf16 [M, I].  h (bf16 [M, 2I], optional) receives the pre-activations that
    the backward pass needs.  Returns (a, h); rows of no segment are left as they were."""
    ldx = _rows_of(x, "x", torch.bfloat16)
    (M, K), dev = x.shape, x.device
    G, I = w.shape[0], w.shape[1] // 2
    _dense(w, "w", dev, torch.bfloat16, (G, 2 * I, K))
    _segments(offsets, counts, G, dev)
    out, lda = _bf16_out(out, (M, I), torch.bfloat16, dev, "out")
    assert out.dtype == torch.bfloat16, "out"
    ldh = 0
    if h is not None:
        ldh = _rows_of(h, "h", torch.bfloat16)
        assert h.shape == (M, 2 * I) and h.device == dev, "h"
    _call("fgg_grouped_gated", dev, G, M, I, K, x.data_ptr(), ldx, w.data_ptr(), _addr(offsets), _addr(counts),
          out.data_ptr(), lda, _addr(h), ldh)
    return out, h


def grouped_gated_backward(dy, w_down, h, offsets=None, counts=None, out=None, a=None):
    """From the gradient of the block's output to that of its pre-activations (fgg_grouped_gated_backward):
    dy bf16 [M, N], w_down bf16 [G, N, I], h bf16 [M, 2I] from grouped_gated; returns (dh bf16 [M, 2I], a).
    a (bf16 [M, I], optional) receives the activation again, which w_down's gradient needs."""
    lddy, ldh = _rows_of(dy, "dy", torch.bfloat16), _rows_of(h, "h", torch.bfloat16)
    (M, N), dev = dy.shape, dy.device
    G, I = w_down.shape[0], w_down.shape[2]
    _dense(w_down, "w_down", dev, torch.bfloat16, (G, N, I))
    assert h.shape == (M, 2 * I) and h.device == dev, "h"
    _segments(offsets, counts, G, dev)
    out, ldo = _bf16_out(out, (M, 2 * I), torch.bfloat16, dev, "out")
    assert out.dtype == torch.bfloat16, "out"
    lda = 0
    if a is not None:
        lda = _rows_of(a, "a", torch.bfloat16)
        assert a.shape == (M, I) and a.device == dev, "a"
    _call("fgg_grouped_gated_backward", dev, G, M, I, N, dy.data_ptr(), lddy, w_down.data_ptr(), h.data_ptr(), ldh,
          _addr(offsets), _addr(counts), out.data_ptr(), ldo, _addr(a), lda)
    return out, a


# ------------------------------------------------------------- low-rank adapters

def lora_workspace_bytes(T: int, L: int, r: int, N: int, K: int) -> int:
    n = ctypes.c_size_t(0)
    _check("fgg_lora_workspace", load_library().fgg_lora_workspace(T, L, r, N, K, ctypes.byref(n)))
    return n.value


def lora_add(base, x, ids, a, b, scales=None, out=None, workspace=None):
    """Low-rank adapters beside a shared projection (fgg_lora_add): out[t] = base[t] + scales[i] (x[t] a[i]^T) b[i]^T,
    i = ids[t] (outside [0, L): base[t]).  base [T, N] fp32 or bf16, x bf16 [T, K], ids int32 [T], a bf16 [L, r, K],
    b bf16 [L, N, r], scales fp32 [L].  ``out`` may be ``base`` itself; workspace: lora_workspace_bytes, uint8."""
    ldb, ldx = _rows_of(base, "base"), _rows_of(x, "x", torch.bfloat16)
    (T, K), N, dev = x.shape, base.shape[1], x.device
    L, r = a.shape[0], a.shape[1]
    assert base.shape[0] == T and base.device == dev, "base"
    _dense(ids, "ids", dev, torch.int32, (T,))
    _dense(a, "a", dev, torch.bfloat16, (L, r, K))
    _dense(b, "b", dev, torch.bfloat16, (L, N, r))
    _dense(scales, "scales", dev, torch.float32, (L,))
    if out is None:
        out, ldo = base.new_empty((T, N)), N
    else:
        ldo = _rows_of(out, "out", base.dtype)
        assert out.shape == (T, N) and out.device == dev, "out"
    if workspace is None:
        nbytes = lora_workspace_bytes(T, L, r, N, K)
        if nbytes > 0:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _dense(workspace, "workspace", dev, torch.uint8)
    _call("fgg_lora_add", dev, T, L, r, N, K, x.data_ptr(), ldx, ids.data_ptr(), a.data_ptr(), b.data_ptr(),
          _addr(scales), base.data_ptr(), ldb, out.data_ptr(), _FLOAT[base.dtype], ldo, _addr(workspace),
          0 if workspace is None else workspace.numel())
    return out
