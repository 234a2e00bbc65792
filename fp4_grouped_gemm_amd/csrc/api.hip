// C ABI of libfgg.so: argument validation, device check and dispatch to the
// kernels.  Every entry point either returns an error before launching
// anything or enqueues its kernels on the caller's stream and returns.
#include <hip/hip_runtime.h>

#include <array>
#include <atomic>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "../../include/fgg.h"
#include "fgg_internal.hpp"

namespace {

thread_local int g_last_hip_error = 0;
std::atomic<int> g_num_cus_override{0};

constexpr int kMaxDevices = 64;
struct DeviceInfo {
  std::once_flag once;
  bool gfx950 = false;
  int num_cus = 0;
};
DeviceInfo g_dev[kMaxDevices];

fgg_status hip_fail(hipError_t e) {
  g_last_hip_error = (int)e;
  return FGG_ERR_HIP;
}

// Current device must be gfx950; fills num_cus.
fgg_status device_check(int* num_cus) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return FGG_ERR_UNSUPPORTED;
  DeviceInfo& d = g_dev[dev];
  std::call_once(d.once, [&] {
    hipDeviceProp_t p;
    if (hipGetDeviceProperties(&p, dev) != hipSuccess) return;
    d.gfx950 = std::strncmp(p.gcnArchName, "gfx950", 6) == 0;
    d.num_cus = p.multiProcessorCount;
  });
  if (!d.gfx950) return FGG_ERR_UNSUPPORTED;
  const int ov = g_num_cus_override.load();
  if (num_cus) *num_cus = ov > 0 ? ov : d.num_cus;
  return FGG_OK;
}

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool same_q(const fgg_qdesc& q, fgg_dtype data, fgg_dtype scale, int br, int bk) {
  return q.data == data && q.scale == scale && q.block_rows == br && q.block_k == bk;
}

fgg_status finish(hipError_t e) { return e == hipSuccess ? FGG_OK : hip_fail(e); }

// The activations' own types: fp32 or bf16, and the alignment of one element.
bool float_type(fgg_dtype t) { return t == FGG_F32 || t == FGG_BF16; }
size_t float_size(fgg_dtype t) { return t == FGG_F32 ? 4 : 2; }

}  // namespace

namespace fgg {

bool debug_enabled() {
  static const bool on = [] {
    const char* e = std::getenv("FGG_DEBUG");
    return e != nullptr && e[0] != '\0' && e[0] != '0';
  }();
  return on;
}

void trace_launch(const KernelInfo& k, dim3 grid, const char* fmt, ...) {
  if (!debug_enabled()) return;
  char what[256];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(what, sizeof what, fmt, ap);
  va_end(ap);
  std::fprintf(stderr, "[fgg] %s: %s | grid=%u threads=%d tile=%dx%dx%d lds=%d B (%d x %d stage + %d) \n", k.name,
               what, grid.x * grid.y * grid.z, k.threads, k.tile_m, k.tile_n, k.tile_k, k.lds_bytes, k.stages,
               k.stage_bytes, k.other_bytes);
}

int kernel_table(const KernelInfo* const** out) {
  static const KernelInfo* const single[] = {
      &kInfoQuantE4m3_1x128, &kInfoQuantE4m3_128x128, &kInfoQuantE2m1_1x16, &kInfoQuantE2m1E8m0_1x32,
      &kInfoPermuteHist,     &kInfoPermuteScan,       &kInfoPermuteScatter, &kInfoPermuteGather,
      &kInfoPermuteQuantize, &kInfoFill,              &kInfoCombine,        &kInfoCombineRows,
      &kInfoCombineRest,     &kInfoFp8Contig,         &kInfoFp8ContigSilu,  &kInfoFp8ContigCombine,
      &kInfoFp8Dense,        &kInfoMaskedFp4Tiled,    &kInfoMaskedFp4,
      &kInfoMaskedFp8,       &kInfoPackFp4,           &kInfoPackFp4Scales,  &kInfoW4a4Prep,
      &kInfoW4a4LowRank,     &kInfoW4a4Gemm,         &kInfoMxfp4Gemm,
      &kInfoRoute,           &kInfoRowsScatter,       &kInfoRowsCollect,    &kInfoRowsScatterDot,
      &kInfoRowsCollectDot,
  };
  constexpr int kSingle = (int)(sizeof single / sizeof single[0]);
  static const auto table = [] {
    std::array<const KernelInfo*, kSingle + kRouteBackwardForms + kGemvForms + kGemmBf16Forms + kLoraForms + 7> t{};
    int n = 0;
    for (const KernelInfo* k : single) t[n++] = k;
    for (const KernelInfo& k : kInfoRouteBackward) t[n++] = &k;
    for (const KernelInfo& k : kInfoGemvFp4) t[n++] = &k;
    for (const KernelInfo& k : kInfoGemmBf16) t[n++] = &k;
    for (const KernelInfo& k : kInfoLora) t[n++] = &k;
    for (const KernelInfo& k : kInfoRowsBf16) t[n++] = &k;
    for (const KernelInfo& k : kInfoDwJoin) t[n++] = &k;
    t[n++] = &kInfoLoraTiles;
    return t;
  }();
  *out = table.data();
  return (int)table.size();
}

}  // namespace fgg

// The C ABI is the library's only export (the build hides everything else).
#pragma GCC visibility push(default)
extern "C" {

const char* fgg_status_string(fgg_status s) {
  switch (s) {
    case FGG_OK: return "FGG_OK";
    case FGG_ERR_INVALID_VALUE: return "FGG_ERR_INVALID_VALUE";
    case FGG_ERR_UNSUPPORTED: return "FGG_ERR_UNSUPPORTED";
    case FGG_ERR_HIP: return "FGG_ERR_HIP";
  }
  return "FGG_ERR_UNKNOWN";
}

int fgg_last_hip_error(void) { return g_last_hip_error; }

fgg_status fgg_set_num_cus(int n) {
  if (n < 0) return FGG_ERR_INVALID_VALUE;
  g_num_cus_override.store(n);
  return FGG_OK;
}

fgg_status fgg_quantize_blockwise(const void* x, fgg_dtype x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                                  fgg_act act, fgg_qdesc q, const int32_t* rows_dev, void* q_out, void* scales_out,
                                  void* stream) {
  if (rows < 0 || cols < 0) return FGG_ERR_INVALID_VALUE;
  if (x_dtype != FGG_F32 && x_dtype != FGG_BF16) return FGG_ERR_UNSUPPORTED;
  if (act != FGG_ACT_NONE && act != FGG_ACT_SILU_MUL) return FGG_ERR_INVALID_VALUE;
  fgg::QuantKind kind;
  if (same_q(q, FGG_E4M3, FGG_F32, 1, 128)) kind = fgg::QuantKind::E4M3_1x128;
  else if (same_q(q, FGG_E4M3, FGG_F32, 128, 128)) kind = fgg::QuantKind::E4M3_128x128;
  else if (same_q(q, FGG_E2M1X2, FGG_F32, 1, 16)) kind = fgg::QuantKind::E2M1_1x16;
  else if (same_q(q, FGG_E2M1X2, FGG_E8M0, 1, 32)) kind = fgg::QuantKind::E2M1_E8M0_1x32;
  else return FGG_ERR_UNSUPPORTED;
  const bool silu = act == FGG_ACT_SILU_MUL;
  if (silu && kind != fgg::QuantKind::E4M3_1x128) return FGG_ERR_UNSUPPORTED;
  if (rows_dev && kind != fgg::QuantKind::E4M3_1x128) return FGG_ERR_UNSUPPORTED;
  if (cols % q.block_k != 0) return FGG_ERR_UNSUPPORTED;
  if (q.block_rows == 128 && rows % 128 != 0) return FGG_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return FGG_OK;
  if (!x || !q_out || !scales_out) return FGG_ERR_INVALID_VALUE;
  const int64_t need = silu ? 2 * cols : cols;
  if (ldx < need) return FGG_ERR_INVALID_VALUE;
  const int64_t esz = x_dtype == FGG_F32 ? 4 : 2;
  if (!aligned(x, 16) || (ldx * esz) % 16 != 0 || !aligned(q_out, 16) || !aligned(scales_out, 4))
    return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_quantize(x, x_dtype == FGG_BF16, rows, cols, ldx, kind, silu, rows_dev, q_out,
                                     scales_out, num_cus, (hipStream_t)stream));
}

fgg_status fgg_moe_permute_workspace(int64_t T, int32_t k, int32_t E, size_t* bytes) {
  if (!bytes || T < 0 || k < 1 || k > 64 || E < 1 || E > 1024) return FGG_ERR_INVALID_VALUE;
  *bytes = fgg::permute_workspace_bytes(T, k, E);
  return FGG_OK;
}

fgg_status fgg_moe_permute(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E, int32_t align,
                           const void* xq, const float* xs, int64_t K, int32_t* offsets, int32_t* counts,
                           int32_t* src_to_row, int32_t* row_to_src, void* a_out, float* sa_out,
                           int64_t M_cap, void* workspace, size_t ws_bytes, void* stream) {
  if (T < 0 || k < 1 || k > 64 || E < 1 || E > 1024 || align < 1 || align > 1024 || M_cap < 0)
    return FGG_ERR_INVALID_VALUE;
  if (!offsets || !counts) return FGG_ERR_INVALID_VALUE;
  if (T > 0 && (!topk_ids || !src_to_row)) return FGG_ERR_INVALID_VALUE;
  if (M_cap > 0 && !row_to_src) return FGG_ERR_INVALID_VALUE;
  if (T * (int64_t)k > (int64_t)INT32_MAX || M_cap > (int64_t)INT32_MAX) return FGG_ERR_UNSUPPORTED;
  if (xq) {
    if (K <= 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
    if (!xs || !a_out || !sa_out) return FGG_ERR_INVALID_VALUE;
    if (!aligned(xq, 16) || !aligned(a_out, 16) || !aligned(xs, 4) || !aligned(sa_out, 4))
      return FGG_ERR_INVALID_VALUE;
  }
  if (T > 0 && (!workspace || ws_bytes < fgg::permute_workspace_bytes(T, k, E))) return FGG_ERR_INVALID_VALUE;
  fgg_status st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_permute(topk_ids, T, k, E, align, (const uint8_t*)xq, xs, K, offsets, counts,
                                    src_to_row, row_to_src, (uint8_t*)a_out, sa_out, M_cap, workspace,
                                    (hipStream_t)stream));
}

fgg_status fgg_moe_permute_quantize(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E, int32_t align,
                                    const void* x, fgg_dtype x_dtype, int64_t K, int64_t ldx, int32_t* offsets,
                                    int32_t* counts, int32_t* src_to_row, int32_t* row_to_src, void* a_out,
                                    float* sa_out, int64_t M_cap, void* workspace, size_t ws_bytes, void* stream) {
  if (T < 0 || k < 1 || k > 64 || E < 1 || E > 1024 || align < 1 || align > 1024 || M_cap < 0 || K < 0)
    return FGG_ERR_INVALID_VALUE;
  if (x_dtype != FGG_BF16 && x_dtype != FGG_F32) return FGG_ERR_UNSUPPORTED;
  if (K == 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
  if (!offsets || !counts) return FGG_ERR_INVALID_VALUE;
  if (T > 0 && (!topk_ids || !src_to_row || !x)) return FGG_ERR_INVALID_VALUE;
  if (M_cap > 0 && (!row_to_src || !a_out || !sa_out)) return FGG_ERR_INVALID_VALUE;
  if (T * (int64_t)k > (int64_t)INT32_MAX || M_cap > (int64_t)INT32_MAX) return FGG_ERR_UNSUPPORTED;
  const int64_t esz = x_dtype == FGG_F32 ? 4 : 2;
  if (T > 0 && (ldx < K || !aligned(x, 16) || (ldx * esz) % 16 != 0)) return FGG_ERR_INVALID_VALUE;
  if (M_cap > 0 && (!aligned(a_out, 16) || !aligned(sa_out, 4))) return FGG_ERR_INVALID_VALUE;
  if (T > 0 && (!workspace || ws_bytes < fgg::permute_workspace_bytes(T, k, E))) return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_permute_quantize(topk_ids, T, k, E, align, x, x_dtype == FGG_BF16, K, ldx, offsets,
                                             counts, src_to_row, row_to_src, (uint8_t*)a_out, sa_out, M_cap,
                                             workspace, num_cus, (hipStream_t)stream));
}

fgg_status fgg_moe_permute_quantize_noalloc(const int32_t* topk_ids, int64_t T, int32_t k, int32_t E, int32_t align,
                                            const void* x, fgg_dtype x_dtype, int64_t K, int64_t ldx,
                                            int32_t* offsets, int32_t* counts, int32_t* src_to_row,
                                            int32_t* row_to_src, void* a_out, float* sa_out, int64_t M_cap,
                                            void* stream) {
  if (T < 0 || k < 1 || k > 64 || E < 1 || E > 1024) return FGG_ERR_INVALID_VALUE;
  if (T > 0 && fgg::permute_workspace_bytes(T, k, E) > fgg::kPermuteScratchBytes) return FGG_ERR_UNSUPPORTED;
  void* ws = nullptr;
  if (T > 0) {
    fgg_status st = device_check(nullptr);
    if (st != FGG_OK) return st;
    const hipError_t e = fgg::permute_scratch(&ws);
    if (e != hipSuccess) return hip_fail(e);
  }
  return fgg_moe_permute_quantize(topk_ids, T, k, E, align, x, x_dtype, K, ldx, offsets, counts, src_to_row,
                                  row_to_src, a_out, sa_out, M_cap, ws, fgg::kPermuteScratchBytes, stream);
}

fgg_status fgg_grouped_gemm_scaled(fgg_layout layout, int32_t G, int64_t M, int64_t N, int64_t K,
                                   const void* a, const void* a_scales, fgg_qdesc aq, const void* b,
                                   const void* b_scales, fgg_qdesc bq, const int32_t* offsets,
                                   const int32_t* masked_m, void* d, int64_t ldd, void* stream) {
  if (G < 1 || G > 1024 || M < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  if (N % 128 != 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
  if (ldd < N || ldd % 8 != 0) return FGG_ERR_INVALID_VALUE;
  if (!same_q(aq, FGG_E4M3, FGG_F32, 1, 128)) return FGG_ERR_UNSUPPORTED;
  // (with K == 0 the operands hold no bytes and are never read: they may be NULL)
  if ((K > 0 && (!a || !a_scales || !b || !b_scales)) || !d) return FGG_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4))
    return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  if (layout == FGG_LAYOUT_CONTIGUOUS) {
    if (!same_q(bq, FGG_E4M3, FGG_F32, 128, 128)) return FGG_ERR_UNSUPPORTED;
    if (K > 16384) return FGG_ERR_UNSUPPORTED;
    if (!offsets) return FGG_ERR_INVALID_VALUE;
    fgg_status st = device_check(&num_cus);
    if (st != FGG_OK) return st;
    if (M == 0 || N == 0) return FGG_OK;
    return finish(fgg::launch_gemm_fp8_contig(G, M, N, K, (const uint8_t*)a, (const float*)a_scales,
                                              (const uint8_t*)b, (const float*)b_scales, offsets, masked_m,
                                              (uint16_t*)d, ldd, num_cus, (hipStream_t)stream));
  }
  if (layout == FGG_LAYOUT_MASKED) {
    const bool tiled = same_q(bq, FGG_E2M1X2_TILED, FGG_E8M0, 1, 32);
    const bool fp4 = tiled || same_q(bq, FGG_E2M1X2, FGG_E8M0, 1, 32);
    if (!fp4 && !same_q(bq, FGG_E4M3, FGG_F32, 128, 128)) return FGG_ERR_UNSUPPORTED;
    if (M > 16 || K == 0) return FGG_ERR_UNSUPPORTED;
    if (!masked_m) return FGG_ERR_INVALID_VALUE;
    if (tiled && !aligned(b_scales, 16)) return FGG_ERR_INVALID_VALUE;
    fgg_status st = device_check(&num_cus);
    if (st != FGG_OK) return st;
    if (M == 0 || N == 0) return FGG_OK;
    return finish(fgg::launch_gemm_masked(fp4, tiled, G, M, N, K, (const uint8_t*)a, (const float*)a_scales,
                                          (const uint8_t*)b, b_scales, masked_m, (uint16_t*)d, ldd,
                                          (hipStream_t)stream));
  }
  return FGG_ERR_INVALID_VALUE;
}

fgg_status fgg_grouped_gemm_silu_quantize(int32_t G, int64_t M, int64_t I, int64_t K, const void* a,
                                          const void* a_scales, fgg_qdesc aq, const void* b, const void* b_scales,
                                          fgg_qdesc bq, const int32_t* offsets, const int32_t* counts, void* q_out,
                                          float* s_out, void* stream) {
  if (G < 1 || G > 1024 || M < 0 || I < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  if (I % 128 != 0 || K % 128 != 0 || K > 16384) return FGG_ERR_UNSUPPORTED;
  if (!same_q(aq, FGG_E4M3, FGG_F32, 1, 128) || !same_q(bq, FGG_E4M3, FGG_F32, 128, 128)) return FGG_ERR_UNSUPPORTED;
  if ((K > 0 && (!a || !a_scales || !b || !b_scales)) || !offsets || !q_out || !s_out) return FGG_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(q_out, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4) ||
      !aligned(s_out, 4))
    return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  if (M == 0 || I == 0) return FGG_OK;
  return finish(fgg::launch_gemm_fp8_silu_quantize(G, M, I, K, (const uint8_t*)a, (const float*)a_scales,
                                                   (const uint8_t*)b, (const float*)b_scales, offsets, counts,
                                                   (uint8_t*)q_out, s_out, num_cus, (hipStream_t)stream));
}

fgg_status fgg_scaled_gemm_workspace(int64_t M, int64_t N, int64_t K, fgg_qdesc aq, fgg_qdesc bq,
                                     const fgg_epilogue* epi, size_t* bytes) {
  if (!bytes || M < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  *bytes = 0;
  if (same_q(aq, FGG_E2M1X2, FGG_F32, 1, 16) && same_q(bq, FGG_E2M1X2, FGG_F32, 1, 16))
    *bytes = fgg::w4a4_workspace_bytes(M, N, K, epi ? epi->rank : 0);
  if (same_q(aq, FGG_E2M1X2, FGG_E8M0, 1, 32) && same_q(bq, FGG_E2M1X2, FGG_E8M0, 1, 32))
    *bytes = fgg::mxfp4_workspace_bytes(M, epi ? epi->rank : 0);
  return FGG_OK;
}

fgg_status fgg_scaled_gemm(int64_t M, int64_t N, int64_t K, const void* a, const void* a_scales, fgg_qdesc aq,
                           const void* b, const void* b_scales, fgg_qdesc bq, const fgg_epilogue* epi, void* d,
                           int64_t ldd, void* workspace, size_t ws_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  // (N % 128 for the FP8 and per-16 W4A4 paths, N % 16 for MXFP4: checked per path below)
  if (N % 16 != 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
  if (ldd < N || ldd % 8 != 0) return FGG_ERR_INVALID_VALUE;
  // (with K == 0 the operands hold no bytes and are never read: they may be NULL)
  if ((K > 0 && (!a || !a_scales || !b || !b_scales)) || !d) return FGG_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4))
    return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  if (same_q(aq, FGG_E4M3, FGG_F32, 1, 128) && same_q(bq, FGG_E4M3, FGG_F32, 128, 128)) {
    if (epi || N % 128 != 0) return FGG_ERR_UNSUPPORTED;
    if (K > 16384) return FGG_ERR_UNSUPPORTED;
    fgg_status st = device_check(&num_cus);
    if (st != FGG_OK) return st;
    if (M == 0 || N == 0) return FGG_OK;
    return finish(fgg::launch_gemm_fp8_contig(1, M, N, K, (const uint8_t*)a, (const float*)a_scales,
                                              (const uint8_t*)b, (const float*)b_scales, nullptr, nullptr,
                                              (uint16_t*)d, ldd, num_cus, (hipStream_t)stream));
  }
  if (same_q(aq, FGG_E2M1X2, FGG_F32, 1, 16) && same_q(bq, FGG_E2M1X2, FGG_F32, 1, 16)) {
    // (the GEMM's per-lane DMA offsets are 32-bit: 128 rows x 2K bytes)
    if (M % 128 != 0 || N % 128 != 0 || K == 0 || K > (int64_t(1) << 22)) return FGG_ERR_UNSUPPORTED;
    if (!aligned(a_scales, 8) || !aligned(b_scales, 8)) return FGG_ERR_INVALID_VALUE;
    const int32_t rank = epi ? epi->rank : 0;
    if (rank != 0 && rank != 32) return FGG_ERR_UNSUPPORTED;
    if (rank == 32) {
      if (!epi->x_bf16 || !epi->l_down || !epi->l_up) return FGG_ERR_INVALID_VALUE;
      if (!aligned(epi->x_bf16, 16) || !aligned(epi->l_down, 2) || !aligned(epi->l_up, 2))
        return FGG_ERR_INVALID_VALUE;
    }
    if (M > 0 && N > 0 &&
        (!workspace || ws_bytes < fgg::w4a4_workspace_bytes(M, N, K, rank) || !aligned(workspace, 256)))
      return FGG_ERR_INVALID_VALUE;
    const void* bias = epi ? epi->bias : nullptr;
    if (bias && !aligned(bias, 2)) return FGG_ERR_INVALID_VALUE;
    fgg_status st = device_check(&num_cus);
    if (st != FGG_OK) return st;
    if (M == 0 || N == 0) return FGG_OK;
    return finish(fgg::launch_w4a4(M, N, K, (const uint8_t*)a, (const float*)a_scales, (const uint8_t*)b,
                                   (const float*)b_scales, rank ? (const uint16_t*)epi->x_bf16 : nullptr,
                                   rank ? (const uint16_t*)epi->l_down : nullptr,
                                   rank ? (const uint16_t*)epi->l_up : nullptr, rank, (const uint16_t*)bias,
                                   (uint16_t*)d, ldd, workspace, num_cus, (hipStream_t)stream));
  }
  if (same_q(aq, FGG_E2M1X2, FGG_E8M0, 1, 32) && same_q(bq, FGG_E2M1X2, FGG_E8M0, 1, 32)) {
    // (per-lane DMA offsets are 32-bit: 256 rows x K/2 bytes)
    if (K == 0 || K > (int64_t(1) << 24)) return FGG_ERR_UNSUPPORTED;
    // (scale rows are read as dwords: K/32 bytes per row, a multiple of 4)
    const int32_t rank = epi ? epi->rank : 0;
    if (rank != 0 && rank != 32) return FGG_ERR_UNSUPPORTED;
    if (rank == 32) {
      if (!epi->x_bf16 || !epi->l_down || !epi->l_up) return FGG_ERR_INVALID_VALUE;
      if (!aligned(epi->x_bf16, 16) || !aligned(epi->l_down, 2) || !aligned(epi->l_up, 2))
        return FGG_ERR_INVALID_VALUE;
      if (M > 0 && N > 0 && (!workspace || ws_bytes < fgg::mxfp4_workspace_bytes(M, rank) || !aligned(workspace, 16)))
        return FGG_ERR_INVALID_VALUE;
    }
    const void* bias = epi ? epi->bias : nullptr;
    if (bias && !aligned(bias, 2)) return FGG_ERR_INVALID_VALUE;
    fgg_status st = device_check(&num_cus);
    if (st != FGG_OK) return st;
    if (M == 0 || N == 0) return FGG_OK;
    return finish(fgg::launch_mxfp4(M, N, K, (const uint8_t*)a, (const uint8_t*)a_scales, (const uint8_t*)b,
                                    (const uint8_t*)b_scales, rank ? (const uint16_t*)epi->x_bf16 : nullptr,
                                    rank ? (const uint16_t*)epi->l_down : nullptr,
                                    rank ? (const uint16_t*)epi->l_up : nullptr, rank, (const uint16_t*)bias,
                                    (uint16_t*)d, ldd, workspace, (hipStream_t)stream));
  }
  return FGG_ERR_UNSUPPORTED;
}

fgg_status fgg_pack_fp4_weights_bytes(int32_t G, int64_t N, int64_t K, size_t* b_bytes, size_t* s_bytes) {
  if (G < 0 || N < 0 || K < 0 || !b_bytes || !s_bytes) return FGG_ERR_INVALID_VALUE;
  if (N % 16 != 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
  fgg::fp4_tiled_bytes(G, N, K, b_bytes, s_bytes);
  return FGG_OK;
}

fgg_status fgg_pack_fp4_weights(const void* b, const void* b_scales, int32_t G, int64_t N, int64_t K,
                                void* b_tiled, void* s_tiled, void* stream) {
  if (G < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  if (N % 16 != 0 || K % 128 != 0) return FGG_ERR_UNSUPPORTED;
  const bool empty = G == 0 || N == 0 || K == 0;
  if (!empty && (!b || !b_scales || !b_tiled || !s_tiled)) return FGG_ERR_INVALID_VALUE;
  if (!aligned(b, 16) || !aligned(b_tiled, 16) || !aligned(s_tiled, 16)) return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  if (empty) return FGG_OK;
  return finish(fgg::launch_pack_fp4(G, N, K, (const uint8_t*)b, (const uint8_t*)b_scales, (uint8_t*)b_tiled,
                                     (uint8_t*)s_tiled, num_cus, (hipStream_t)stream));
}

fgg_status fgg_moe_combine(const void* y, int64_t ldy, const int32_t* src_to_row, const float* topk_w, int64_t T,
                           int32_t k, int64_t N, void* out, int64_t ldo, void* stream) {
  if (T < 0 || k < 1 || k > 64 || N < 0) return FGG_ERR_INVALID_VALUE;
  if (N % 8 != 0) return FGG_ERR_UNSUPPORTED;
  if (ldy < N || ldo < N || ldy % 8 != 0 || ldo % 8 != 0) return FGG_ERR_INVALID_VALUE;
  if (T == 0 || N == 0) return FGG_OK;
  if (!y || !src_to_row || !topk_w || !out) return FGG_ERR_INVALID_VALUE;
  if (!aligned(y, 16) || !aligned(out, 16) || !aligned(topk_w, 4)) return FGG_ERR_INVALID_VALUE;
  fgg_status st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_combine((const uint16_t*)y, ldy, src_to_row, topk_w, T, k, N, (uint16_t*)out, ldo,
                                    (hipStream_t)stream));
}

fgg_status fgg_moe_down_combine_workspace(int64_t M, size_t* bytes) {
  if (!bytes || M < 0) return FGG_ERR_INVALID_VALUE;
  *bytes = (size_t)((M + 127) / 128 * 128) * 8;
  return FGG_OK;
}

fgg_status fgg_moe_down_combine(int32_t G, int64_t M, int64_t N, int64_t K, const void* a, const void* a_scales,
                                fgg_qdesc aq, const void* b, const void* b_scales, fgg_qdesc bq,
                                const int32_t* offsets, const int32_t* counts, const int32_t* src_to_row,
                                const int32_t* row_to_src, const float* topk_w, int64_t T, int32_t k, void* y,
                                int64_t ldy, void* workspace, size_t ws_bytes, void* out, int64_t ldo,
                                void* stream) {
  if (G < 1 || G > 1024 || M < 0 || N < 0 || K < 0 || T < 0 || k < 1 || k > 64) return FGG_ERR_INVALID_VALUE;
  if (N % 128 != 0 || K % 128 != 0 || K > 16384) return FGG_ERR_UNSUPPORTED;
  if (!same_q(aq, FGG_E4M3, FGG_F32, 1, 128) || !same_q(bq, FGG_E4M3, FGG_F32, 128, 128)) return FGG_ERR_UNSUPPORTED;
  if (ldy < N || ldy % 8 != 0 || ldo < N || ldo % 8 != 0) return FGG_ERR_INVALID_VALUE;
  if ((K > 0 && (!a || !a_scales || !b || !b_scales)) || !offsets || !counts || !src_to_row || !row_to_src ||
      !topk_w || !y || !out)
    return FGG_ERR_INVALID_VALUE;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(y, 16) || !aligned(out, 16) || !aligned(a_scales, 4) ||
      !aligned(b_scales, 4) || !aligned(topk_w, 4))
    return FGG_ERR_INVALID_VALUE;
  size_t need = 0;
  fgg_moe_down_combine_workspace(M, &need);
  if (M > 0 && (!workspace || !aligned(workspace, 16) || ws_bytes < need)) return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  const hipStream_t hs = (hipStream_t)stream;
  uint8_t* ri = (uint8_t*)workspace;
  hipError_t e = fgg::launch_combine_rows(row_to_src, src_to_row, topk_w, T, k, M, ri, hs);
  if (e == hipSuccess)
    e = fgg::launch_gemm_fp8_combine(G, M, N, K, (const uint8_t*)a, (const float*)a_scales, (const uint8_t*)b,
                                     (const float*)b_scales, offsets, counts, (uint16_t*)y, ldy, ri, (uint16_t*)out,
                                     ldo, num_cus, hs);
  if (e == hipSuccess)
    e = fgg::launch_combine_rest((const uint16_t*)y, ldy, src_to_row, topk_w, T, k, N, (uint16_t*)out, ldo, hs);
  return finish(e);
}

static fgg_status route_check(fgg_dtype dtype, int64_t T, int32_t E, int64_t ld, int32_t k, fgg_gate gate, float scale) {
  if (T < 0 || E < 1 || E > 1024 || k < 1 || k > 64 || k > E || ld < E) return FGG_ERR_INVALID_VALUE;
  if (gate != FGG_GATE_SOFTMAX && gate != FGG_GATE_SIGMOID) return FGG_ERR_INVALID_VALUE;
  if (!(scale - scale == 0.0f)) return FGG_ERR_INVALID_VALUE;   // finite
  if (!float_type(dtype)) return FGG_ERR_UNSUPPORTED;
  // (one group of lanes per token: 256-thread blocks of 4, 8 or 16 tokens, and int32 pairs)
  if (T > (int64_t)fgg::kMaxRowBlocks * 4 || T * (int64_t)k > (int64_t)INT32_MAX) return FGG_ERR_UNSUPPORTED;
  return FGG_OK;
}

fgg_status fgg_moe_route(const void* logits, fgg_dtype dtype, int64_t T, int32_t E, int64_t ld, int32_t k,
                         fgg_gate gate, const float* bias, int32_t renormalize, float scale, int32_t* topk_ids,
                         float* topk_w, void* stream) {
  fgg_status st = route_check(dtype, T, E, ld, k, gate, scale);
  if (st != FGG_OK) return st;
  if (T == 0) return FGG_OK;
  if (!logits || !topk_ids || !topk_w) return FGG_ERR_INVALID_VALUE;
  if (!aligned(logits, float_size(dtype)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(bias, 4))
    return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_route(logits, dtype == FGG_BF16, T, E, ld, k, gate == FGG_GATE_SIGMOID, bias,
                                  renormalize != 0, scale, topk_ids, topk_w, (hipStream_t)stream));
}

fgg_status fgg_moe_route_backward(const void* logits, fgg_dtype dtype, int64_t T, int32_t E, int64_t ld, int32_t k,
                                  fgg_gate gate, int32_t renormalize, float scale, const int32_t* topk_ids,
                                  const float* dtopk_w, void* dlogits, int64_t ldd, void* stream) {
  fgg_status st = route_check(dtype, T, E, ld, k, gate, scale);
  if (st != FGG_OK) return st;
  if (ldd < E) return FGG_ERR_INVALID_VALUE;
  if (T == 0) return FGG_OK;
  if (!logits || !topk_ids || !dtopk_w || !dlogits) return FGG_ERR_INVALID_VALUE;
  if (!aligned(logits, float_size(dtype)) || !aligned(dlogits, float_size(dtype)) || !aligned(topk_ids, 4) ||
      !aligned(dtopk_w, 4))
    return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_route_backward(logits, dtype == FGG_BF16, T, E, ld, k, gate == FGG_GATE_SIGMOID,
                                           renormalize != 0, scale, topk_ids, dtopk_w, dlogits, ldd,
                                           (hipStream_t)stream));
}

// Arguments of the four row calls: tokens [T][ldt], rows [M][ldr], both of `dtype`.
static fgg_status rows_check(fgg_dtype dtype, int64_t T, int32_t k, int64_t N, int64_t M, int64_t ldt, int64_t ldr) {
  if (T < 0 || k < 1 || k > 64 || N < 1 || M < 0 || ldt < N || ldr < N) return FGG_ERR_INVALID_VALUE;
  if (!float_type(dtype)) return FGG_ERR_UNSUPPORTED;
  if (T * (int64_t)k > (int64_t)INT32_MAX || M > (int64_t)INT32_MAX || T > fgg::kMaxRowBlocks ||
      T + M / 16 + 1 > fgg::kMaxRowBlocks || N > (int64_t(1) << 26))
    return FGG_ERR_UNSUPPORTED;
  return FGG_OK;
}

fgg_status fgg_moe_permute_rows(const void* x, fgg_dtype dtype, int64_t T, int32_t k, int64_t N, int64_t ldx,
                                const float* topk_w, const int32_t* src_to_row, const int32_t* row_to_src,
                                const int32_t* offsets, int32_t E, int64_t M, void* rows, int64_t ldr,
                                void* stream) {
  fgg_status st = rows_check(dtype, T, k, N, M, ldx, ldr);
  if (st != FGG_OK) return st;
  if (E < 1 || E > 1024) return FGG_ERR_INVALID_VALUE;
  if (T == 0 || M == 0) return FGG_OK;
  if (!x || !src_to_row || !row_to_src || !offsets || !rows) return FGG_ERR_INVALID_VALUE;
  const size_t el = float_size(dtype);
  if (!aligned(x, el) || !aligned(rows, el) || !aligned(topk_w, 4)) return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_rows_scatter(x, dtype == FGG_BF16, ldx, nullptr, 0, topk_w, src_to_row, row_to_src,
                                         offsets, E, T, k, N, M, rows, ldr, nullptr, (hipStream_t)stream));
}

fgg_status fgg_moe_permute_rows_backward(const void* drows, fgg_dtype dtype, int64_t M, int64_t lddr, const void* x,
                                         int64_t ldx, const float* topk_w, const int32_t* src_to_row, int64_t T,
                                         int32_t k, int64_t N, void* dx, int64_t lddx, float* dtopk_w, void* stream) {
  fgg_status st = rows_check(dtype, T, k, N, M, lddx, lddr);
  if (st != FGG_OK) return st;
  if (dtopk_w && ldx < N) return FGG_ERR_INVALID_VALUE;
  if (T == 0) return FGG_OK;
  if ((M > 0 && !drows) || !src_to_row || !dx || (dtopk_w && !x)) return FGG_ERR_INVALID_VALUE;
  const size_t el = float_size(dtype);
  if (!aligned(drows, el) || !aligned(dx, el) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4) ||
      (dtopk_w && !aligned(x, el)))
    return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_rows_collect(drows, dtype == FGG_BF16, lddr, x, ldx, topk_w, src_to_row, T, k, N, M, dx,
                                         lddx, dtopk_w, (hipStream_t)stream));
}

fgg_status fgg_moe_unpermute_rows(const void* rows, fgg_dtype dtype, int64_t M, int64_t ldr, const float* topk_w,
                                  const int32_t* src_to_row, int64_t T, int32_t k, int64_t N, void* out, int64_t ldo,
                                  void* stream) {
  fgg_status st = rows_check(dtype, T, k, N, M, ldo, ldr);
  if (st != FGG_OK) return st;
  if (T == 0) return FGG_OK;
  if ((M > 0 && !rows) || !src_to_row || !out) return FGG_ERR_INVALID_VALUE;
  const size_t el = float_size(dtype);
  if (!aligned(rows, el) || !aligned(out, el) || !aligned(topk_w, 4)) return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_rows_collect(rows, dtype == FGG_BF16, ldr, nullptr, 0, topk_w, src_to_row, T, k, N, M, out,
                                         ldo, nullptr, (hipStream_t)stream));
}

fgg_status fgg_moe_unpermute_rows_backward(const void* dout, fgg_dtype dtype, int64_t T, int32_t k, int64_t N,
                                           int64_t lddo, const void* rows, int64_t ldr, const float* topk_w,
                                           const int32_t* src_to_row, const int32_t* row_to_src,
                                           const int32_t* offsets, int32_t E, int64_t M, void* drows, int64_t lddr,
                                           float* dtopk_w, void* stream) {
  fgg_status st = rows_check(dtype, T, k, N, M, lddo, lddr);
  if (st != FGG_OK) return st;
  if (E < 1 || E > 1024 || (dtopk_w && ldr < N)) return FGG_ERR_INVALID_VALUE;
  if (T == 0 || (M == 0 && !dtopk_w)) return FGG_OK;
  if (!dout || !src_to_row || !offsets || (M > 0 && (!row_to_src || !drows || (dtopk_w && !rows))))
    return FGG_ERR_INVALID_VALUE;
  const size_t el = float_size(dtype);
  if (!aligned(dout, el) || !aligned(drows, el) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4) ||
      (dtopk_w && !aligned(rows, el)))
    return FGG_ERR_INVALID_VALUE;
  st = device_check(nullptr);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_rows_scatter(dout, dtype == FGG_BF16, lddo, rows, ldr, topk_w, src_to_row, row_to_src,
                                         offsets, E, T, k, N, M, drows, lddr, dtopk_w, (hipStream_t)stream));
}

fgg_status fgg_moe_gemv_fp4(int32_t G, int64_t T, int32_t k, int64_t N, int64_t K, const void* x, fgg_dtype x_dtype,
                            int64_t ldx, int32_t x_per_slot, const void* b, const void* b_scales, fgg_qdesc bq,
                            const int32_t* topk_ids, const float* topk_w, fgg_act act, void* out,
                            fgg_dtype out_dtype, int64_t ldo, void* stream) {
  if (G < 1 || G > 1024 || T < 0 || k < 1 || k > 64 || N < 0 || K < 0 || ldx < K || ldo < N)
    return FGG_ERR_INVALID_VALUE;
  if (act != FGG_ACT_NONE && act != FGG_ACT_SILU_MUL) return FGG_ERR_INVALID_VALUE;
  // one set of weights has one slot per token; a weighted sum needs slots
  if (!topk_ids && T > 0 && (G != 1 || k != 1 || topk_w)) return FGG_ERR_INVALID_VALUE;
  if (!float_type(x_dtype) || !float_type(out_dtype)) return FGG_ERR_UNSUPPORTED;
  if (topk_w && act != FGG_ACT_NONE) return FGG_ERR_UNSUPPORTED;
  const bool tiled = same_q(bq, FGG_E2M1X2_TILED, FGG_E8M0, 1, 32);
  if (!tiled && !same_q(bq, FGG_E2M1X2, FGG_E8M0, 1, 32)) return FGG_ERR_UNSUPPORTED;
  if (K == 0 || K % (tiled ? 128 : 32) != 0 || (tiled && N % 16 != 0)) return FGG_ERR_UNSUPPORTED;
  // (grid limits: 16 rows and 16 tokens per workgroup)
  if (N > (int64_t(1) << 26) || K > (int64_t(1) << 26) || T > 16 * (int64_t)65535) return FGG_ERR_UNSUPPORTED;
  if (T == 0 || N == 0) return FGG_OK;
  if (!x || !b || !b_scales || !out) return FGG_ERR_INVALID_VALUE;
  if (!aligned(x, float_size(x_dtype)) || !aligned(out, float_size(out_dtype)) || !aligned(b, 16) ||
      (tiled && !aligned(b_scales, 16)) || !aligned(topk_ids, 4) || !aligned(topk_w, 4))
    return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  fgg_status st = device_check(&num_cus);
  if (st != FGG_OK) return st;
  return finish(fgg::launch_gemv_fp4(tiled, G, T, k, N, K, x, x_dtype == FGG_BF16, ldx, x_per_slot != 0,
                                     (const uint8_t*)b, (const uint8_t*)b_scales, topk_ids, topk_w,
                                     act == FGG_ACT_SILU_MUL, out, out_dtype == FGG_BF16, ldo, num_cus,
                                     (hipStream_t)stream));
}

// Shapes of the bf16 products: segments of M rows, weights [G][N][K].
static fgg_status segments_check(int32_t G, int64_t M, int64_t N, int64_t K, const int32_t* offsets,
                                 const int32_t* counts) {
  if (G < 1 || G > 1024 || M < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  if ((!offsets && (G != 1 || counts)) || !aligned(offsets, 4) || !aligned(counts, 4)) return FGG_ERR_INVALID_VALUE;
  // (16-byte pieces of a row, and 32-bit offsets of 256 rows)
  if (N == 0 || K == 0 || N % 8 != 0 || K % 8 != 0 || N > fgg::kMaxBf16Width || K > fgg::kMaxBf16Width ||
      M > (int64_t)INT32_MAX)
    return FGG_ERR_UNSUPPORTED;
  return FGG_OK;
}

// A matrix of `cols` columns and rows of 16-byte pieces; NULL only where `needed` is false.
static fgg_status rows_operand(const void* p, int64_t ld, int64_t cols, int64_t el, bool needed) {
  if (needed && !p) return FGG_ERR_INVALID_VALUE;
  if (ld < cols || (ld * el) % 16 != 0 || !aligned(p, 16)) return FGG_ERR_INVALID_VALUE;
  return ld > fgg::kMaxBf16Width ? FGG_ERR_UNSUPPORTED : FGG_OK;
}

#define FGG_TRY(call)                     \
  do {                                    \
    const fgg_status s_ = (call);         \
    if (s_ != FGG_OK) return s_;          \
  } while (0)

fgg_status fgg_grouped_linear(int32_t G, int64_t M, int64_t N, int64_t K, const void* x, int64_t ldx, const void* w,
                              const int32_t* offsets, const int32_t* counts, void* y, fgg_dtype y_dtype, int64_t ldy,
                              void* stream) {
  FGG_TRY(segments_check(G, M, N, K, offsets, counts));
  if (!float_type(y_dtype)) return FGG_ERR_UNSUPPORTED;
  FGG_TRY(rows_operand(x, ldx, K, 2, M > 0));
  FGG_TRY(rows_operand(w, K, K, 2, M > 0));
  FGG_TRY(rows_operand(y, ldy, N, (int64_t)float_size(y_dtype), M > 0));
  if (fgg::gemm_bf16_tiles(offsets, G, M, N, false) > fgg::kMaxBf16Tiles) return FGG_ERR_UNSUPPORTED;
  if (M == 0) return FGG_OK;
  int num_cus = 0;
  FGG_TRY(device_check(&num_cus));
  return finish(fgg::launch_grouped_linear({offsets, counts, G, M, num_cus}, N, K, (const uint16_t*)x, ldx, (const uint16_t*)w,
                                           y, y_dtype == FGG_F32, ldy, (hipStream_t)stream));
}

fgg_status fgg_grouped_linear_backward_input(int32_t G, int64_t M, int64_t N, int64_t K, const void* dy, int64_t lddy,
                                             const void* w, const int32_t* offsets, const int32_t* counts, void* dx,
                                             fgg_dtype dx_dtype, int64_t lddx, void* stream) {
  FGG_TRY(segments_check(G, M, N, K, offsets, counts));
  if (!float_type(dx_dtype)) return FGG_ERR_UNSUPPORTED;
  FGG_TRY(rows_operand(dy, lddy, N, 2, M > 0));
  FGG_TRY(rows_operand(w, K, K, 2, M > 0));
  FGG_TRY(rows_operand(dx, lddx, K, (int64_t)float_size(dx_dtype), M > 0));
  if (fgg::gemm_bf16_tiles(offsets, G, M, K, false) > fgg::kMaxBf16Tiles) return FGG_ERR_UNSUPPORTED;
  if (M == 0) return FGG_OK;
  int num_cus = 0;
  FGG_TRY(device_check(&num_cus));
  return finish(fgg::launch_grouped_dx({offsets, counts, G, M, num_cus}, N, K, (const uint16_t*)dy, lddy, (const uint16_t*)w, dx,
                                       dx_dtype == FGG_F32, lddx, (hipStream_t)stream));
}

fgg_status fgg_grouped_linear_backward_weight_workspace(int32_t G, int64_t M, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes || G < 1 || G > 1024 || M < 0 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  if (N > fgg::kMaxBf16Width || K > fgg::kMaxBf16Width || M > (int64_t)INT32_MAX) return FGG_ERR_UNSUPPORTED;
  *bytes = fgg::gemm_bf16_dw_workspace(G, M, N, K);
  return FGG_OK;
}

fgg_status fgg_grouped_linear_backward_weight(int32_t G, int64_t M, int64_t N, int64_t K, const void* dy, int64_t lddy,
                                              const void* x, int64_t ldx, const int32_t* offsets,
                                              const int32_t* counts, void* dw, fgg_dtype dw_dtype,
                                              int32_t accumulate, void* workspace, size_t ws_bytes, void* stream) {
  FGG_TRY(segments_check(G, M, N, K, offsets, counts));
  if (!float_type(dw_dtype)) return FGG_ERR_UNSUPPORTED;
  FGG_TRY(rows_operand(dy, lddy, N, 2, M > 0));
  FGG_TRY(rows_operand(x, ldx, K, 2, M > 0));
  FGG_TRY(rows_operand(dw, K, K, (int64_t)float_size(dw_dtype), true));
  if (fgg::gemm_bf16_dw_tiles(G, N, K) > fgg::kMaxBf16Tiles) return FGG_ERR_UNSUPPORTED;
  const size_t need = fgg::gemm_bf16_dw_workspace(G, M, N, K);
  if (need > 0 && (!workspace || ws_bytes < need || !aligned(workspace, 16))) return FGG_ERR_INVALID_VALUE;
  int num_cus = 0;
  FGG_TRY(device_check(&num_cus));
  return finish(fgg::launch_grouped_dw({offsets, counts, G, M, num_cus}, N, K, (const uint16_t*)dy, lddy, (const uint16_t*)x,
                                       ldx, dw, dw_dtype == FGG_F32, accumulate != 0, (float*)workspace,
                                       (hipStream_t)stream));
}

fgg_status fgg_grouped_gated(int32_t G, int64_t M, int64_t I, int64_t K, const void* x, int64_t ldx, const void* w,
                             const int32_t* offsets, const int32_t* counts, void* a, int64_t lda, void* h,
                             int64_t ldh, void* stream) {
  FGG_TRY(segments_check(G, M, I, K, offsets, counts));
  FGG_TRY(rows_operand(x, ldx, K, 2, M > 0));
  FGG_TRY(rows_operand(w, K, K, 2, M > 0));
  FGG_TRY(rows_operand(a, lda, I, 2, M > 0));
  if (h) FGG_TRY(rows_operand(h, ldh, 2 * I, 2, true));
  if (fgg::gemm_bf16_tiles(offsets, G, M, I, true) > fgg::kMaxBf16Tiles) return FGG_ERR_UNSUPPORTED;
  if (M == 0) return FGG_OK;
  int num_cus = 0;
  FGG_TRY(device_check(&num_cus));
  return finish(fgg::launch_grouped_gated({offsets, counts, G, M, num_cus}, I, K, (const uint16_t*)x, ldx, (const uint16_t*)w,
                                          (uint16_t*)a, lda, (uint16_t*)h, ldh, (hipStream_t)stream));
}

fgg_status fgg_grouped_gated_backward(int32_t G, int64_t M, int64_t I, int64_t N, const void* dy, int64_t lddy,
                                      const void* w_down, const void* h, int64_t ldh, const int32_t* offsets,
                                      const int32_t* counts, void* dh, int64_t lddh, void* a, int64_t lda,
                                      void* stream) {
  FGG_TRY(segments_check(G, M, I, N, offsets, counts));
  FGG_TRY(rows_operand(dy, lddy, N, 2, M > 0));
  FGG_TRY(rows_operand(w_down, I, I, 2, M > 0));
  FGG_TRY(rows_operand(h, ldh, 2 * I, 2, M > 0));
  FGG_TRY(rows_operand(dh, lddh, 2 * I, 2, M > 0));
  if (a) FGG_TRY(rows_operand(a, lda, I, 2, true));
  if (fgg::gemm_bf16_tiles(offsets, G, M, I, false) > fgg::kMaxBf16Tiles) return FGG_ERR_UNSUPPORTED;
  if (M == 0) return FGG_OK;
  int num_cus = 0;
  FGG_TRY(device_check(&num_cus));
  return finish(fgg::launch_grouped_gated_backward({offsets, counts, G, M, num_cus}, I, N, (const uint16_t*)dy, lddy,
                                                   (const uint16_t*)w_down, (const uint16_t*)h, ldh, (uint16_t*)dh,
                                                   lddh, (uint16_t*)a, lda, (hipStream_t)stream));
}

static fgg_status lora_check(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K) {
  if (T < 0 || L < 1 || r < 1 || N < 0 || K < 0) return FGG_ERR_INVALID_VALUE;
  // (16-byte pieces of a row; 32-bit counts of items, and grids of 16 tokens by 32 columns)
  if (N == 0 || K == 0 || N % 8 != 0 || K % 8 != 0 || r % 8 != 0 || r > 128 || N > (int64_t(1) << 20) ||
      K > (int64_t(1) << 20) || T > (int64_t(1) << 26))
    return FGG_ERR_UNSUPPORTED;
  return FGG_OK;
}

fgg_status fgg_lora_workspace(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K, size_t* bytes) {
  if (!bytes) return FGG_ERR_INVALID_VALUE;
  FGG_TRY(lora_check(T, L, r, N, K));
  *bytes = fgg::lora_workspace_bytes(T, L, r, N, K);
  return FGG_OK;
}

fgg_status fgg_lora_add(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K, const void* x, int64_t ldx,
                        const int32_t* ids, const void* a, const void* b, const float* scales, const void* base,
                        int64_t ldb, void* out, fgg_dtype dtype, int64_t ldo, void* workspace, size_t ws_bytes,
                        void* stream) {
  FGG_TRY(lora_check(T, L, r, N, K));
  if (!float_type(dtype)) return FGG_ERR_UNSUPPORTED;
  const int64_t el = (int64_t)float_size(dtype);
  if (ldx > fgg::kMaxBf16Width) return FGG_ERR_UNSUPPORTED;   // (32-bit offsets of 64 rows)
  if (ldx < K || ldx % 8 != 0 || ldb < N || ldo < N || ldb * el % 16 != 0 || ldo * el % 16 != 0)
    return FGG_ERR_INVALID_VALUE;
  if (T == 0) return FGG_OK;
  if (base == out && ldb != ldo) return FGG_ERR_INVALID_VALUE;
  const size_t need = fgg::lora_workspace_bytes(T, L, r, N, K);
  if (!x || !ids || !a || !b || !base || !out || (need > 0 && !workspace)) return FGG_ERR_INVALID_VALUE;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 16) || !aligned(out, 16) ||
      !aligned(ids, 4) || !aligned(scales, 4) || !aligned(workspace, 16) || ws_bytes < need)
    return FGG_ERR_INVALID_VALUE;
  FGG_TRY(device_check(nullptr));
  return finish(fgg::launch_lora(T, L, r, N, K, (const uint16_t*)x, ldx, ids, (const uint16_t*)a, (const uint16_t*)b,
                                 scales, base, ldb, out, dtype == FGG_F32, ldo, (float*)workspace,
                                 (hipStream_t)stream));
}

int32_t fgg_kernel_count(void) {
  const fgg::KernelInfo* const* t = nullptr;
  return (int32_t)fgg::kernel_table(&t);
}

fgg_status fgg_kernel_info_get(int32_t i, fgg_kernel_info* info) {
  const fgg::KernelInfo* const* t = nullptr;
  const int n = fgg::kernel_table(&t);
  if (i < 0 || i >= n || !info) return FGG_ERR_INVALID_VALUE;
  const fgg::KernelInfo& k = *t[i];
  info->kernel = k.name;
  info->entry = k.entry;
  info->tile_m = k.tile_m;
  info->tile_n = k.tile_n;
  info->tile_k = k.tile_k;
  info->threads = k.threads;
  info->stages = k.stages;
  info->stage_bytes = k.stage_bytes;
  info->other_bytes = k.other_bytes;
  info->lds_bytes = k.lds_bytes;
  return FGG_OK;
}

fgg_status fgg_kernel_compiled_lds(int32_t i, int64_t* bytes) {
  const fgg::KernelInfo* const* t = nullptr;
  const int n = fgg::kernel_table(&t);
  if (i < 0 || i >= n || !bytes) return FGG_ERR_INVALID_VALUE;
  fgg_status st = device_check(nullptr);
  if (st != FGG_OK) return st;
  hipFuncAttributes attr;
  const hipError_t e = hipFuncGetAttributes(&attr, t[i]->fn);
  if (e != hipSuccess) return hip_fail(e);
  *bytes = (int64_t)attr.sharedSizeBytes;
  return FGG_OK;
}

}  // extern "C"
#pragma GCC visibility pop
