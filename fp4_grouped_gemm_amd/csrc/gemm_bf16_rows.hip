// bf16 products of few rows per segment with the segment's weights (gfx950): the form of the
// linear layer and of the gated block for single tokens and small batches.
//
//   linear  y[r][n] = sum_k x[r][k] W_g[n][k];   gated  h with W_g = [gate | up], a = silu(h_gate) h_up
//
// What bounds it is reading the weights once, by enough waves (one row, 7168 -> 4096: 11.9 us for 59 MB, 4.9
// TB/s; the smallest tiles of gemm_bf16.hip, 64 of them, take 30).  A workgroup takes 16 weight rows of one
// segment (gated: 8 gate and the 8 up rows of the same index) against 64 of the segment's rows: eight
// waves share the sum over k in pieces of 64 (a whole 128-byte line of each weight row per piece), weights go
// from memory straight into the operands of v_mfma_f32_16x16x32_bf16 (first operand: weight rows, second: 16
// rows of x, which come from the caches), with several pieces' loads in flight per wave.  The waves' sums
// meet in LDS, in their order, and the epilogue writes from there.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_segments.hpp"

namespace fgg {

namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kPiece = 64;
constexpr int kPass = 64;                // rows that a workgroup takes at a time

}  // namespace

template <bool GATED>
__global__ void __launch_bounds__(kThreads, 4)
rows_bf16_kernel(const uint16_t* __restrict__ x, int64_t ldx, const uint16_t* __restrict__ w,
                 const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts, int64_t M, int64_t N,
                 int64_t K, void* __restrict__ out, int64_t ldo, int out_f32, uint16_t* __restrict__ h, int64_t ldh) {
  __shared__ float red[kWaves][16][16 + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int g = blockIdx.y;
  const Segment seg = offsets ? segment_of(offsets, counts, g, M) : Segment{0, (int)M};
  const int first = kPass * blockIdx.z;
  if (first >= seg.rows) return;

  // columns of the output per workgroup, and each lane's weight row (one inside the matrix
  // for columns past the edge: their sums are dropped)
  constexpr int kCols = GATED ? 8 : 16;
  const int64_t n0 = (int64_t)blockIdx.x * kCols;
  int64_t n_lane = n0 + l16 % kCols;
  if (n_lane >= N) n_lane = N - 1;
  if (l16 >= kCols) n_lane += N;
  const uint16_t* wl = w + ((int64_t)g * (GATED ? 2 * N : N) + n_lane) * K + 16 * q;
  const int pieces = (int)(K / kPiece), rest = (int)(K % kPiece);

  auto body = [&](auto ct_tag, int r0) {
    constexpr int CT = decltype(ct_tag)::value;
    constexpr int U = CT == 4 ? 1 : CT == 2 ? 2 : 4;   // pieces whose loads fly together (what the registers hold)
    const uint16_t* xl[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      int r = r0 + 16 * c + l16;
      if (r >= seg.rows) r = seg.rows - 1;       // (its column is dropped)
      xl[c] = x + (seg.first + r) * ldx + 16 * q;
    }
    v4f acc[CT];
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[c] = v4f{0.f, 0.f, 0.f, 0.f};
    auto take = [&](auto u_tag, int p) {
      constexpr int UU = decltype(u_tag)::value;
      v8bf wf[UU][2], xf[UU][CT][2];
#pragma unroll
      for (int u = 0; u < UU; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s)
          wf[u][s] = *reinterpret_cast<const v8bf*>(wl + (int64_t)(p + u * kWaves) * kPiece + 8 * s);
#pragma unroll
      for (int u = 0; u < UU; ++u)
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
          for (int s = 0; s < 2; ++s)
            xf[u][c][s] = *reinterpret_cast<const v8bf*>(xl[c] + (int64_t)(p + u * kWaves) * kPiece + 8 * s);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < UU; ++u)
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
          for (int c = 0; c < CT; ++c)
            acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[u][s], xf[u][c][s], acc[c], 0, 0, 0);
    };
    int p = wave;
    for (; p + (U - 1) * kWaves < pieces; p += U * kWaves) take(std::integral_constant<int, U>{}, p);
    for (; p < pieces; p += kWaves) take(std::integral_constant<int, 1>{}, p);
    if (rest && p == pieces) {                   // the end of the sum, by the wave whose turn it is: zeros past it
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const bool on = 16 * q + 8 * s < rest;
        const v8bf zero = __builtin_bit_cast(v8bf, make_uint4(0, 0, 0, 0));
        v8bf wf = zero, xf[CT];
        if (on) wf = *reinterpret_cast<const v8bf*>(wl + (int64_t)p * kPiece + 8 * s);
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          xf[c] = zero;
          if (on) xf[c] = *reinterpret_cast<const v8bf*>(xl[c] + (int64_t)p * kPiece + 8 * s);
        }
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf, xf[c], acc[c], 0, 0, 0);
      }
    }

#pragma unroll
    for (int c = 0; c < CT; ++c) {
      if (r0 + 16 * c >= seg.rows) break;
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][4 * q + e][l16] = acc[c][e];
      __syncthreads();
      if (threadIdx.x < kCols * 16) {
        const int n = threadIdx.x % kCols, r = r0 + 16 * c + threadIdx.x / kCols, col = threadIdx.x / kCols;
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int v = 0; v < kWaves; ++v) {
          a += red[v][n][col];
          if constexpr (GATED) b += red[v][kCols + n][col];
        }
        if (r < seg.rows && n0 + n < N) {
          const int64_t row = seg.first + r;
          if constexpr (GATED) {
            if (h) {
              h[row * ldh + n0 + n] = (uint16_t)bf16x2_rne(a, 0.0f);
              h[row * ldh + N + n0 + n] = (uint16_t)bf16x2_rne(b, 0.0f);
            }
            a = a * sigmoid(a) * b;
          }
          if (out_f32) ((float*)out)[row * ldo + n0 + n] = a;
          else ((uint16_t*)out)[row * ldo + n0 + n] = (uint16_t)bf16x2_rne(a, 0.0f);
        }
      }
      __syncthreads();
    }
  };

  const int here = seg.rows - first;
  if (here <= 16) body(std::integral_constant<int, 1>{}, first);
  else if (here <= 32) body(std::integral_constant<int, 2>{}, first);
  else body(std::integral_constant<int, kPass / 16>{}, first);
}

#define FGG_ROWS_INFO(gated, name, entry) \
  {"rows_bf16_kernel<" name ">", entry, 64, gated ? 8 : 16, kPiece, kThreads, 0, 0, kWaves * 16 * 17 * 4, \
   kWaves * 16 * 17 * 4, (const void*)rows_bf16_kernel<gated>}
const KernelInfo kInfoRowsBf16[2] = {FGG_ROWS_INFO(false, "linear", "fgg_grouped_linear"),
                                     FGG_ROWS_INFO(true, "gated", "fgg_grouped_gated")};
#undef FGG_ROWS_INFO

hipError_t launch_rows_bf16(const Segments& s, bool gated, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                            const uint16_t* w, void* out, bool out_f32, int64_t ldo, uint16_t* h, int64_t ldh,
                            hipStream_t st) {
  const int cols = gated ? 8 : 16;
  // (a segment may have all the rows: a workgroup for each pass, which ends at once where the segment has fewer)
  const dim3 grid((unsigned)((N + cols - 1) / cols), (unsigned)s.G, (unsigned)((s.M + kPass - 1) / kPass));
  trace_launch(kInfoRowsBf16[gated ? 1 : 0], grid, "G=%d M=%lld columns=%lld sum=%lld%s", s.G, (long long)s.M,
               (long long)N, (long long)K, s.counts ? " counts" : "");
  auto go = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, x, ldx, w, s.offsets, s.counts, s.M, N, K, out, ldo,
                       (int)out_f32, h, ldh);
  };
  gated ? go(rows_bf16_kernel<true>) : go(rows_bf16_kernel<false>);
  return hipGetLastError();
}

}  // namespace fgg
