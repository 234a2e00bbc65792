// Rows of the permuted order and back, in the activations' own type, with the gate
// weights applied on either way, and the gradients.  Pair p = t * k + j of token t has row
// src_to_row[p] (-1: none).  Four operators on two data movements:
//
//   scatter  rows[src_to_row[p]] = w[p] * tok[t]          permute_rows, gradient of unpermute_rows
//   collect  tok[t] = sum_j w[p] * rows[src_to_row[p]]    unpermute_rows, gradient of permute_rows
//
// and in both gradients, where the weights are learned,  dw[p] = <tok[t], rows[src_to_row[p]]>,
// in the same pass over the rows.  Products and sums run in fp32 and are rounded once; the
// sum over a token's slots runs in increasing j, a dot product as per-thread partial sums
// joined by a fixed tree, so every result is the same from run to run (no atomics).
//
// All of it is bound by memory: a token row is read (or written) once however many slots
// it has, a permuted row once.  Measured (a 4 GiB copy on the same card: 4.5 TB/s): permute of
// 8192 x 7168 bf16 onto 32 of 256 experts, 224 MB in 49 us (4.6 TB/s); gradient of a permute,
// 4096 x 2 x 4096 fp32, 201 MB in 34 us (5.9); gradients of an unpermute with its weights',
// 8192 x 4 x 4096 bf16, 621 MB in 121 us (5.1).  The permuted rows are stored through the caches:
// past them the first took 38 us, but with the reader that follows (a copy of the rows) 36 us instead
// of 31 for 68 MB, 128 instead of 129 for 206 MB and 657 instead of 625 for 1 GB.  Rows are moved 16 bytes per lane; the loads and stores are
// declared with the element's alignment (this part's vector memory takes any), so odd
// widths and strides run the same path, and only a width that is not a whole number of 16
// bytes has a scalar tail.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_wave.hpp"

namespace fgg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

template <class T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  using Packed = u32x4_a2;
  static __device__ float get(const u32x4& v, int i) {
    const uint32_t w = v[i >> 1];
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  static __device__ u32x4 pack(const float* f) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = bf16x2_rne(f[2 * i], f[2 * i + 1]);
    return o;
  }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  using Packed = u32x4_a4;
  static __device__ float get(const u32x4& v, int i) { return __uint_as_float(v[i]); }
  static __device__ u32x4 pack(const float* f) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(f[i]);
    return o;
  }
};

// Elements [col, col + kVec) of a row of N; those at or past N are zero.  col < N.
// ONCE: nothing else reads them (no place in the caches is asked for).
template <class T, bool ONCE = false>
__device__ inline u32x4 load_vec(const T* row, int64_t col, int64_t N) {
  constexpr int V = Elem<T>::kVec;
  if (col + V <= N) {
    const auto* p = reinterpret_cast<const typename Elem<T>::Packed*>(row + col);
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    else return *p;
  }
  union {
    u32x4 v;
    T e[V];
  } u;
  u.v = u32x4{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (col + i < N) u.e[i] = row[col + i];
  return u.v;
}

template <class T>
__device__ inline void store_vec(T* row, int64_t col, int64_t N, u32x4 v) {
  constexpr int V = Elem<T>::kVec;
  if (col + V <= N) {
    *reinterpret_cast<typename Elem<T>::Packed*>(row + col) = v;
    return;
  }
  union {
    u32x4 v;
    T e[V];
  } u;
  u.v = v;
#pragma unroll
  for (int i = 0; i < V - 1; ++i)
    if (col + i < N) row[col + i] = u.e[i];
}

constexpr int kPadRows = 16;    // rows of the permuted order that one padding block looks at, four per wave

// Zeros in the padding rows among [r0, r0 + kPadRows), columns from `col` on in steps of `step`.
template <class T>
__device__ inline void clear_padding(const int32_t* row_to_src, int64_t total, int64_t r0, int64_t N, T* rows,
                                     int64_t ldr, int64_t col0, int64_t col_end) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = 0; i < kPadRows / 4; ++i) {
    const int64_t r = r0 + wave * (kPadRows / 4) + i;
    if (r >= total || row_to_src[r] >= 0) continue;
    for (int64_t c = col0 + (int64_t)lane * Elem<T>::kVec; c < col_end; c += 64 * Elem<T>::kVec)
      store_vec<T>(rows + r * ldr, c, N, u32x4{0, 0, 0, 0});
  }
}

}  // namespace

namespace {

// The rows of token t, slot j in lane j (k <= 64), and which slots have one: every wave on its
// own, so that all of a token's rows are known before the first is touched.
__device__ inline uint64_t token_rows(const int32_t* src_to_row, int64_t t, int k, int64_t M, int& row) {
  const int lane = threadIdx.x & 63;
  row = lane < k ? src_to_row[t * k + lane] : -1;
  return __ballot(row >= 0 && row < M);
}
__device__ inline int lane_int(int v, int lane) { return __builtin_amdgcn_readlane(v, lane); }
__device__ inline float lane_float(float v, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), lane));
}
// The lowest slot of the mask, taken out of it.
__device__ inline int next_slot(uint64_t& m) {
  const int j = __ffsll((unsigned long long)m) - 1;
  m &= m - 1;
  return j;
}

}  // namespace

// Scatter: block (t, y) takes columns [y * C * 256 vectors) of token t, one pass, and writes them
// to each of the token's rows (a token without a row is not read); the blocks behind the last
// token clear padding rows.
template <class T, bool W, int C>
__global__ void __launch_bounds__(256) rows_scatter_kernel(const T* __restrict__ tok, int64_t ldt,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ src_to_row,
                                                           const int32_t* __restrict__ row_to_src,
                                                           const int32_t* __restrict__ offsets, int E, int64_t tokens,
                                                           int k, int64_t N, int64_t M, T* __restrict__ rows,
                                                           int64_t ldr) {
  constexpr int V = Elem<T>::kVec;
  const int64_t span = (int64_t)C * 256 * V, col0 = blockIdx.y * span;
  if ((int64_t)blockIdx.x >= tokens) {
    int64_t total = offsets[E];
    if (total > M) total = M;
    clear_padding<T>(row_to_src, total, ((int64_t)blockIdx.x - tokens) * kPadRows, N, rows, ldr, col0,
                     col0 + span < N ? col0 + span : N);
    return;
  }
  const int64_t t = blockIdx.x;
  int row;
  uint64_t live = token_rows(src_to_row, t, k, M, row);
  if (live == 0) return;
  float wt = 1.0f;
  if constexpr (W) wt = (int)(threadIdx.x & 63) < k ? w[t * k + (threadIdx.x & 63)] : 0.0f;
  u32x4 x[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
    if (col < N) x[c] = load_vec<T>(tok + t * ldt, col, N);
  }
  while (live) {
    const int j = next_slot(live);
    T* out = rows + (int64_t)lane_int(row, j) * ldr;
    const float wj = lane_float(wt, j);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
      if (col >= N) continue;
      if constexpr (W) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = wj * Elem<T>::get(x[c], i);
        store_vec<T>(out, col, N, Elem<T>::pack(f));
      } else {
        store_vec<T>(out, col, N, x[c]);
      }
    }
  }
}

// Collect: block (t, y) sums the token's rows over columns [y * C * 256 vectors), B rows' loads at
// a time, added in slot order.
template <class T, bool W, int C, int B>
__device__ inline void collect_rows(const T* rows, int64_t ldr, int64_t col0, int64_t N, int row, float wt,
                                    uint64_t& live, float (&acc)[C][Elem<T>::kVec]) {
  constexpr int V = Elem<T>::kVec;
  u32x4 y[B][C];
  float wj[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const int j = next_slot(live);
    const T* in = rows + (int64_t)lane_int(row, j) * ldr;
    wj[b] = lane_float(wt, j);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
      if (col < N) y[b][c] = load_vec<T>(in, col, N);
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[c][i] = fmaf(wj[b], Elem<T>::get(y[b][c], i), acc[c][i]);
}

template <class T, bool W, int C>
__global__ void __launch_bounds__(256) rows_collect_kernel(const T* __restrict__ rows, int64_t ldr,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ src_to_row, int k, int64_t N,
                                                           int64_t M, T* __restrict__ tok, int64_t ldt) {
  constexpr int V = Elem<T>::kVec;
  const int64_t t = blockIdx.x, col0 = (int64_t)blockIdx.y * C * 256 * V;
  int row;
  uint64_t live = token_rows(src_to_row, t, k, M, row);
  float wt = 1.0f;
  if constexpr (W) wt = (int)(threadIdx.x & 63) < k ? w[t * k + (threadIdx.x & 63)] : 0.0f;
  float acc[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[c][i] = 0.0f;
  while (__popcll(live) >= 4) collect_rows<T, W, C, 4>(rows, ldr, col0, N, row, wt, live, acc);
  if (__popcll(live) >= 2) collect_rows<T, W, C, 2>(rows, ldr, col0, N, row, wt, live, acc);
  if (live) collect_rows<T, W, C, 1>(rows, ldr, col0, N, row, wt, live, acc);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
    if (col < N) store_vec<T>(tok + t * ldt, col, N, Elem<T>::pack(acc[c]));
  }
}

// The gradients with dw: one block per token over the whole row, since dw[p] is a sum over it.
// SCATTER: tok (the gradient of the output) goes to the rows' gradients `out`, dotted with the
// forward's rows.  Otherwise the rows (gradients) are summed into the token's gradient `out`,
// each dotted with the forward's token.  Partial dots: per thread, then per wave, then the four
// waves of LDS in order.
template <class T, bool SCATTER, int C, int B>
__device__ inline void dot_rows(const T* rows, int64_t ldr, T* out, int64_t ldo, int64_t col0, int64_t N, int row,
                                float wt, const u32x4 (&x)[C], uint64_t& live, float (&acc)[C][Elem<T>::kVec],
                                float* part) {
  constexpr int V = Elem<T>::kVec;
  u32x4 y[B][C];
  int slot[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    slot[b] = next_slot(live);
    const T* in = rows + (int64_t)lane_int(row, slot[b]) * ldr;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
      y[b][c] = u32x4{0, 0, 0, 0};
      if (col < N) y[b][c] = load_vec<T, true>(in, col, N);
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const float wj = lane_float(wt, slot[b]);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dot = fmaf(Elem<T>::get(x[c], i), Elem<T>::get(y[b][c], i), dot);
        if constexpr (!SCATTER) acc[c][i] = fmaf(wj, Elem<T>::get(y[b][c], i), acc[c][i]);
      }
      if constexpr (SCATTER) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = wj * Elem<T>::get(x[c], i);
        if (col < N) store_vec<T>(out + (int64_t)lane_int(row, slot[b]) * ldo, col, N, Elem<T>::pack(f));
      }
    }
    dot = group_reduce<64>(dot, OpAdd());
    if ((threadIdx.x & 63) == 0) part[slot[b]] += dot;
  }
}

template <class T, bool W, bool SCATTER, int C>
__global__ void __launch_bounds__(256) rows_dot_kernel(const T* __restrict__ tok, int64_t ldt,
                                                       const T* __restrict__ rows, int64_t ldr,
                                                       const float* __restrict__ w,
                                                       const int32_t* __restrict__ src_to_row,
                                                       const int32_t* __restrict__ row_to_src,
                                                       const int32_t* __restrict__ offsets, int E, int64_t tokens,
                                                       int k, int64_t N, int64_t M, T* __restrict__ out, int64_t ldo,
                                                       float* __restrict__ dw) {
  constexpr int V = Elem<T>::kVec;
  __shared__ float part[4][64];
  if (SCATTER && (int64_t)blockIdx.x >= tokens) {
    int64_t total = offsets[E];
    if (total > M) total = M;
    clear_padding<T>(row_to_src, total, ((int64_t)blockIdx.x - tokens) * kPadRows, N, out, ldo, 0, N);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = blockIdx.x;
  int row;
  const uint64_t slots = token_rows(src_to_row, t, k, M, row);
  float wt = 1.0f;
  if constexpr (W) wt = lane < k ? w[t * k + lane] : 0.0f;
  part[wave][lane] = 0.0f;                            // (each wave its own row)
  wave_sync();
  for (int64_t col0 = 0; col0 < N; col0 += (int64_t)C * 256 * V) {
    if (SCATTER && slots == 0) break;
    u32x4 x[C];
    float acc[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
      x[c] = u32x4{0, 0, 0, 0};
      if (col < N && slots != 0) x[c] = load_vec<T>(tok + t * ldt, col, N);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[c][i] = 0.0f;
    }
    uint64_t live = slots;
    while (__popcll(live) >= 4) dot_rows<T, SCATTER, C, 4>(rows, ldr, out, ldo, col0, N, row, wt, x, live, acc, part[wave]);
    if (__popcll(live) >= 2) dot_rows<T, SCATTER, C, 2>(rows, ldr, out, ldo, col0, N, row, wt, x, live, acc, part[wave]);
    if (live) dot_rows<T, SCATTER, C, 1>(rows, ldr, out, ldo, col0, N, row, wt, x, live, acc, part[wave]);
    if constexpr (!SCATTER) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t col = col0 + ((int64_t)c * 256 + threadIdx.x) * V;
        if (col < N) store_vec<T>(out + t * ldo, col, N, Elem<T>::pack(acc[c]));
      }
    }
  }
  __syncthreads();
  if ((int)threadIdx.x < k) {
    const int j = threadIdx.x;
    dw[t * k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
  }
}

const KernelInfo kInfoRowsScatter = {"rows_scatter_kernel", "fgg_moe_permute_rows, fgg_moe_unpermute_rows_backward", 1,
                                     0, 0, 256, 0, 0, 0, 0, (const void*)rows_scatter_kernel<uint16_t, false, 2>};
const KernelInfo kInfoRowsCollect = {"rows_collect_kernel", "fgg_moe_unpermute_rows, fgg_moe_permute_rows_backward", 1,
                                     0, 0, 256, 0, 0, 0, 0, (const void*)rows_collect_kernel<uint16_t, true, 2>};
const KernelInfo kInfoRowsScatterDot = {"rows_dot_kernel<scatter>", "fgg_moe_unpermute_rows_backward", 1, 0, 0, 256, 0,
                                        0, 1024, 1024, (const void*)rows_dot_kernel<uint16_t, true, true, 2>};
const KernelInfo kInfoRowsCollectDot = {"rows_dot_kernel<collect>", "fgg_moe_permute_rows_backward", 1, 0, 0, 256, 0,
                                        0, 1024, 1024, (const void*)rows_dot_kernel<uint16_t, true, false, 2>};

template <class T>
static hipError_t scatter_impl(const T* tok, int64_t ldt, const T* fwd_rows, int64_t ldf, const float* w,
                               const int32_t* src_to_row, const int32_t* row_to_src, const int32_t* offsets,
                               int32_t E, int64_t tokens, int32_t k, int64_t N, int64_t M, T* rows, int64_t ldr,
                               float* dw, hipStream_t st) {
  constexpr int C = 2;
  const int64_t pad = (M + kPadRows - 1) / kPadRows;
  const int64_t span = (int64_t)C * 256 * Elem<T>::kVec;
  if (dw) {
    const dim3 grid((unsigned)(tokens + pad));
    trace_launch(kInfoRowsScatterDot, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens, (int)k, (long long)N,
                 (long long)M);
    if (w)
      hipLaunchKernelGGL((rows_dot_kernel<T, true, true, C>), grid, dim3(256), 0, st, tok, ldt, fwd_rows, ldf, w,
                         src_to_row, row_to_src, offsets, (int)E, tokens, (int)k, N, M, rows, ldr, dw);
    else
      hipLaunchKernelGGL((rows_dot_kernel<T, false, true, C>), grid, dim3(256), 0, st, tok, ldt, fwd_rows, ldf, w,
                         src_to_row, row_to_src, offsets, (int)E, tokens, (int)k, N, M, rows, ldr, dw);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(tokens + pad), (unsigned)((N + span - 1) / span));
  trace_launch(kInfoRowsScatter, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens, (int)k, (long long)N,
               (long long)M);
  if (w)
    hipLaunchKernelGGL((rows_scatter_kernel<T, true, C>), grid, dim3(256), 0, st, tok, ldt, w, src_to_row, row_to_src,
                       offsets, (int)E, tokens, (int)k, N, M, rows, ldr);
  else
    hipLaunchKernelGGL((rows_scatter_kernel<T, false, C>), grid, dim3(256), 0, st, tok, ldt, w, src_to_row,
                       row_to_src, offsets, (int)E, tokens, (int)k, N, M, rows, ldr);
  return hipGetLastError();
}

template <class T>
static hipError_t collect_impl(const T* rows, int64_t ldr, const T* fwd_tok, int64_t ldf, const float* w,
                               const int32_t* src_to_row, int64_t tokens, int32_t k, int64_t N, int64_t M, T* tok,
                               int64_t ldt, float* dw, hipStream_t st) {
  constexpr int C = 2;
  const int64_t span = (int64_t)C * 256 * Elem<T>::kVec;
  if (dw) {
    const dim3 grid((unsigned)tokens);
    trace_launch(kInfoRowsCollectDot, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens, (int)k, (long long)N,
                 (long long)M);
    if (w)
      hipLaunchKernelGGL((rows_dot_kernel<T, true, false, C>), grid, dim3(256), 0, st, fwd_tok, ldf, rows, ldr, w,
                         src_to_row, nullptr, nullptr, 0, tokens, (int)k, N, M, tok, ldt, dw);
    else
      hipLaunchKernelGGL((rows_dot_kernel<T, false, false, C>), grid, dim3(256), 0, st, fwd_tok, ldf, rows, ldr, w,
                         src_to_row, nullptr, nullptr, 0, tokens, (int)k, N, M, tok, ldt, dw);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)tokens, (unsigned)((N + span - 1) / span));
  trace_launch(kInfoRowsCollect, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens, (int)k, (long long)N,
               (long long)M);
  if (w)
    hipLaunchKernelGGL((rows_collect_kernel<T, true, C>), grid, dim3(256), 0, st, rows, ldr, w, src_to_row, (int)k, N,
                       M, tok, ldt);
  else
    hipLaunchKernelGGL((rows_collect_kernel<T, false, C>), grid, dim3(256), 0, st, rows, ldr, w, src_to_row, (int)k, N,
                       M, tok, ldt);
  return hipGetLastError();
}

hipError_t launch_rows_scatter(const void* tok, bool bf16, int64_t ldt, const void* fwd_rows, int64_t ldf,
                               const float* w, const int32_t* src_to_row, const int32_t* row_to_src,
                               const int32_t* offsets, int32_t E, int64_t T, int32_t k, int64_t N, int64_t M,
                               void* rows, int64_t ldr, float* dw, hipStream_t st) {
  if (bf16)
    return scatter_impl<uint16_t>((const uint16_t*)tok, ldt, (const uint16_t*)fwd_rows, ldf, w, src_to_row, row_to_src,
                                  offsets, E, T, k, N, M, (uint16_t*)rows, ldr, dw, st);
  return scatter_impl<float>((const float*)tok, ldt, (const float*)fwd_rows, ldf, w, src_to_row, row_to_src, offsets,
                             E, T, k, N, M, (float*)rows, ldr, dw, st);
}

hipError_t launch_rows_collect(const void* rows, bool bf16, int64_t ldr, const void* fwd_tok, int64_t ldf,
                               const float* w, const int32_t* src_to_row, int64_t T, int32_t k, int64_t N, int64_t M,
                               void* tok, int64_t ldt, float* dw, hipStream_t st) {
  if (bf16)
    return collect_impl<uint16_t>((const uint16_t*)rows, ldr, (const uint16_t*)fwd_tok, ldf, w, src_to_row, T, k, N, M,
                                  (uint16_t*)tok, ldt, dw, st);
  return collect_impl<float>((const float*)rows, ldr, (const float*)fwd_tok, ldf, w, src_to_row, T, k, N, M,
                             (float*)tok, ldt, dw, st);
}

}  // namespace fgg
