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
// 4096 x 2 x 4096 fp32, 201 MB in 34 us (5.9; 40 where every call has an output of its own);
// gradients of an unpermute with its weights', 8192 x 4 x 4096 bf16, 621 MB in 121 us (5.1).  The
// permuted rows are stored through the caches: past them the first took 38 us, but with the reader
// that follows (a copy of the rows) 36 us instead of 31 for 68 MB, 128 instead of 129 for 206 MB and
// 657 instead of 625 for 1 GB.  Rows are moved 16 bytes per lane; the loads and stores are declared
// with the element's alignment (this part's vector memory takes any), so odd widths and strides run
// the same path; the last vector of a row ends with it, overlapping the one before (its elements are
// written twice alike, and counted once in a dot product).  A token has a wave to itself up to 128
// vectors, four waves beyond.  (With element-wise tails and four waves for every token, 8192 x 4 x
// 500 bf16: permute 16.4 us, its gradient 70.6, unpermute 22.8, its gradient 64.4; now 10.7, 14.5,
// 9.3 and 18.9.)
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
  static __device__ u32x4 mask_from(int n) {   // all bits of elements n and on
    u32x4 m;
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = (2 * i < n ? 0u : 0xFFFFu) | (2 * i + 1 < n ? 0u : 0xFFFF0000u);
    return m;
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
  static __device__ u32x4 mask_from(int n) {
    u32x4 m;
#pragma unroll
    for (int i = 0; i < 4; ++i) m[i] = i < n ? 0u : ~0u;
    return m;
  }
};

// The vector of lane-vector number v in a row of N: its first column (the last vector ends with the row),
// or with TINY (N < kVec, one vector) column 0.
template <class T, bool TINY>
__device__ inline int64_t vec_col(int64_t v, int64_t N) {
  if constexpr (TINY) return 0;
  const int64_t col = v * Elem<T>::kVec;
  return col < N - Elem<T>::kVec ? col : N - Elem<T>::kVec;
}

// kVec elements from `col` of a row (TINY: the row's N, then zeros).  ONCE: nothing else reads them (no
// place in the caches is asked for).
template <class T, bool TINY, bool ONCE = false>
__device__ inline u32x4 load_vec(const T* row, int64_t col, int64_t N) {
  if constexpr (!TINY) {
    const auto* p = reinterpret_cast<const typename Elem<T>::Packed*>(row + col);
    if constexpr (ONCE) return __builtin_nontemporal_load(p);
    else return *p;
  } else {
    union {
      u32x4 v;
      T e[Elem<T>::kVec];
    } u;
    u.v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < Elem<T>::kVec - 1; ++i)
      if (i < N) u.e[i] = row[i];
    return u.v;
  }
}

template <class T, bool TINY>
__device__ inline void store_vec(T* row, int64_t col, int64_t N, u32x4 v) {
  if constexpr (!TINY) {
    *reinterpret_cast<typename Elem<T>::Packed*>(row + col) = v;
  } else {
    union {
      u32x4 v;
      T e[Elem<T>::kVec];
    } u;
    u.v = v;
#pragma unroll
    for (int i = 0; i < Elem<T>::kVec - 1; ++i)
      if (i < N) row[i] = u.e[i];
  }
}

constexpr int kPadRows = 16;    // rows of the permuted order that one padding block looks at, four per wave

// Zeros in vectors [v0, v1) of the padding rows among [r0, r0 + kPadRows).
template <class T, bool TINY>
__device__ inline void clear_padding(const int32_t* row_to_src, int64_t total, int64_t r0, int64_t N, T* rows,
                                     int64_t ldr, int64_t v0, int64_t v1) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = 0; i < kPadRows / 4; ++i) {
    const int64_t r = r0 + wave * (kPadRows / 4) + i;
    if (r >= total || row_to_src[r] >= 0) continue;
    for (int64_t v = v0 + lane; v < v1; v += 64)
      store_vec<T, TINY>(rows + r * ldr, vec_col<T, TINY>(v, N), N, u32x4{0, 0, 0, 0});
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

// The place of a thread: WPT waves (1 or 4) share a token, a 256-thread block has 4 / WPT tokens.  The
// thread's vectors are lane_vec() + c * 64 * WPT.
template <int WPT>
__device__ inline int64_t block_token() {
  return (int64_t)blockIdx.x * (4 / WPT) + (WPT == 1 ? threadIdx.x >> 6 : 0);
}
template <int WPT>
__device__ inline int lane_vec() { return WPT == 1 ? threadIdx.x & 63 : threadIdx.x; }

// Scatter: a token's part (t, y) takes C * 64 * WPT vectors of the token, one pass, and writes them
// to each of the token's rows (a token without a row is not read); the blocks behind the last
// token clear padding rows.
template <class T, bool W, int C, int WPT, bool TINY>
__global__ void __launch_bounds__(256) rows_scatter_kernel(const T* __restrict__ tok, int64_t ldt,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ src_to_row,
                                                           const int32_t* __restrict__ row_to_src,
                                                           const int32_t* __restrict__ offsets, int E, int64_t tokens,
                                                           int k, int64_t N, int64_t M, T* __restrict__ rows,
                                                           int64_t ldr) {
  constexpr int V = Elem<T>::kVec;
  const int64_t nv = (N + V - 1) / V, v0 = (int64_t)blockIdx.y * (C * 64 * WPT);
  const int64_t token_blocks = (tokens + 4 / WPT - 1) / (4 / WPT);
  if ((int64_t)blockIdx.x >= token_blocks) {
    int64_t total = offsets[E];
    if (total > M) total = M;
    clear_padding<T, TINY>(row_to_src, total, ((int64_t)blockIdx.x - token_blocks) * kPadRows, N, rows, ldr, v0,
                           v0 + C * 64 * WPT < nv ? v0 + C * 64 * WPT : nv);
    return;
  }
  const int64_t t = block_token<WPT>();
  if (t >= tokens) return;
  int row;
  uint64_t live = token_rows(src_to_row, t, k, M, row);
  if (live == 0) return;
  float wt = 1.0f;
  if constexpr (W) wt = (int)(threadIdx.x & 63) < k ? w[t * k + (threadIdx.x & 63)] : 0.0f;
  u32x4 x[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
    if (v < nv) x[c] = load_vec<T, TINY>(tok + t * ldt, vec_col<T, TINY>(v, N), N);
  }
  while (live) {
    const int j = next_slot(live);
    T* out = rows + (int64_t)lane_int(row, j) * ldr;
    const float wj = lane_float(wt, j);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
      if (v >= nv) continue;
      u32x4 y = x[c];
      if constexpr (W) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = wj * Elem<T>::get(x[c], i);
        y = Elem<T>::pack(f);
      }
      store_vec<T, TINY>(out, vec_col<T, TINY>(v, N), N, y);
    }
  }
}

// Collect: a token's part (t, y) sums C * 64 * WPT vectors of its rows, B rows' loads at a time, added in
// slot order.
template <class T, int C, int WPT, bool TINY, int B>
__device__ inline void collect_rows(const T* rows, int64_t ldr, int64_t v0, int64_t nv, int64_t N, int row, float wt,
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
      const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
      if (v < nv) y[b][c] = load_vec<T, TINY>(in, vec_col<T, TINY>(v, N), N);
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < V; ++i) acc[c][i] = fmaf(wj[b], Elem<T>::get(y[b][c], i), acc[c][i]);
}

template <class T, bool W, int C, int WPT, bool TINY>
__global__ void __launch_bounds__(256) rows_collect_kernel(const T* __restrict__ rows, int64_t ldr,
                                                           const float* __restrict__ w,
                                                           const int32_t* __restrict__ src_to_row, int64_t tokens,
                                                           int k, int64_t N, int64_t M, T* __restrict__ tok,
                                                           int64_t ldt) {
  constexpr int V = Elem<T>::kVec;
  const int64_t t = block_token<WPT>(), nv = (N + V - 1) / V, v0 = (int64_t)blockIdx.y * (C * 64 * WPT);
  if (t >= tokens) return;
  int row;
  uint64_t live = token_rows(src_to_row, t, k, M, row);
  float wt = 1.0f;
  if constexpr (W) wt = (int)(threadIdx.x & 63) < k ? w[t * k + (threadIdx.x & 63)] : 0.0f;
  float acc[C][V];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[c][i] = 0.0f;
  while (__popcll(live) >= 4) collect_rows<T, C, WPT, TINY, 4>(rows, ldr, v0, nv, N, row, wt, live, acc);
  if (__popcll(live) >= 2) collect_rows<T, C, WPT, TINY, 2>(rows, ldr, v0, nv, N, row, wt, live, acc);
  if (live) collect_rows<T, C, WPT, TINY, 1>(rows, ldr, v0, nv, N, row, wt, live, acc);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
    if (v < nv) store_vec<T, TINY>(tok + t * ldt, vec_col<T, TINY>(v, N), N, Elem<T>::pack(acc[c]));
  }
}

// The gradients with dw: a token's waves go over the whole row, since dw[p] is a sum over it.
// SCATTER: tok (the gradient of the output) goes to the rows' gradients `out`, dotted with the
// forward's rows.  Otherwise the rows (gradients) are summed into the token's gradient `out`,
// each dotted with the forward's token.  Partial dots: per thread, then per wave, then the four
// waves of LDS in order.  once: the elements that count in the dot product (those of the last vector
// that the one before has do not); both factors are masked with it, since 0 * inf is a NaN.
template <class T, bool SCATTER, int C, int WPT, bool TINY, int B>
__device__ inline void dot_rows(const T* rows, int64_t ldr, T* out, int64_t ldo, int64_t v0, int64_t nv, int64_t N,
                                int row, float wt, const u32x4 (&x)[C], const u32x4 (&once)[C], uint64_t& live,
                                float (&acc)[C][Elem<T>::kVec], float* part) {
  constexpr int V = Elem<T>::kVec;
  u32x4 y[B][C];
  int slot[B];
#pragma unroll
  for (int b = 0; b < B; ++b) {
    slot[b] = next_slot(live);
    const T* in = rows + (int64_t)lane_int(row, slot[b]) * ldr;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
      y[b][c] = u32x4{0, 0, 0, 0};
      if (v < nv) y[b][c] = load_vec<T, TINY, true>(in, vec_col<T, TINY>(v, N), N);
    }
  }
#pragma unroll
  for (int b = 0; b < B; ++b) {
    const float wj = lane_float(wt, slot[b]);
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
      const u32x4 xd = x[c] & once[c], yd = y[b][c] & once[c];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        dot = fmaf(Elem<T>::get(xd, i), Elem<T>::get(yd, i), dot);
        if constexpr (!SCATTER) acc[c][i] = fmaf(wj, Elem<T>::get(y[b][c], i), acc[c][i]);
      }
      if constexpr (SCATTER) {
        float f[V];
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = wj * Elem<T>::get(x[c], i);
        if (v < nv)
          store_vec<T, TINY>(out + (int64_t)lane_int(row, slot[b]) * ldo, vec_col<T, TINY>(v, N), N, Elem<T>::pack(f));
      }
    }
    dot = group_reduce<64>(dot, OpAdd());
    if ((threadIdx.x & 63) == 0) part[slot[b]] += dot;
  }
}

template <class T, bool W, bool SCATTER, int C, int WPT, bool TINY>
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
  const int64_t nv = (N + V - 1) / V, token_blocks = (tokens + 4 / WPT - 1) / (4 / WPT);
  if (SCATTER && (int64_t)blockIdx.x >= token_blocks) {
    int64_t total = offsets[E];
    if (total > M) total = M;
    clear_padding<T, TINY>(row_to_src, total, ((int64_t)blockIdx.x - token_blocks) * kPadRows, N, out, ldo, 0, nv);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = block_token<WPT>();
  if (WPT == 1 && t >= tokens) return;                // (no barrier with a wave to a token)
  int row;
  const uint64_t slots = token_rows(src_to_row, t, k, M, row);
  float wt = 1.0f;
  if constexpr (W) wt = lane < k ? w[t * k + lane] : 0.0f;
  part[wave][lane] = 0.0f;                            // (each wave its own row)
  wave_sync();
  for (int64_t v0 = 0; v0 < nv; v0 += C * 64 * WPT) {
    if (SCATTER && slots == 0) break;
    u32x4 x[C], once[C];
    float acc[C][V];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
      x[c] = u32x4{0, 0, 0, 0};
      if (v < nv && slots != 0) x[c] = load_vec<T, TINY>(tok + t * ldt, vec_col<T, TINY>(v, N), N);
      once[c] = Elem<T>::mask_from(!TINY && v == nv - 1 ? (int)(nv * V - N) : 0);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[c][i] = 0.0f;
    }
    uint64_t live = slots;
    while (__popcll(live) >= 4)
      dot_rows<T, SCATTER, C, WPT, TINY, 4>(rows, ldr, out, ldo, v0, nv, N, row, wt, x, once, live, acc, part[wave]);
    if (__popcll(live) >= 2)
      dot_rows<T, SCATTER, C, WPT, TINY, 2>(rows, ldr, out, ldo, v0, nv, N, row, wt, x, once, live, acc, part[wave]);
    if (live)
      dot_rows<T, SCATTER, C, WPT, TINY, 1>(rows, ldr, out, ldo, v0, nv, N, row, wt, x, once, live, acc, part[wave]);
    if constexpr (!SCATTER) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t v = v0 + c * 64 * WPT + lane_vec<WPT>();
        if (v < nv) store_vec<T, TINY>(out + t * ldo, vec_col<T, TINY>(v, N), N, Elem<T>::pack(acc[c]));
      }
    }
  }
  if constexpr (WPT == 1) {
    wave_sync();
    if (lane < k) dw[t * k + lane] = part[wave][lane];
  } else {
    __syncthreads();
    if ((int)threadIdx.x < k) {
      const int j = threadIdx.x;
      dw[t * k + j] = (part[0][j] + part[1][j]) + (part[2][j] + part[3][j]);
    }
  }
}

const KernelInfo kInfoRowsScatter = {"rows_scatter_kernel", "fgg_moe_permute_rows, fgg_moe_unpermute_rows_backward", 1,
                                     0, 0, 256, 0, 0, 0, 0, (const void*)rows_scatter_kernel<uint16_t, false, 2, 4, false>};
const KernelInfo kInfoRowsCollect = {"rows_collect_kernel", "fgg_moe_unpermute_rows, fgg_moe_permute_rows_backward", 1,
                                     0, 0, 256, 0, 0, 0, 0, (const void*)rows_collect_kernel<uint16_t, true, 2, 4, false>};
const KernelInfo kInfoRowsScatterDot = {"rows_dot_kernel<scatter>", "fgg_moe_unpermute_rows_backward", 1, 0, 0, 256, 0,
                                        0, 1024, 1024, (const void*)rows_dot_kernel<uint16_t, true, true, 2, 4, false>};
const KernelInfo kInfoRowsCollectDot = {"rows_dot_kernel<collect>", "fgg_moe_permute_rows_backward", 1, 0, 0, 256, 0,
                                        0, 1024, 1024, (const void*)rows_dot_kernel<uint16_t, true, false, 2, 4, false>};

// Calls f(waves per token, whether the row is shorter than a vector) as compile-time constants.
template <class T, class F>
static void with_row_shape(int64_t N, F f) {
  using std::integral_constant;
  if (N < Elem<T>::kVec) f(integral_constant<int, 1>(), std::true_type());
  else if (N <= 128 * Elem<T>::kVec) f(integral_constant<int, 1>(), std::false_type());
  else f(integral_constant<int, 4>(), std::false_type());
}

template <class T>
static hipError_t scatter_impl(const T* tok, int64_t ldt, const T* fwd_rows, int64_t ldf, const float* w,
                               const int32_t* src_to_row, const int32_t* row_to_src, const int32_t* offsets,
                               int32_t E, int64_t tokens, int32_t k, int64_t N, int64_t M, T* rows, int64_t ldr,
                               float* dw, hipStream_t st) {
  constexpr int C = 2;
  const int64_t pad = (M + kPadRows - 1) / kPadRows, nv = (N + Elem<T>::kVec - 1) / Elem<T>::kVec;
  with_row_shape<T>(N, [&](auto wpt, auto tiny) {
    constexpr int WPT = decltype(wpt)::value;
    constexpr bool TINY = decltype(tiny)::value;
    const int64_t blocks = (tokens + 4 / WPT - 1) / (4 / WPT) + pad;
    const dim3 grid((unsigned)blocks, dw ? 1u : (unsigned)((nv + C * 64 * WPT - 1) / (C * 64 * WPT)));
    trace_launch(dw ? kInfoRowsScatterDot : kInfoRowsScatter, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens,
                 (int)k, (long long)N, (long long)M);
    auto go = [&](auto weighted) {
      constexpr bool W = decltype(weighted)::value;
      if (dw)
        hipLaunchKernelGGL((rows_dot_kernel<T, W, true, C, WPT, TINY>), grid, dim3(256), 0, st, tok, ldt, fwd_rows,
                           ldf, w, src_to_row, row_to_src, offsets, (int)E, tokens, (int)k, N, M, rows, ldr, dw);
      else
        hipLaunchKernelGGL((rows_scatter_kernel<T, W, C, WPT, TINY>), grid, dim3(256), 0, st, tok, ldt, w, src_to_row,
                           row_to_src, offsets, (int)E, tokens, (int)k, N, M, rows, ldr);
    };
    if (w) go(std::true_type());
    else go(std::false_type());
  });
  return hipGetLastError();
}

template <class T>
static hipError_t collect_impl(const T* rows, int64_t ldr, const T* fwd_tok, int64_t ldf, const float* w,
                               const int32_t* src_to_row, int64_t tokens, int32_t k, int64_t N, int64_t M, T* tok,
                               int64_t ldt, float* dw, hipStream_t st) {
  constexpr int C = 2;
  const int64_t nv = (N + Elem<T>::kVec - 1) / Elem<T>::kVec;
  with_row_shape<T>(N, [&](auto wpt, auto tiny) {
    constexpr int WPT = decltype(wpt)::value;
    constexpr bool TINY = decltype(tiny)::value;
    const dim3 grid((unsigned)((tokens + 4 / WPT - 1) / (4 / WPT)),
                    dw ? 1u : (unsigned)((nv + C * 64 * WPT - 1) / (C * 64 * WPT)));
    trace_launch(dw ? kInfoRowsCollectDot : kInfoRowsCollect, grid, "T=%lld k=%d N=%lld M=%lld", (long long)tokens,
                 (int)k, (long long)N, (long long)M);
    auto go = [&](auto weighted) {
      constexpr bool W = decltype(weighted)::value;
      if (dw)
        hipLaunchKernelGGL((rows_dot_kernel<T, W, false, C, WPT, TINY>), grid, dim3(256), 0, st, fwd_tok, ldf, rows,
                           ldr, w, src_to_row, nullptr, nullptr, 0, tokens, (int)k, N, M, tok, ldt, dw);
      else
        hipLaunchKernelGGL((rows_collect_kernel<T, W, C, WPT, TINY>), grid, dim3(256), 0, st, rows, ldr, w, src_to_row,
                           tokens, (int)k, N, M, tok, ldt);
    };
    if (w) go(std::true_type());
    else go(std::false_type());
  });
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
