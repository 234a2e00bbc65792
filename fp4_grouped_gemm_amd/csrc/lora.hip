// Low-rank adapters of many requests beside one shared projection (gfx950):
//
//   out[t] = base[t] + scales[i] (x[t] A_i^T) B_i^T,   i = ids[t];   out[t] = base[t] without an adapter
//
// Few tokens: one kernel for both products (lora_few_kernel).  Else two: x A^T into fp32 sums per token (the sum over
// K cut into chunks, a workgroup per chunk and tile of tokens; lora_shrink_kernel, for many tokens lora_tiles_kernel),
// and the product with B on top of base (lora_expand_kernel).  What bounds them: many tokens are near memory (every
// adapter's factors once, x, base and out: 8192 tokens of 8 prompts, rank 64, 4096 -> 4096: 52 us for 203 MB, 3.9
// TB/s), less the start of two launches; few are a chain of latencies, ids, A with x, then B (16 tokens of 16
// requests, rank 16, 7168 -> 4096: 5.8 us for 4.2 MB); many in any order are the first product's passes, one for each
// of a tile's adapters (the same 8192 tokens 206 us).
//
//  * tokens come in any order, in tiles of 16 to 64.  A wave finds the tile's distinct adapters by
//    ballots over the tokens' ids; the work is cut into items of one adapter and one piece of the
//    sum (or of the columns), dealt to the workgroup's eight waves in turn, so that sixteen requests
//    with an adapter each and one prompt with one keep all waves loading.
//  * v_mfma_f32_16x16x32_bf16 with the factor's rows as the first operand and 16 tokens as the second;
//    only an item's own tokens are loaded, and only their columns of the result are taken, so what
//    stands in other adapters or tokens (NaN, infinities) never reaches a token.
//  * the low-rank sums stay exact to fp32 for the second product: they are split into two bf16 parts
//    (three when out is fp32), which costs matrix instructions that memory hides.
//  * the partial sums of the chunks and waves are added in a fixed order.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_segments.hpp"
#include "fgg_wave.hpp"

namespace fgg {

namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kFewWaves = 16, kFewThreads = 64 * kFewWaves;
constexpr int kSpan = 128;               // of the sum over K per item
constexpr int kCols = 32;                // columns per item of the second product
constexpr float kMaxBf16 = 0x1.FEp127f;

__device__ inline v8bf load_or_zero(const uint16_t* p, bool on) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (on) u = *reinterpret_cast<const uint4*>(p);
  return __builtin_bit_cast(v8bf, u);
}

// Bit 15 of each half whose exponent is all ones: an infinity or NaN among two bf16 values.
__device__ inline uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// The lane's token's adapter, -1 where it has none (or there is no token).
__device__ inline int lane_adapter(const int32_t* ids, int64_t t0, int tokens, int64_t T, int L, int lane) {
  int id = -1;
  if (lane < tokens && t0 + lane < T) id = ids[t0 + lane];
  return id >= 0 && id < L ? id : -1;
}

}  // namespace

// This wave's items of a tile: each adapter of the tile that is this workgroup's (every `parts`-th) with each step of
// [from, to), dealt to the workgroup's waves in turn.
struct Items {
  uint64_t left;         // tokens whose adapter is still to come
  uint64_t match;        // the current adapter's tokens
  int cur;               // the current adapter
  int64_t at, from, to;  // current place
  int step, item, wave;
  int parts, wait;       // workgroups that share the tile's adapters; adapters before this one's next
  uint64_t mine;         // tokens of this workgroup's adapters so far

  // The next item of this wave; false when there is none.
  __device__ bool next(int id) {
    while (true) {
      if (at >= to) {
        if (!left) return false;
        cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        match = __ballot(id == cur);
        left &= ~match;
        if (wait-- > 0) continue;
        wait = parts - 1;
        mine |= match;
        at = from - step;
      }
      // (the steps up to the wave's own are passed over at once)
      const int skip = (wave - item) & (kWaves - 1);
      const int64_t rest = (to - at - 1) / step;      // steps left after `at`
      if (skip + 1 > rest) {
        item = (int)((item + rest) & (kWaves - 1));
        at = to;
        continue;
      }
      at += (int64_t)(skip + 1) * step;
      item = (item + skip + 1) & (kWaves - 1);
      return true;
    }
  }
};

// part[chunk][t][j] = sum over the chunk's k of x[t][k] A[ids[t]][j][k] for a tile of 16 tokens; RT tiles of 16 ranks.
template <int RT>
__global__ void __launch_bounds__(kThreads, RT == 1 || RT == 4 ? 4 : 2)
lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
                   const uint16_t* __restrict__ a, int64_t T, int L, int r, int64_t K, int chunk,
                   float* __restrict__ part) {
  __shared__ float red[kWaves][16][16 + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int64_t k0 = (int64_t)blockIdx.y * chunk, k1 = k0 + chunk < K ? k0 + chunk : K;
  const int id = lane_adapter(ids, t0, 16, T, L, lane);

  v4f sum[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) sum[i] = v4f{0.f, 0.f, 0.f, 0.f};
  constexpr int kSteps = kSpan / 32;
  struct Operands {
    v8bf x[kSteps], a[RT][kSteps];
    uint64_t match;
  };
  auto load_a = [&](const Items& it, Operands& o, int i) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t k = it.at + 32 * s + 8 * q;
      const int row = 16 * i + l16;
      o.a[i][s] = load_or_zero(a + ((int64_t)it.cur * r + row) * K + k, row < r && k < k1);
    }
  };
  auto load_x = [&](const Items& it, Operands& o) {
    o.match = it.match;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t k = it.at + 32 * s + 8 * q;
      o.x[s] = load_or_zero(x + (t0 + l16) * ldx + k, (it.match >> l16 & 1) && k < k1);
    }
  };
  auto load = [&](const Items& it, Operands& o) {
    load_x(it, o);
#pragma unroll
    for (int i = 0; i < RT; ++i) load_a(it, o, i);
  };
  auto use = [&](const Operands& o, int from, int to) {
#pragma unroll
    for (int i = from; i < to; ++i) {
      v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o.a[i][s], o.x[s], d, 0, 0, 0);
      const bool on = o.match >> l16 & 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] += on ? d[e] : 0.0f;
    }
  };
  Items it = {__ballot(id >= 0), 0, -1, k1, k0, k1, kSpan, kWaves - 1, wave, (int)gridDim.z, (int)blockIdx.z, 0};
  if constexpr (RT <= 2) {               // the next item's operands are loaded before this one's are waited for
    Operands o[2];
    bool more = it.next(id);
    if (more) load(it, o[0]);
    while (more) {
      more = it.next(id);
      if (more) load(it, o[1]);
      use(o[0], 0, RT);
      if (!more) break;
      more = it.next(id);
      if (more) load(it, o[0]);
      use(o[1], 0, RT);
    }
  } else {                               // (more would not fit the registers: other waves cover the waits)
    Operands o;
    while (it.next(id)) {
      load_x(it, o);
      load_a(it, o, 0);
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        if (i + 1 < RT) load_a(it, o, i + 1);
        use(o, i, i + 1);
      }
    }
  }

  // the eight waves' sums, in their order
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    if (16 * i >= r) break;
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][l16][4 * q + e] = sum[i][e];
    __syncthreads();
    if (threadIdx.x < 256) {
      const int t = threadIdx.x >> 4, j = threadIdx.x & 15;
      float total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += red[w][t][j];
      if ((it.mine >> t & 1) && 16 * i + j < r) part[((int64_t)blockIdx.y * T + t0 + t) * r + 16 * i + j] = total;
    }
    __syncthreads();
  }
}

// out[t][n] = base[t][n] + sum_j v[t][j] B[ids[t]][n][j],  v = scales[ids[t]] times the chunks' sums.
// TT tiles of 16 tokens, rank up to 32 RS.
template <int TT, int RS, bool F32>
__global__ void __launch_bounds__(kThreads, TT == 4 && (RS == 4 || F32) ? 2 : 4)
lora_expand_kernel(const float* __restrict__ part, int chunks, const int32_t* __restrict__ ids,
                   const uint16_t* __restrict__ b, const float* __restrict__ scales, const void* base, int64_t ldb,
                   void* out, int64_t ldo, int64_t T, int L, int r, int64_t N, int cols) {
  constexpr int kParts = F32 ? 3 : 2, kVRow = 32 * RS + 8, kElem = F32 ? 4 : 2;
  __shared__ __align__(16) uint16_t vs[kParts][16 * TT][kVRow];
  __shared__ float4 red[kThreads];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int64_t n_from = (int64_t)blockIdx.y * cols, n_to = n_from + cols < N ? n_from + cols : N;
  const int id = lane_adapter(ids, t0, 16 * TT, T, L, lane);

  // an item's operands: rows of two fragments are dealt so that a lane's results are eight consecutive columns
  struct Operands {
    v8bf b[2][RS];
    uint4 y[TT][kElem / 2];
    uint64_t match;
    int64_t at;
    int cur;
  };
  // (of high ranks, an item's addresses are formed anew: held, they would spill)
  auto fresh_lane = [&]() {
    int l = lane;
    if constexpr (RS == 4) asm volatile("" : "+v"(l));
    return l;
  };
  auto load = [&](const Items& it, Operands& o) {
    const int l = fresh_lane(), l16 = l & 15, q = l >> 4;
    o.match = it.match;
    o.at = it.at;
    o.cur = it.cur;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const int64_t n = it.at + 8 * (l16 >> 2) + 4 * f + (l16 & 3);
        const int j = 32 * s + 8 * q;
        o.b[f][s] = load_or_zero(b + ((int64_t)it.cur * N + n) * r + j, n < n_to && j < r);
      }
#pragma unroll
    for (int f = 0; f < TT; ++f) {
      const int64_t t = t0 + 16 * f + l16, n = it.at + 8 * q;
      if ((it.match >> (16 * f + l16) & 1) && n < n_to) {
        const uint4* p = reinterpret_cast<const uint4*>((const char*)base + (t * ldb + n) * kElem);
#pragma unroll
        for (int k = 0; k < kElem / 2; ++k) o.y[f][k] = p[k];
      }
    }
  };
  auto store = [&](int64_t t, int64_t n, const float* y) {
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>((float*)out + t * ldo + n);
      o[0] = make_float4(y[0], y[1], y[2], y[3]);
      o[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
      *reinterpret_cast<uint4*>((uint16_t*)out + t * ldo + n) =
          make_uint4(bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]), bf16x2_rne(y[6], y[7]));
    }
  };
  // Whether an item has an infinity or NaN among its factors.  An infinite one makes NaN with the later parts of v, which
  // may be 0 or of the other sign: the columns of such factors are done again, with v as a whole.
  auto not_all_finite = [&](const Operands& o) {
    uint32_t odd = 0;
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        const uint4 u = __builtin_bit_cast(uint4, o.b[f][s]);
        odd |= not_finite(u.x) | not_finite(u.y) | not_finite(u.z) | not_finite(u.w);
      }
    return __ballot(odd != 0) != 0;
  };
  auto unpack = [&](const Operands& o, int f, float* y) {
    if constexpr (F32) {
      __builtin_memcpy(y, o.y[f], 32);
    } else {
      const uint32_t w[4] = {o.y[f][0].x, o.y[f][0].y, o.y[f][0].z, o.y[f][0].w};
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
  };
  // The columns of an item whose factors are not all finite, one by one.
  auto again = [&](const Operands& o) {
#pragma unroll
    for (int f = 0; f < TT; ++f) {
      const int at = 16 * f + l16;
      if (!(o.match >> at & 1)) continue;
      float y[8];
      unpack(o, f, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t t = t0 + at, n = o.at + 8 * q + e;
        if (n >= n_to) continue;
        const uint16_t* bl = b + ((int64_t)o.cur * N + n) * r;
        bool finite = true;
        float d = 0.0f;
#pragma unroll 1
        for (int j = 0; j < r; ++j) {
          float v = 0.0f;
#pragma unroll
          for (int p = kParts - 1; p >= 0; --p) v += bf16_to_f32(vs[p][at][j]);
          finite &= not_finite(bl[j]) == 0;
          d = fmaf(v, bf16_to_f32(bl[j]), d);
        }
        if (finite) continue;
        if constexpr (F32) ((float*)out)[t * ldo + n] = y[e] + d;
        else ((uint16_t*)out)[t * ldo + n] = (uint16_t)bf16x2_rne(y[e] + d, 0.0f);
      }
    }
  };
  auto use = [&](const Operands& o) {
    const int l = fresh_lane(), l16 = l & 15, q = l >> 4;
#pragma unroll
    for (int f = 0; f < TT; ++f) {
      if ((o.match >> (16 * f) & 0xFFFF) == 0) continue;
      v4f d[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p) {
          const v8bf v = *reinterpret_cast<const v8bf*>(&vs[p][16 * f + l16][32 * s + 8 * q]);
          d[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o.b[0][s], v, d[0], 0, 0, 0);
          d[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(o.b[1][s], v, d[1], 0, 0, 0);
        }
      const int64_t n = o.at + 8 * q;
      if ((o.match >> (16 * f + l16) & 1) && n < n_to) {
        float y[8];
        unpack(o, f, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += d[e >> 2][e & 3];
        store(t0 + 16 * f + l16, n, y);
      }
    }
    // (asked after the products and their stores: before, they would wait for it.  8192 tokens of 8 runs, 4096 -> 4096,
    // without / with: rank 16 40.1 / 41.4 us, rank 64 51.0 / 51.4; 64 adapters in any order 98 / 103.)
    if (__builtin_expect(not_all_finite(o), 0)) again(o);
  };

  Items it = {__ballot(id >= 0), 0, -1, n_to, n_from, n_to, kCols, kWaves - 1, wave, 1, 0, 0};
  Operands o[2];
  bool more = it.next(id);
  if (more) load(it, o[0]);

  // The tokens' low-rank sums in bf16 parts, zeros past the rank, four at a time.  With many chunks several threads
  // share them, each a run of chunks in order, and the runs are added in order.
  constexpr int kQuads = 16 * TT * 8 * RS;
  auto sum_of = [&](int quad, int c0, int c1) {
    const int t = quad / (8 * RS), j = quad % (8 * RS) * 4;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t0 + t < T && j < r) {
      const float4* p = reinterpret_cast<const float4*>(part + (t0 + t) * r + j);
      const int64_t stride = T * r / 4;
      for (int c = c0; c < c1; c += 4) {
        float4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = c + k < c1 ? p[(c + k) * stride] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 4; ++k) s.x += v[k].x, s.y += v[k].y, s.z += v[k].z, s.w += v[k].w;
      }
    }
    return s;
  };
  auto keep = [&](int quad, float4 s) {
    const int t = quad / (8 * RS), j = quad % (8 * RS) * 4;
    const int i = t0 + t < T ? ids[t0 + t] : -1;
    const bool on = i >= 0 && i < L;
    const float scale = on && scales ? scales[i] : 1.0f;
    float v[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = on ? v[e] * scale : 0.0f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      float c[4];                        // (a finite sum past the largest bf16 value stays finite)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = fabsf(v[e]) < INFINITY ? __builtin_amdgcn_fmed3f(v[e], -kMaxBf16, kMaxBf16) : v[e];
      const uint32_t w[2] = {bf16x2_rne(c[0], c[1]), bf16x2_rne(c[2], c[3])};
      *reinterpret_cast<uint2*>(&vs[p][t][j]) = make_uint2(w[0], w[1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {      // (an infinite or NaN part carries the whole)
        const float v0 = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
        v[e] = fabsf(v0) < INFINITY ? v[e] - v0 : 0.0f;
      }
    }
  };
  if constexpr (kQuads < kThreads) {
    constexpr int kRuns = kThreads / kQuads;
    const int quad = threadIdx.x % kQuads, run = threadIdx.x / kQuads, each = (chunks + kRuns - 1) / kRuns;
    const int c0 = run * each, c1 = c0 + each < chunks ? c0 + each : chunks;
    red[threadIdx.x] = sum_of(quad, c0, c1);
    __syncthreads();
    if (threadIdx.x < kQuads) {
      float4 s = red[threadIdx.x];
#pragma unroll
      for (int k = 1; k < kRuns; ++k) {
        const float4 v = red[k * kQuads + threadIdx.x];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
      }
      keep(threadIdx.x, s);
    }
  } else {
    for (int quad = threadIdx.x; quad < kQuads; quad += kThreads) keep(quad, sum_of(quad, 0, chunks));
  }
  __syncthreads();

  while (more) {
    more = it.next(id);
    if (more) load(it, o[1]);
    use(o[0]);
    if (!more) break;
    more = it.next(id);
    if (more) load(it, o[0]);
    use(o[1]);
  }

  if (out != base) {                     // tokens without an adapter: copied
    const uint64_t none = __ballot(id < 0 && lane < 16 * TT && t0 + lane < T);
    for (int64_t n0 = n_from + wave * kCols; none && n0 < n_to; n0 += kWaves * kCols) {
#pragma unroll
      for (int f = 0; f < TT; ++f) {
        const int64_t t = t0 + 16 * f + l16, n = n0 + 8 * q;
        if ((none >> (16 * f + l16) & 1) && n < n_to) {
          const uint4* p = reinterpret_cast<const uint4*>((const char*)base + (t * ldb + n) * kElem);
          uint4* to = reinterpret_cast<uint4*>((char*)out + (t * ldo + n) * kElem);
#pragma unroll
          for (int k = 0; k < kElem / 2; ++k) to[k] = p[k];
        }
      }
    }
  }
}

// Few tokens: one workgroup of sixteen waves takes a token and 1024 columns, and both products (no workspace, one
// launch).  Each workgroup forms its token's low-rank sums anew: reading A again from the caches costs less than a
// second launch.  The waves share the sum over K in pieces of 64; a load takes whole 128-byte lines of eight rows
// of A (a compute unit's cache serves lines, not bytes: the matrix operand's order, half lines of sixteen rows,
// ran at half the rate), eight lanes a row, whose products meet by lane exchanges.  Then a thread takes a column.
// RG: groups of eight ranks.
template <int RG, bool F32>
__global__ void __launch_bounds__(kFewThreads, 4)
lora_few_kernel(const uint16_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
                const uint16_t* __restrict__ a, const uint16_t* __restrict__ b, const float* __restrict__ scales,
                const void* base, int64_t ldb, void* out, int64_t ldo, int L, int r, int64_t N, int64_t K) {
  __shared__ float red[kFewWaves][8 * RG];
  __shared__ float vs[8 * RG];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = blockIdx.y;
  const int n = (int)blockIdx.x * kFewThreads + threadIdx.x;       // (N is at most 2^20)
  const int id = ids[t];
  const bool has = id >= 0 && id < L;
  if (!has && out == base) return;
  float y = 0.0f;
  if (n < N) y = F32 ? ((const float*)base)[t * ldb + n] : bf16_to_f32(((const uint16_t*)base)[t * ldb + n]);
  if (has) {
    float acc[RG];
#pragma unroll
    for (int g = 0; g < RG; ++g) acc[g] = 0.0f;
    // (row addresses in scalar registers, and a lane's 32-bit offset in bytes: 64-bit addresses of 128 ranks spill)
    const uint16_t *xt = x + t * ldx, *at = a + (int64_t)id * r * K;
    const uint32_t row = (uint32_t)(lane >> 3) * (uint32_t)(K * 2);
    // kU pieces' loads fly together; ALL: all of them lie inside the sum (else what is past it is zero)
    constexpr int kU = RG <= 2 ? 4 : RG == 4 ? 3 : RG == 8 ? 2 : 1;
    auto take = [&](auto all_tag, int64_t p) {
      constexpr bool ALL = decltype(all_tag)::value;
      uint4 aw[kU][RG], xw[kU];
      // (past the sum: some piece inside it, then zeros in its place; ranks past r: the first rows again, dropped)
      bool on[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        uint32_t k = (uint32_t)(p + u * kFewWaves) * 64 + 8 * (lane & 7);
        on[u] = ALL || k < K;
        k = on[u] ? 2 * k : 0;
        xw[u] = *reinterpret_cast<const uint4*>((const char*)xt + k);
#pragma unroll
        for (int g = 0; g < RG; ++g)
          aw[u][g] = *reinterpret_cast<const uint4*>((const char*)(at + (8 * g < r ? 8 * g : 0) * K) + (row + k));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (!ALL) {
        auto keep = [](uint4 v, bool on) { return make_uint4(on ? v.x : 0, on ? v.y : 0, on ? v.z : 0, on ? v.w : 0); };
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          xw[u] = keep(xw[u], on[u]);
#pragma unroll
          for (int g = 0; g < RG; ++g) aw[u][g] = keep(aw[u][g], on[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t xs[4] = {xw[u].x, xw[u].y, xw[u].z, xw[u].w};
#pragma unroll
        for (int g = 0; g < RG; ++g) {
          const uint32_t as[4] = {aw[u][g].x, aw[u][g].y, aw[u][g].z, aw[u][g].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[g] = fmaf(__uint_as_float(as[e] << 16), __uint_as_float(xs[e] << 16), acc[g]);
            acc[g] = fmaf(__uint_as_float(as[e] & 0xFFFF0000u), __uint_as_float(xs[e] & 0xFFFF0000u), acc[g]);
          }
        }
      }
    };
    int64_t p = wave;
    for (; (p + (kU - 1) * kFewWaves + 1) * 64 <= K; p += kU * kFewWaves) take(std::true_type{}, p);
    for (; p * 64 < K; p += kU * kFewWaves) take(std::false_type{}, p);
#pragma unroll
    for (int g = 0; g < RG; ++g) {
      float v = acc[g];
      v += dpp_move<0xB1>(v);              // lane ^ 1, ^ 2, mirror of 8
      v += dpp_move<0x4E>(v);
      v += dpp_move<0x141>(v);
      if ((lane & 7) == 0) red[wave][8 * g + (lane >> 3)] = v;
    }
    __syncthreads();
    if (threadIdx.x < 8 * RG) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kFewWaves; ++w) v += red[w][threadIdx.x];
      vs[threadIdx.x] = scales ? v * scales[id] : v;
    }
    __syncthreads();
    if (n < N) {
      const uint16_t* bl = b + ((int64_t)id * N + n) * r;
      float s = 0.0f;
#pragma unroll 4
      for (int j = 0; j < r; j += 8) {
        float w[8];
        load8<true>(bl, j, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = fmaf(vs[j + e], w[e], s);
      }
      y += s;
    }
  }
  if (n < N) {
    if (F32) ((float*)out)[t * ldo + n] = y;
    else ((uint16_t*)out)[t * ldo + n] = (uint16_t)bf16x2_rne(y, 0.0f);
  }
}

namespace {

// A launch's shape.  Many tokens (512): tiles of 64, the first product staged through LDS (lora_tiles_kernel, whose
// loads take whole lines), the sum over K cut so that about 512 workgroups run (operands from memory, 8192 tokens of 8
// runs, rank 64: 84 us, with 256 workgroups 85 to 94).  Fewer: tiles of 16, the sum cut into up to 32 chunks, a tile's
// adapters shared between workgroups.  The second product: 512 workgroups (8192 tokens of 8 runs, rank 64, replayed:
// 50 us; with 256 55, with 1024 53).
struct LoraPlan {
  int tile, chunk, chunks, parts;   // of the first product; workgroups that share a tile's adapters
  int tile2, cols;             // of the second
};

// Whether the one-launch kernel takes the call.  One of its workgroups fills a compute unit for about 1.5 us, the
// time that A takes at 65 bytes a nanosecond, and 0.053 us a rank for the rows of B, of which a lane has one; the two
// kernels take 10 to 20 us for the token counts in question (captured; the second launch and the workspace cost the
// host 4 us more).  Measured, one / two launches: 16 tokens of 16 requests, N 4096, K 7168, r 16 5.8 / 10.1 us, K 4096,
// r 64 12.8 / 12.7; 256 of 32, K 4096, r 16 16.7 / 21; 256 of 2, r 64 43 / 12; 512 of 8, r 16 29 / 13; 168 of 6,
// N 6104, K 104, r 64 25 / 17.
bool few_tokens(int64_t T, int32_t r, int64_t N, int64_t K) {
  if (T > 65535) return false;
  const int64_t rounds = (T * ((N + kFewThreads - 1) / kFewThreads) + 255) / 256;
  return (double)rounds * (1.5 + (double)r * ((double)K * 2.0 / 65000.0 + 0.053)) <= 18.0;
}

LoraPlan plan(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K) {
  LoraPlan p;
  p.tile = p.tile2 = T < 512 ? 16 : 64;
  auto distinct = [&](int64_t tile) {
    const int64_t n = T < tile ? T : tile;
    return n < L ? n : (int64_t)L;
  };
  const int64_t tiles = (T + p.tile - 1) / p.tile, spans = (K + kSpan - 1) / kSpan;
  int64_t per = (spans * tiles + 511) / 512;
  if (per < (spans + 31) / 32) per = (spans + 31) / 32;
  if (p.tile == 64 && per < 2) per = 2;                // (four stages at least)
  if (per > spans) per = spans;
  p.chunk = (int)per * kSpan;
  p.chunks = (int)((spans + per - 1) / per);
  // about one item a wave while there are compute units without a workgroup
  p.parts = (int)((distinct(p.tile) * per + kWaves - 1) / kWaves);
  const int64_t most = 256 / (tiles * p.chunks);
  if (p.parts > most) p.parts = most < 1 ? 1 : (int)most;

  const int64_t tiles2 = (T + p.tile2 - 1) / p.tile2, steps = (N + kCols - 1) / kCols;
  int64_t cols = (steps * tiles2 + 511) / 512;
  const int64_t least = (2 * kWaves + distinct(p.tile2) - 1) / distinct(p.tile2);
  if (T >= 512 && cols < least) cols = least;
  if (cols > steps) cols = steps;
  p.cols = (int)cols * kCols;
  return p;
}

#define FGG_LORA_SHRINK(rt) \
  {"lora_shrink_kernel<" #rt ">", "fgg_lora_add", 16, 16 * rt, kSpan, kThreads, 0, 0, kWaves * 16 * 17 * 4, \
   kWaves * 16 * 17 * 4, (const void*)lora_shrink_kernel<rt>}
#define FGG_LORA_EXPAND(tt, rs, f32, name) \
  {"lora_expand_kernel<" #tt "," #rs "," name ">", "fgg_lora_add", 16 * tt, kCols, 32 * rs, kThreads, 0, 0, \
   (f32 ? 3 : 2) * 16 * tt * (32 * rs + 8) * 2 + kRed(tt, rs), \
   (f32 ? 3 : 2) * 16 * tt * (32 * rs + 8) * 2 + kRed(tt, rs), (const void*)lora_expand_kernel<tt, rs, f32>}
#define FGG_LORA_FEW(rg, f32, name) \
  {"lora_few_kernel<" #rg "," name ">", "fgg_lora_add", 1, kFewThreads, 64, kFewThreads, 0, 0, \
   (kFewWaves + 1) * 8 * rg * 4, (kFewWaves + 1) * 8 * rg * 4, (const void*)lora_few_kernel<rg, f32>}
// (the runs' sums: only where a tile has fewer quads than threads)
constexpr int kRed(int tt, int rs) { return 16 * tt * 8 * rs < kThreads ? kThreads * 16 : 0; }

}  // namespace

const KernelInfo kInfoLora[kLoraForms] = {
    FGG_LORA_SHRINK(1), FGG_LORA_SHRINK(2), FGG_LORA_SHRINK(4), FGG_LORA_SHRINK(8),
    FGG_LORA_EXPAND(1, 1, false, "bf16"), FGG_LORA_EXPAND(1, 2, false, "bf16"), FGG_LORA_EXPAND(1, 4, false, "bf16"),
    FGG_LORA_EXPAND(1, 1, true, "f32"), FGG_LORA_EXPAND(1, 2, true, "f32"), FGG_LORA_EXPAND(1, 4, true, "f32"),
    FGG_LORA_EXPAND(4, 1, false, "bf16"), FGG_LORA_EXPAND(4, 2, false, "bf16"), FGG_LORA_EXPAND(4, 4, false, "bf16"),
    FGG_LORA_EXPAND(4, 1, true, "f32"), FGG_LORA_EXPAND(4, 2, true, "f32"), FGG_LORA_EXPAND(4, 4, true, "f32"),
    FGG_LORA_FEW(1, false, "bf16"), FGG_LORA_FEW(2, false, "bf16"), FGG_LORA_FEW(4, false, "bf16"),
    FGG_LORA_FEW(8, false, "bf16"), FGG_LORA_FEW(16, false, "bf16"), FGG_LORA_FEW(1, true, "f32"),
    FGG_LORA_FEW(2, true, "f32"), FGG_LORA_FEW(4, true, "f32"), FGG_LORA_FEW(8, true, "f32"),
    FGG_LORA_FEW(16, true, "f32"),
};

size_t lora_workspace_bytes(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K) {
  return T == 0 || few_tokens(T, r, N, K) ? 0 : (size_t)plan(T, L, r, N, K).chunks * (size_t)T * (size_t)r * 4;
}

hipError_t launch_lora(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                       const int32_t* ids, const uint16_t* a, const uint16_t* b, const float* scales, const void* base,
                       int64_t ldb, void* out, bool f32, int64_t ldo, float* ws, hipStream_t st) {
  const int ranks = r <= 16 ? 0 : r <= 32 ? 1 : r <= 64 ? 2 : 3;
  if (few_tokens(T, r, N, K)) {
    const dim3 grid((unsigned)((N + kFewThreads - 1) / kFewThreads), (unsigned)T);
    const int form = (f32 ? 5 : 0) + (r <= 8 ? 0 : ranks + 1);
    trace_launch(kInfoLora[16 + form], grid, "T=%lld L=%d r=%d N=%lld K=%lld", (long long)T, L, r, (long long)N,
                 (long long)K);
    auto few = [&](auto* kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kFewThreads), 0, st, x, ldx, ids, a, b, scales, base, ldb, out, ldo, L, r,
                         N, K);
    };
    switch (form) {
      case 0: few(lora_few_kernel<1, false>); break;
      case 1: few(lora_few_kernel<2, false>); break;
      case 2: few(lora_few_kernel<4, false>); break;
      case 3: few(lora_few_kernel<8, false>); break;
      case 4: few(lora_few_kernel<16, false>); break;
      case 5: few(lora_few_kernel<1, true>); break;
      case 6: few(lora_few_kernel<2, true>); break;
      case 7: few(lora_few_kernel<4, true>); break;
      case 8: few(lora_few_kernel<8, true>); break;
      default: few(lora_few_kernel<16, true>); break;
    }
    return hipGetLastError();
  }
  const LoraPlan p = plan(T, L, r, N, K);
  if (p.tile == 64) {
    const hipError_t e = launch_lora_tiles(T, L, r, K, x, ldx, ids, a, p.chunk, p.chunks, ws, st);
    if (e != hipSuccess) return e;
  } else {
    const dim3 grid((unsigned)((T + p.tile - 1) / p.tile), (unsigned)p.chunks, (unsigned)p.parts);
    trace_launch(kInfoLora[ranks], grid, "T=%lld L=%d r=%d K=%lld", (long long)T, L, r, (long long)K);
    auto shrink = [&](auto* kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, st, x, ldx, ids, a, T, L, r, K, p.chunk, ws);
    };
    switch (ranks) {
      case 0: shrink(lora_shrink_kernel<1>); break;
      case 1: shrink(lora_shrink_kernel<2>); break;
      case 2: shrink(lora_shrink_kernel<4>); break;
      default: shrink(lora_shrink_kernel<8>); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const dim3 g2((unsigned)((T + p.tile2 - 1) / p.tile2), (unsigned)((N + p.cols - 1) / p.cols));
  const int second = (p.tile2 == 16 ? 0 : 6) + (f32 ? 3 : 0) + (r <= 32 ? 0 : r <= 64 ? 1 : 2);
  trace_launch(kInfoLora[4 + second], g2, "T=%lld L=%d r=%d N=%lld", (long long)T, L, r, (long long)N);
  auto expand = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, g2, dim3(kThreads), 0, st, ws, p.chunks, ids, b, scales, base, ldb, out, ldo, T, L, r,
                       N, p.cols);
  };
  switch (second) {
    case 0: expand(lora_expand_kernel<1, 1, false>); break;
    case 1: expand(lora_expand_kernel<1, 2, false>); break;
    case 2: expand(lora_expand_kernel<1, 4, false>); break;
    case 3: expand(lora_expand_kernel<1, 1, true>); break;
    case 4: expand(lora_expand_kernel<1, 2, true>); break;
    case 5: expand(lora_expand_kernel<1, 4, true>); break;
    case 6: expand(lora_expand_kernel<4, 1, false>); break;
    case 7: expand(lora_expand_kernel<4, 2, false>); break;
    case 8: expand(lora_expand_kernel<4, 4, false>); break;
    case 9: expand(lora_expand_kernel<4, 1, true>); break;
    case 10: expand(lora_expand_kernel<4, 2, true>); break;
    default: expand(lora_expand_kernel<4, 4, true>); break;
  }
  return hipGetLastError();
}

}  // namespace fgg
