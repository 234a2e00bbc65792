// Few tokens times 4-bit expert weights, activations unquantized: the generation step's
// form of the experts' products.
//
//   y[t, j][n] = sum_K x[t (, j)][K] * B[e][n][K],   e = topk_ids[t][j],
//   B = E2M1 code * 2^(scale byte - 127), one scale byte per 32 along K
//
// plain (y per slot), with SiLU(gate)*up (B holds [gate | up] rows), or summed over the
// token's slots with the gate weights.
//
// Bound by the weights' bytes: every distinct expert of up to 16 tokens is read once, whatever
// number of them chose it.  An E2M1 code times a power of two is a bf16 number, so the weights
// go through v_cvt_scalef32_pk_bf16_fp4 (two codes and their scale per instruction) into the
// bf16 matrix instruction 16x16x32 with 16 weight rows as its rows and the tokens as its
// columns: products are exact, sums in fp32.  One 16-byte load per lane (row lane % 16, 32
// consecutive K at 32 * (lane / 16): one scale) feeds four of them; K runs through the
// instructions in that order on both operands.  fp32 activations are split into three bf16 parts
// (8 + 8 + 8 bits, exact) and take three instructions.
//
// A workgroup owns a tile of weight rows; its eight waves split the K blocks (of every expert,
// in the summed form) and their partial sums are joined through LDS in a fixed order, so no
// result depends on the order of arrival.  Tokens are columns: the experts to visit are the
// distinct ids among the tokens' slots, found per workgroup by an LDS table of first
// occurrences; a token that names one expert twice has its second slot visited on its own.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"

namespace fgg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kMaxPairs = 1024;    // 16 tokens x 64 slots
constexpr int kMaxGroups = 1024;

enum { kPlain = 0, kSilu = 1, kSum = 2 };

struct GemvArgs {
  int G;
  int64_t T;
  int k;
  int64_t N, K;          // N: output columns (the weights have 2N rows in the SiLU form)
  const void* x;
  int64_t ldx;
  int per_slot;          // x rows are t * k + j (else t)
  const uint8_t* b;
  const uint8_t* s;
  const int32_t* ids;    // null: one set of weights, every token
  const float* w;
  void* out;
  int64_t ldo;
};

// Four codes pairs of one 32-bit word, times 2^(byte - 127), as eight bf16.
__device__ inline bf16x8 dequant8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// The 32 activations of a lane's K chunk: four operands of eight bf16 (per part).
template <class TX>
struct Frag;
template <>
struct Frag<uint16_t> {
  u32x4 v[4];
  __device__ void load(const uint16_t* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const u32x4_a2*>(p + 8 * i);
  }
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = u32x4{0, 0, 0, 0};
  }
  __device__ v4f mul(int i, bf16x8 a, v4f acc) const {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, v[i]), acc, 0, 0, 0);
  }
};
template <>
struct Frag<float> {
  u32x4 v[8];
  __device__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4_a4*>(p + 4 * i);
  }
  __device__ void clear() {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = u32x4{0, 0, 0, 0};
  }
  // x = hi + mid + lo: the top 16 bits, then the top 16 bits of each exact remainder
  __device__ v4f mul(int i, bf16x8 a, v4f acc) const {
    u32x4 part[3];
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      uint32_t h[3][2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t u = v[2 * i + (d >> 1)][2 * (d & 1) + e];
        const float f = __uint_as_float(u);
        const bool finite = (u & 0x7F800000u) != 0x7F800000u;
        const bool nan = !finite && (u & 0x007FFFFFu) != 0;
        h[0][e] = nan ? 0x7FC00000u : u & 0xFFFF0000u;
        const float r = finite ? f - __uint_as_float(h[0][e]) : 0.0f;
        h[1][e] = __float_as_uint(r) & 0xFFFF0000u;
        h[2][e] = __float_as_uint(r - __uint_as_float(h[1][e]));
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) part[q][d] = (h[q][0] >> 16) | (h[q][1] & 0xFFFF0000u);
    }
#pragma unroll
    for (int q = 2; q >= 0; --q)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, part[q]), acc, 0, 0, 0);
    return acc;
  }
};

__device__ inline void put(uint16_t* p, float v) { *p = bf16_bits_rne(v); }
__device__ inline void put(float* p, float v) { *p = v; }

// Which experts a workgroup visits for its tokens.
struct Items {
  int ids[kMaxPairs];        // expert of each pair, -1: none
  int first[kMaxGroups];     // lowest pair that names the expert (as a first occurrence in its token)
  uint16_t item[kMaxPairs];  // the pairs that stand for one visit each, in increasing order
  uint8_t again[kMaxPairs];  // the pair's expert is named by an earlier slot of its token
  int count[2 * kWaves];
};

// Builds the list for tokens [t0, t0 + Tn); returns the number of visits.  All threads call it.
__device__ inline int list_items(Items& L, const int32_t* ids, int64_t t0, int Tn, int k, int G) {
  const int tid = threadIdx.x, P = Tn * k;
  for (int i = tid; i < G; i += 64 * kWaves) L.first[i] = 0x7FFFFFFF;
  for (int p = tid; p < P; p += 64 * kWaves) {
    const int e = ids[t0 * k + p];
    L.ids[p] = (e >= 0 && e < G) ? e : -1;
  }
  __syncthreads();
  for (int p = tid; p < P; p += 64 * kWaves) {
    const int e = L.ids[p];
    bool again = false;
    for (int q = p / k * k; q < p; ++q) again |= L.ids[q] == e;
    L.again[p] = again;
    if (e >= 0 && !again) atomicMin(&L.first[e], p);
  }
  __syncthreads();
  bool lead[2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int p = c * 64 * kWaves + tid;
    const int e = p < P ? L.ids[p] : -1;
    lead[c] = e >= 0 && (L.again[p] || L.first[e] == p);
    const uint64_t m = __ballot(lead[c]);
    if ((tid & 63) == 0) L.count[c * kWaves + (tid >> 6)] = __popcll(m);
  }
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint64_t m = __ballot(lead[c]);
    int before = 0;
    for (int i = 0; i < c * kWaves + (tid >> 6); ++i) before += L.count[i];
    if (lead[c]) L.item[before + __popcll(m & ((1ull << (tid & 63)) - 1))] = (uint16_t)(c * 64 * kWaves + tid);
  }
  for (int i = 0; i < 2 * kWaves; ++i) total += L.count[i];
  __syncthreads();
  return total;
}

// The slot of token `t` (of the workgroup's) that visit `p0` serves, -1: none.
__device__ inline int slot_of(const Items& L, int p0, int t, int Tn, int k) {
  const int e = L.ids[p0];
  if (L.again[p0]) return p0 / k == t ? p0 % k : -1;
  if (t >= Tn) return -1;
  for (int j = 0; j < k; ++j)
    if (L.ids[t * k + j] == e) return j;
  return -1;
}

// One wave's share: K blocks [kb0, kb1) of NT row tiles of one expert, added to acc.
// xrow: the lane's token row (null: no token in this column).
template <class TX, bool TILED, int NT, int U>
__device__ inline void gemv_run(const uint8_t* const (&wp)[NT], const uint8_t* const (&sp)[NT], const TX* xrow,
                                int64_t K, int kb0, int kb1, v4f (&acc)[NT]) {
  const int lane = threadIdx.x & 63, c = lane >> 4;
  for (int kb = kb0; kb < kb1; kb += U) {
    u32x4 q[U][NT];
    uint32_t e[U][NT];
    Frag<TX> f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = kb + u < kb1 && (int64_t)(kb + u) * 128 + 32 * c < K;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        q[u][i] = u32x4{0, 0, 0, 0};
        e[u][i] = 127;
        if (in) {
          if constexpr (TILED) {
            q[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[i] + (int64_t)(kb + u) * 1024));
            e[u][i] = sp[i][(int64_t)((kb + u) >> 2) * 256 + 4 * ((kb + u) & 3)];
          } else {
            q[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[i] + (int64_t)(kb + u) * 64));
            e[u][i] = sp[i][(int64_t)(kb + u) * 4];
          }
        }
      }
      if (in && xrow) f[u].load(xrow + (int64_t)(kb + u) * 128);
      else f[u].clear();
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const float scale = __uint_as_float(e[u][i] << 23);
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[i] = f[u].mul(d, dequant8(q[u][i][d], scale), acc[i]);
      }
  }
}

}  // namespace

template <int MODE, bool TILED, class TX, class TO, int RT>
__global__ void __launch_bounds__(64 * kWaves) gemv_fp4_kernel(GemvArgs a) {
  constexpr int NT = MODE == kSilu ? 2 * RT : RT;    // row tiles: RT of gate, then RT of up
  constexpr int U = sizeof(TX) == 2 ? 4 : 2;
  __shared__ Items L;
  __shared__ float part[kWaves][NT][16][16];         // [wave][tile][token][row]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, c = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * RT;
  const int64_t t0 = (int64_t)blockIdx.z * 16;
  const int Tn = a.T - t0 < 16 ? (int)(a.T - t0) : 16;
  const int64_t width = MODE == kSilu ? 2 * a.N : a.N, nkb = (a.K + 127) / 128;
  const TX* x = (const TX*)a.x;
  TO* out = (TO*)a.out;

  const int items = a.ids ? list_items(L, a.ids, t0, Tn, a.k, a.G) : 1;

  // weight and scale pointers of this lane in row tile i of expert e
  const uint8_t* wp[NT];
  const uint8_t* sp[NT];
  auto at_expert = [&](int e) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int64_t r0 = n0 + 16 * (i % RT);
      if constexpr (TILED) {
        const int64_t last = a.N / 16 - 1;
        int64_t nb = r0 / 16 < last ? r0 / 16 : last;
        if (i >= RT) nb += a.N / 16;
        wp[i] = a.b + ((int64_t)e * (width / 16) + nb) * (a.K / 128) * 1024 + 16 * lane;
        sp[i] = a.s + ((int64_t)e * (width / 16) + nb) * ((a.K + 511) / 512) * 256 + 16 * col + c;
      } else {
        int64_t n = r0 + col < a.N ? r0 + col : a.N - 1;   // rows past the end: any row, not stored
        if (i >= RT) n += a.N;
        wp[i] = a.b + ((int64_t)e * width + n) * (a.K / 2) + 16 * c;
        sp[i] = a.s + ((int64_t)e * width + n) * (a.K / 32) + c;
      }
    }
  };
  auto row_of = [&](int j) -> const TX* {
    if (j < 0) return nullptr;
    return x + (a.per_slot ? (t0 + col) * a.k + j : t0 + col) * a.ldx + 32 * c;
  };
  // the sum over the waves of one value, in wave order
  auto joined = [&](int i, int t, int r) {
    float v = part[0][i][t][r];
#pragma unroll
    for (int q = 1; q < kWaves; ++q) v += part[q][i][t][r];
    return v;
  };
  auto publish = [&](const v4f (&acc)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<v4f*>(&part[wave][i][col][4 * c]) = acc[i];
  };

  if constexpr (MODE == kSum) {
    // the waves split the K blocks of all visits, expert by expert
    const int64_t units = (int64_t)items * nkb;
    int64_t at = units * wave / kWaves;
    const int64_t end = units * (wave + 1) / kWaves;
    v4f total[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) total[i] = v4f{0, 0, 0, 0};
    while (at < end) {
      const int it = (int)(at / nkb), kb0 = (int)(at - it * nkb);
      const int kb1 = (int)(end - it * nkb < nkb ? end - it * nkb : nkb);
      const int p0 = L.item[it], j = slot_of(L, p0, col, Tn, a.k);
      v4f acc[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = v4f{0, 0, 0, 0};
      at_expert(L.ids[p0]);
      gemv_run<TX, TILED, NT, U>(wp, sp, row_of(j), a.K, kb0, kb1, acc);
      if (j >= 0) {
        const float g = a.w[(t0 + col) * a.k + j];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) total[i][r] = fmaf(g, acc[i][r], total[i][r]);
      }
      at += kb1 - kb0;
    }
    publish(total);
    __syncthreads();
    for (int i = tid; i < RT * 256; i += 64 * kWaves) {
      const int t = (i >> 4) & 15, r = i & 15;
      const int64_t n = n0 + 16 * (i >> 8) + r;
      if (t < Tn && n < a.N) put(out + (t0 + t) * a.ldo + n, joined(i >> 8, t, r));
    }
  } else {
    const int kb0 = (int)(nkb * wave / kWaves), kb1 = (int)(nkb * (wave + 1) / kWaves);
    for (int it = blockIdx.y; it < items; it += gridDim.y) {
      int j, p0 = 0;
      if (a.ids) {
        p0 = L.item[it];
        j = slot_of(L, p0, col, Tn, a.k);
      } else {
        j = col < Tn ? 0 : -1;
      }
      v4f acc[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) acc[i] = v4f{0, 0, 0, 0};
      at_expert(a.ids ? L.ids[p0] : 0);
      gemv_run<TX, TILED, NT, U>(wp, sp, row_of(j), a.K, kb0, kb1, acc);
      publish(acc);
      __syncthreads();
      for (int i = tid; i < RT * 256; i += 64 * kWaves) {
        const int t = (i >> 4) & 15, r = i & 15;
        const int64_t n = n0 + 16 * (i >> 8) + r;
        const int jt = a.ids ? slot_of(L, p0, t, Tn, a.k) : (t < Tn ? 0 : -1);
        if (jt < 0 || n >= a.N) continue;
        float v = joined(i >> 8, t, r);
        if constexpr (MODE == kSilu) v = v / (1.0f + expf(-v)) * joined(RT + (i >> 8), t, r);
        put(out + ((t0 + t) * a.k + jt) * a.ldo + n, v);
      }
      __syncthreads();
    }
    if (a.ids && blockIdx.y == 0) {                  // slots without an expert
      for (int p = tid >> 4; p < Tn * a.k; p += 4 * kWaves) {
        if (L.ids[p] >= 0) continue;
        for (int r = tid & 15; r < 16 * RT; r += 16)
          if (n0 + r < a.N) put(out + (t0 * a.k + p) * a.ldo + n0 + r, 0.0f);
      }
    }
  }
}

static constexpr int gemv_lds(int nt) { return (int)sizeof(Items) + kWaves * nt * 1024; }
const KernelInfo kInfoGemvFp4 = {"gemv_fp4_kernel", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kWaves, 0, 0, gemv_lds(1),
                                 gemv_lds(1), (const void*)gemv_fp4_kernel<kPlain, true, uint16_t, uint16_t, 1>};
const KernelInfo kInfoGemvFp4Silu = {"gemv_fp4_kernel<silu>", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kWaves, 0, 0,
                                     gemv_lds(2), gemv_lds(2),
                                     (const void*)gemv_fp4_kernel<kSilu, true, uint16_t, uint16_t, 1>};
const KernelInfo kInfoGemvFp4Sum = {"gemv_fp4_kernel<sum>", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kWaves, 0, 0,
                                    gemv_lds(1), gemv_lds(1),
                                    (const void*)gemv_fp4_kernel<kSum, true, uint16_t, uint16_t, 1>};

hipError_t launch_gemv_fp4(bool tiled, int32_t G, int64_t T, int32_t k, int64_t N, int64_t K, const void* x,
                           bool x_bf16, int64_t ldx, bool per_slot, const uint8_t* b, const uint8_t* s,
                           const int32_t* ids, const float* w, bool silu, void* out, bool out_bf16, int64_t ldo,
                           hipStream_t st) {
  const GemvArgs a = {G, T, k, N, K, x, ldx, per_slot, b, s, ids, w, out, ldo};
  const int64_t pairs = (T < 16 ? T : 16) * k;
  const unsigned visits = ids && !w ? (unsigned)(pairs < G ? pairs : G) : 1;
  const dim3 grid((unsigned)((N + 15) / 16), visits, (unsigned)((T + 15) / 16));
  const KernelInfo& info = w ? kInfoGemvFp4Sum : silu ? kInfoGemvFp4Silu : kInfoGemvFp4;
  trace_launch(info, grid, "G=%d T=%lld k=%d N=%lld K=%lld %s %s->%s", (int)G, (long long)T, (int)k, (long long)N,
               (long long)K, tiled ? "tiled" : "rows", x_bf16 ? "bf16" : "fp32", out_bf16 ? "bf16" : "fp32");
  auto go = [&](auto mode, auto til, auto tx, auto to) {
    using TX = decltype(tx);
    using TO = decltype(to);
    hipLaunchKernelGGL((gemv_fp4_kernel<decltype(mode)::value, decltype(til)::value, TX, TO, 1>), grid,
                       dim3(64 * kWaves), 0, st, a);
  };
  auto with_types = [&](auto mode, auto til) {
    if (x_bf16 && out_bf16) go(mode, til, uint16_t(), uint16_t());
    else if (x_bf16) go(mode, til, uint16_t(), float());
    else if (out_bf16) go(mode, til, float(), uint16_t());
    else go(mode, til, float(), float());
  };
  auto with_mode = [&](auto til) {
    if (w) with_types(std::integral_constant<int, kSum>(), til);
    else if (silu) with_types(std::integral_constant<int, kSilu>(), til);
    else with_types(std::integral_constant<int, kPlain>(), til);
  };
  if (tiled) with_mode(std::true_type());
  else with_mode(std::false_type());
  return hipGetLastError();
}

}  // namespace fgg
