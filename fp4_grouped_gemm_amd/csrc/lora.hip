// Low-rank adapters of many requests beside one shared projection (gfx950):
//
//   out[t] = base[t] + scales[i] (x[t] A_i^T) B_i^T,   i = ids[t];   out[t] = base[t] without an adapter
//
// Two kernels: x A^T into fp32 sums per token (the sum over K cut into chunks, one workgroup and
// tile of tokens each), and the product with B on top of base.  What bounds them is memory: every
// adapter's factors once, x, base and out.
//
//  * tokens come in any order, in tiles of 16 or 64.  A wave finds the tile's distinct adapters by
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

namespace fgg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kSpan = 128;               // of the sum over K per item
constexpr int kCols = 32;                // columns per item of the second product
constexpr int kMaxRank = 128;
constexpr int kVRow = kMaxRank + 8;      // a token's row in LDS, in bf16 elements (16 bytes past a multiple of the banks)

__device__ inline v8bf load_or_zero(const uint16_t* p, bool on) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (on) u = *reinterpret_cast<const uint4*>(p);
  return __builtin_bit_cast(v8bf, u);
}

// The lane's token's adapter, -1 where it has none (or there is no token).
__device__ inline int lane_adapter(const int32_t* ids, int64_t t0, int tokens, int64_t T, int L, int lane) {
  int id = -1;
  if (lane < tokens && t0 + lane < T) id = ids[t0 + lane];
  return id >= 0 && id < L ? id : -1;
}

}  // namespace

// part[chunk][t][j] = sum over the chunk's k of x[t][k] A[ids[t]][j][k];  TT tiles of 16 tokens, RT of 16 ranks.
template <int TT, int RT>
__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const uint16_t* __restrict__ x, int64_t ldx,
                                                               const int32_t* __restrict__ ids,
                                                               const uint16_t* __restrict__ a, int64_t T, int L, int r,
                                                               int64_t K, int chunk, float* __restrict__ part) {
  __shared__ float red[kWaves][16 * TT][16 + 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int64_t k0 = (int64_t)blockIdx.y * chunk, k1 = k0 + chunk < K ? k0 + chunk : K;
  const int id = lane_adapter(ids, t0, 16 * TT, T, L, lane);

  v4f sum[RT][TT];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int f = 0; f < TT; ++f) sum[i][f] = v4f{0.f, 0.f, 0.f, 0.f};

  int item = 0;
  for (uint64_t left = __ballot(id >= 0); left;) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t match = __ballot(id == cur);
    left &= ~match;
    const uint16_t* mine = a + (int64_t)cur * r * K;
    for (int64_t k = k0; k < k1; k += kSpan) {
      if ((item++ & (kWaves - 1)) != wave) continue;
      v8bf xf[TT][kSpan / 32];
#pragma unroll
      for (int f = 0; f < TT; ++f)
#pragma unroll
        for (int s = 0; s < kSpan / 32; ++s) {
          const int64_t at = k + 32 * s + 8 * q;
          const bool on = (match >> (16 * f + l16) & 1) && at < k1;
          xf[f][s] = load_or_zero(x + (t0 + 16 * f + l16) * ldx + at, on);
        }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        v8bf af[kSpan / 32];
#pragma unroll
        for (int s = 0; s < kSpan / 32; ++s) {
          const int64_t at = k + 32 * s + 8 * q;
          const int row = 16 * i + l16;
          af[s] = load_or_zero(mine + (int64_t)row * K + at, row < r && at < k1);
        }
#pragma unroll
        for (int f = 0; f < TT; ++f) {
          v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int s = 0; s < kSpan / 32; ++s) d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[s], xf[f][s], d, 0, 0, 0);
          const bool on = match >> (16 * f + l16) & 1;
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[i][f][e] += on ? d[e] : 0.0f;
        }
      }
    }
  }

  // the eight waves' sums, in their order
  for (int i = 0; i < RT && 16 * i < r; ++i) {
    v4f s[TT];
#pragma unroll
    for (int j = 0; j < RT; ++j)
      if (j == i) {
#pragma unroll
        for (int f = 0; f < TT; ++f) s[f] = sum[j][f];
      }
#pragma unroll
    for (int f = 0; f < TT; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) red[wave][16 * f + l16][4 * q + e] = s[f][e];
    __syncthreads();
    for (int v = threadIdx.x; v < 256 * TT; v += kThreads) {
      const int t = v >> 4, j = v & 15;
      float total = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) total += red[w][t][j];
      if (t0 + t < T && 16 * i + j < r) part[((int64_t)blockIdx.y * T + t0 + t) * r + 16 * i + j] = total;
    }
    __syncthreads();
  }
}

// out[t][n] = base[t][n] + sum_j v[t][j] B[ids[t]][n][j],  v = scales[ids[t]] times the chunks' sums.
template <int TT, bool F32>
__global__ void __launch_bounds__(kThreads) lora_expand_kernel(const float* __restrict__ part, int chunks,
                                                               const int32_t* __restrict__ ids,
                                                               const uint16_t* __restrict__ b,
                                                               const float* __restrict__ scales, const void* base,
                                                               int64_t ldb, void* out, int64_t ldo, int64_t T, int L,
                                                               int r, int64_t N, int cols) {
  constexpr int kParts = F32 ? 3 : 2;
  __shared__ __align__(16) uint16_t vs[kParts][16 * TT][kVRow];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.x * (16 * TT);
  const int64_t n_from = (int64_t)blockIdx.y * cols, n_to = n_from + cols < N ? n_from + cols : N;
  const int id = lane_adapter(ids, t0, 16 * TT, T, L, lane);

  // a token's low-rank sums in bf16 parts, zeros past the rank
  const int wide = (r + 31) & ~31;
  for (int v = threadIdx.x; v < 16 * TT * wide; v += kThreads) {
    const int t = v / wide, j = v - t * wide;
    float s = 0.0f;
    if (t0 + t < T && j < r) {
      const int i = ids[t0 + t];
      if (i >= 0 && i < L) {
        for (int c = 0; c < chunks; ++c) s += part[((int64_t)c * T + t0 + t) * r + j];
        if (scales) s *= scales[i];
      }
    }
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const uint16_t bits = (uint16_t)bf16x2_rne(s, 0.0f);
      vs[p][t][j] = bits;
      // (an infinite or NaN part carries the whole)
      const float v0 = bf16_to_f32(bits);
      s = fabsf(v0) < INFINITY ? s - v0 : 0.0f;
    }
  }
  __syncthreads();

  int item = 0;
  auto columns = [&](int cur, uint64_t match) {
    for (int64_t n0 = n_from; n0 < n_to; n0 += kCols) {
      if ((item++ & (kWaves - 1)) != wave) continue;
      // rows of two fragments are dealt so that a lane's results are eight consecutive columns
      v8bf bf[2][kMaxRank / 32];
      if (cur >= 0) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
          for (int s = 0; s < kMaxRank / 32; ++s) {
            if (32 * s >= r) break;
            const int64_t n = n0 + 8 * (l16 >> 2) + 4 * f + (l16 & 3);
            const int j = 32 * s + 8 * q;
            bf[f][s] = load_or_zero(b + ((int64_t)cur * N + n) * r + j, n < n_to && j < r);
          }
      }
#pragma unroll
      for (int f = 0; f < TT; ++f) {
        if ((match >> (16 * f) & 0xFFFF) == 0) continue;
        const int64_t t = t0 + 16 * f + l16, n = n0 + 8 * q;
        const bool on = (match >> (16 * f + l16) & 1) && n < n_to;
        float y[8];
        if (on) load8<!F32>(base, t * ldb + n, y);
        if (cur >= 0) {
          v4f d[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int s = 0; s < kMaxRank / 32; ++s) {
            if (32 * s >= r) break;
#pragma unroll
            for (int p = kParts - 1; p >= 0; --p) {
              const v8bf v = *reinterpret_cast<const v8bf*>(&vs[p][16 * f + l16][32 * s + 8 * q]);
              d[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[0][s], v, d[0], 0, 0, 0);
              d[1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[1][s], v, d[1], 0, 0, 0);
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] += d[e >> 2][e & 3];
        }
        if (on) {
          if constexpr (F32) {
            float4* o = reinterpret_cast<float4*>((float*)out + t * ldo + n);
            o[0] = make_float4(y[0], y[1], y[2], y[3]);
            o[1] = make_float4(y[4], y[5], y[6], y[7]);
          } else {
            *reinterpret_cast<uint4*>((uint16_t*)out + t * ldo + n) =
                make_uint4(bf16x2_rne(y[0], y[1]), bf16x2_rne(y[2], y[3]), bf16x2_rne(y[4], y[5]),
                           bf16x2_rne(y[6], y[7]));
          }
        }
      }
    }
  };
  for (uint64_t left = __ballot(id >= 0); left;) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t match = __ballot(id == cur);
    left &= ~match;
    columns(cur, match);
  }
  if (out != base) {
    const uint64_t none = __ballot(id < 0 && lane < 16 * TT && t0 + lane < T);
    if (none) columns(-1, none);
  }
}

namespace {

// A launch's shape.  Tiles of 64 tokens read each factor a quarter as often where tokens share them (32 over rank
// 64, whose sums would not fit the registers).  The sum over K is cut so that few tokens still give every
// compute unit loads to wait for.
struct LoraPlan {
  int tile, chunk, chunks;
};

LoraPlan plan(int64_t T, int32_t L, int32_t r, int64_t K) {
  LoraPlan p;
  p.tile = T < 512 ? 16 : r <= 64 ? 64 : 32;
  const int64_t tiles = (T + p.tile - 1) / p.tile;
  const int64_t spans = (K + kSpan - 1) / kSpan;
  const int64_t adapters = T < L ? (T < p.tile ? T : p.tile) : (L < p.tile ? L : p.tile);
  // two items a wave, as long as there are fewer workgroups than 512
  int64_t per = (2 * kWaves + adapters - 1) / adapters;
  const int64_t fill = (spans * tiles + 511) / 512;
  if (per < fill) per = fill;
  if (per > spans) per = spans;
  while ((spans + per - 1) / per > 32) ++per;
  p.chunk = (int)per * kSpan;
  p.chunks = (int)((spans + per - 1) / per);
  return p;
}

#define FGG_LORA_SHRINK(tt, rt) \
  {"lora_shrink_kernel<" #tt "," #rt ">", "fgg_lora_add", 16 * tt, 16 * rt, kSpan, kThreads, 0, 0, \
   kWaves * 16 * tt * 17 * 4, kWaves * 16 * tt * 17 * 4, (const void*)lora_shrink_kernel<tt, rt>}
#define FGG_LORA_EXPAND(tt, f32, name) \
  {"lora_expand_kernel<" #tt "," name ">", "fgg_lora_add", 16 * tt, kCols, kMaxRank, kThreads, 0, 0, \
   (f32 ? 3 : 2) * 16 * tt * kVRow * 2, (f32 ? 3 : 2) * 16 * tt * kVRow * 2, (const void*)lora_expand_kernel<tt, f32>}

}  // namespace

const KernelInfo kInfoLora[kLoraForms] = {
    FGG_LORA_SHRINK(1, 1), FGG_LORA_SHRINK(1, 2), FGG_LORA_SHRINK(1, 4), FGG_LORA_SHRINK(1, 8),
    FGG_LORA_SHRINK(4, 1), FGG_LORA_SHRINK(4, 2), FGG_LORA_SHRINK(4, 4), FGG_LORA_SHRINK(2, 8),
    FGG_LORA_EXPAND(1, false, "bf16"), FGG_LORA_EXPAND(1, true, "f32"), FGG_LORA_EXPAND(2, false, "bf16"),
    FGG_LORA_EXPAND(2, true, "f32"), FGG_LORA_EXPAND(4, false, "bf16"), FGG_LORA_EXPAND(4, true, "f32"),
};

size_t lora_workspace_bytes(int64_t T, int32_t L, int32_t r, int64_t K) {
  return T == 0 ? 0 : (size_t)plan(T, L, r, K).chunks * (size_t)T * (size_t)r * 4;
}

hipError_t launch_lora(int64_t T, int32_t L, int32_t r, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                       const int32_t* ids, const uint16_t* a, const uint16_t* b, const float* scales, const void* base,
                       int64_t ldb, void* out, bool f32, int64_t ldo, float* ws, hipStream_t st) {
  const LoraPlan p = plan(T, L, r, K);
  const unsigned tiles = (unsigned)((T + p.tile - 1) / p.tile);
  const bool wide = p.tile > 16;
  const int ranks = r <= 16 ? 0 : r <= 32 ? 1 : r <= 64 ? 2 : 3;
  const dim3 g1(tiles, (unsigned)p.chunks);
  trace_launch(kInfoLora[(wide ? 4 : 0) + ranks], g1, "T=%lld L=%d r=%d K=%lld", (long long)T, L, r, (long long)K);
  auto shrink = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, g1, dim3(kThreads), 0, st, x, ldx, ids, a, T, L, r, K, p.chunk, ws);
  };
  switch ((wide ? 4 : 0) + ranks) {
    case 0: shrink(lora_shrink_kernel<1, 1>); break;
    case 1: shrink(lora_shrink_kernel<1, 2>); break;
    case 2: shrink(lora_shrink_kernel<1, 4>); break;
    case 3: shrink(lora_shrink_kernel<1, 8>); break;
    case 4: shrink(lora_shrink_kernel<4, 1>); break;
    case 5: shrink(lora_shrink_kernel<4, 2>); break;
    case 6: shrink(lora_shrink_kernel<4, 4>); break;
    default: shrink(lora_shrink_kernel<2, 8>); break;
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // columns of a workgroup: about 1024 workgroups, at least one item a wave where one adapter takes the tile
  int64_t steps = (N + kCols - 1) / kCols;
  int64_t per = (steps * tiles + 1023) / 1024;
  const int64_t adapters = T < L ? (T < p.tile ? T : p.tile) : (L < p.tile ? L : p.tile);
  const int64_t least = (kWaves + adapters - 1) / adapters;
  if (per < least) per = least;
  if (per > steps) per = steps;
  const dim3 g2(tiles, (unsigned)((steps + per - 1) / per));
  trace_launch(kInfoLora[8 + (p.tile >> 5) * 2 + (f32 ? 1 : 0)], g2, "T=%lld L=%d r=%d N=%lld", (long long)T, L, r,
               (long long)N);
  auto expand = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, g2, dim3(kThreads), 0, st, ws, p.chunks, ids, b, scales, base, ldb, out, ldo, T, L, r,
                       N, (int)per * kCols);
  };
  if (p.tile == 64) f32 ? expand(lora_expand_kernel<4, true>) : expand(lora_expand_kernel<4, false>);
  else if (p.tile == 32) f32 ? expand(lora_expand_kernel<2, true>) : expand(lora_expand_kernel<2, false>);
  else f32 ? expand(lora_expand_kernel<1, true>) : expand(lora_expand_kernel<1, false>);
  return hipGetLastError();
}

}  // namespace fgg
