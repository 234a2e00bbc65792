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
#include "fgg_wave.hpp"

namespace fgg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_a1 __attribute__((aligned(1)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxWaves = 8;
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
  int out_bf16;
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

// Activations of one K block for up to NC tokens (4, 8 or 16).  The matrix instruction has 16
// columns and a K block takes four of them (operand d: elements 8d .. 8d + 7 of each lane's 32).
// With few tokens the columns hold several operands at once: column NC * i + t holds token t's
// operand s * F + i of register set s (F = 16 / NC operands per set), so a K block takes NC / 4
// 16-byte loads per lane instead of four.  Instruction d multiplies set d / F into accumulator
// d % F, of which only columns NC * (d % F) + t mean anything: those are picked at the end.
template <class TX, int NC>
struct Frag;
template <int NC>
struct Frag<uint16_t, NC> {
  static constexpr int F = 16 / NC;
  u32x4 v[NC / 4];
  __device__ void load(const uint16_t* p) {
#pragma unroll
    for (int s = 0; s < NC / 4; ++s) v[s] = *reinterpret_cast<const u32x4_a2*>(p + 8 * F * s);
  }
  __device__ void clear() {
#pragma unroll
    for (int s = 0; s < NC / 4; ++s) v[s] = u32x4{0, 0, 0, 0};
  }
  __device__ void mul(int d, bf16x8 a, v4f (&acc)[F]) const {
    acc[d % F] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, v[d / F]), acc[d % F], 0, 0, 0);
  }
};
template <>
struct Frag<float, 16> {
  static constexpr int F = 1;
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
  __device__ void mul(int i, bf16x8 a, v4f (&acc)[1]) const {
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
      acc[0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, part[q]), acc[0], 0, 0, 0);
  }
};

__device__ inline void put(void* out, bool bf16, int64_t i, float v) {
  if (bf16) ((uint16_t*)out)[i] = bf16_bits_rne(v);
  else ((float*)out)[i] = v;
}

// Which experts a workgroup visits for its tokens.
struct Items {
  int ids[kMaxPairs];        // expert of each pair, -1: none
  int first[kMaxGroups];     // lowest pair that names the expert (as a first occurrence in its token)
  uint16_t item[kMaxPairs];  // the pairs that stand for one visit each, in increasing order
  uint8_t again[kMaxPairs];  // the pair's expert is named by an earlier slot of its token
  int count[kMaxWaves];
  uint16_t column[kMaxWaves][16];   // each wave's visit: token + 16 * slot of each column in use
};

// The list of at most 64 pairs, by each wave on its own: lane p holds pair p and looks at the
// pairs before it one by one.  Every wave writes the same values to LDS and reads only what it
// wrote itself, so there is no barrier.
__device__ inline int list_few_items(Items& L, const int32_t* ids, int64_t t0, int P, int k, int G) {
  const int p = threadIdx.x & 63, t = p / k;
  int e = p < P ? ids[t0 * k + p] : -1;
  if (e < 0 || e >= G) e = -1;
  int again = 0, covered = 0;
  for (int q = 0; q + 1 < P; ++q) {
    const int eq = __builtin_amdgcn_readlane(e, q), aq = __builtin_amdgcn_readlane(again, q);
    if (p > q && e == eq) {
      if (t == q / k) again = 1;
      else if (!aq) covered = 1;
    }
  }
  const bool lead = e >= 0 && (again || !covered);
  const uint64_t m = __ballot(lead);
  if (p < P) {
    L.ids[p] = e;
    L.again[p] = (uint8_t)again;
    if (lead) L.item[__popcll(m & ((1ull << p) - 1))] = (uint16_t)p;
  }
  return __popcll(m);
}

// Builds the list for tokens [t0, t0 + Tn); returns the number of visits.  All threads call it.
__device__ inline int list_items(Items& L, const int32_t* ids, int64_t t0, int Tn, int k, int G) {
  const int tid = threadIdx.x, P = Tn * k, threads = blockDim.x;
  for (int i = tid; i < G; i += threads) L.first[i] = 0x7FFFFFFF;
  for (int p = tid; p < P; p += threads) {
    const int e = ids[t0 * k + p];
    L.ids[p] = (e >= 0 && e < G) ? e : -1;
  }
  __syncthreads();
  for (int p = tid; p < P; p += threads) {
    const int e = L.ids[p];
    bool again = false;
    for (int q = p / k * k; q < p; ++q) again |= L.ids[q] == e;
    L.again[p] = again;
    if (e >= 0 && !again) atomicMin(&L.first[e], p);
  }
  __syncthreads();
  int total = 0;
  for (int p0 = 0; p0 < P; p0 += threads) {
    const int p = p0 + tid, e = p < P ? L.ids[p] : -1;
    const bool lead = e >= 0 && (L.again[p] || L.first[e] == p);
    const uint64_t m = __ballot(lead);
    if ((tid & 63) == 0) L.count[tid >> 6] = __popcll(m);
    __syncthreads();
    int before = total;
    for (int i = 0; i < threads >> 6; ++i) {
      if (i < tid >> 6) before += L.count[i];
      total += L.count[i];
    }
    if (lead) L.item[before + __popcll(m & ((1ull << (tid & 63)) - 1))] = (uint16_t)p;
    __syncthreads();
  }
  return __builtin_amdgcn_readfirstlane(total);
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

// The weights of NT row tiles of one expert: wave-uniform pointers to each tile's first K block,
// and this lane's offsets (row lane % 16, piece lane / 16) in a block of codes and of scales.
// (code_high, scale_high: from the lane's row to the one eight below, for the paired form.)
template <int NT>
struct Tiles {
  const uint8_t* codes[NT];
  const uint8_t* scales[NT];
  uint32_t code_lane[NT], scale_lane[NT];
  uint32_t code_high[NT], scale_high[NT];
};

// n <= U K blocks from kb on of NT row tiles of one expert, added to acc: every load is issued
// before the first is used, and none is conditional (a load under a branch is waited for at
// the branch's end; past n the last block is read again).  WIDE (kb a multiple of 4): a row's 16
// scale bytes of four blocks in one load; a byte per block otherwise.  LAST: the block that K ends
// in, whose lanes past the end read the block's first piece and multiply it by zeros.
template <class TX, bool TILED, int NT, int NC, int U, bool WIDE, bool LAST>
__device__ inline void gemv_step(const Tiles<NT>& w, const TX* xrow, int64_t K, int kb, int n,
                                 v4f (&acc)[NT][Frag<TX, NC>::F]) {
  const int c = (threadIdx.x & 63) >> 4;
  const bool in = !LAST || (int64_t)kb * 128 + 32 * c < K;
  const int back = in ? 0 : c;                       // pieces back to the block's first one
  u32x4 q[U][NT], wide[WIDE ? U / 4 : 1][NT];
  uint32_t e[WIDE ? 1 : U][NT];
  Frag<TX, NC> f[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int b = kb + (u < n ? u : n - 1);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // (a block's codes and scales: uniform pointer + 32-bit lane offset)
      const uint8_t* wb = w.codes[i] + (int64_t)b * (TILED ? 1024 : 64);
      q[u][i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wb + (w.code_lane[TILED ? 0 : i] - 16u * back)));
      if constexpr (!WIDE) {
        const uint8_t* sb = w.scales[i] + (TILED ? (int64_t)(b >> 2) * 256 + 4 * (b & 3) : (int64_t)b * 4);
        e[u][i] = sb[w.scale_lane[TILED ? 0 : i] + (uint32_t)(c - back)];
      } else if (u % 4 == 0) {
        const uint8_t* sb = w.scales[i] + (int64_t)(b >> 2) * (TILED ? 256 : 16);
        wide[u / 4][i] = *reinterpret_cast<const u32x4_a1*>(sb + w.scale_lane[TILED ? 0 : i]);
      }
    }
    f[u].load(xrow + (int64_t)b * 128 - 32 * back);
    if (LAST && !in) f[u].clear();
  }
  __builtin_amdgcn_sched_barrier(0);                 // keep the loads together, ahead of their uses
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= n) break;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint32_t byte = WIDE ? (wide[WIDE ? u / 4 : 0][i][u % 4] >> (8 * c)) & 0xFFu : e[WIDE ? 0 : u][i];
      const float scale = __uint_as_float(byte << 23);
#pragma unroll
      for (int d = 0; d < 4; ++d) f[u].mul(d, dequant8(q[u][i][d], scale), acc[i]);
    }
    __builtin_amdgcn_sched_barrier(0);               // and the converted codes of one block at a time
  }
}

// One wave's share: K blocks [kb0, kb1), kb0 a multiple of 4; the sums of column t (t < NC) in the
// lanes of column t.  xrow: the lane's activations at operand col / NC (in a column without a token
// any: a column's sums depend on its own activations only).
template <class TX, bool TILED, int NT, int NC>
__device__ inline void gemv_run(const Tiles<NT>& w, const TX* xrow, int64_t K, int kb0, int kb1, v4f (&sum)[NT]) {
  constexpr int F = Frag<TX, NC>::F;
  // blocks in flight: as many as about 70 registers of operands hold
  constexpr int U = sizeof(TX) == 4 ? (NT == 1 ? 2 : 1) : NT == 1 ? (NC == 4 ? 8 : 4) : NC == 16 ? 2 : 4;
  v4f acc[NT][F];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[i][f] = v4f{0, 0, 0, 0};
  const int whole = (int64_t)kb1 * 128 <= K ? kb1 : kb1 - 1;
  int kb = kb0;
  if constexpr (U >= 4) {
    for (; kb + U <= whole; kb += U) gemv_step<TX, TILED, NT, NC, U, true, false>(w, xrow, K, kb, U, acc);
    if constexpr (U == 8) {
      if (kb + 4 <= whole) gemv_step<TX, TILED, NT, NC, 4, true, false>(w, xrow, K, kb, 4, acc), kb += 4;
    }
    // one to three blocks of a span of four (a plain row has no bytes behind it, a tiled one is padded)
    if (kb < whole) gemv_step<TX, TILED, NT, NC, 4, TILED, false>(w, xrow, K, kb, whole - kb, acc);
  } else {
    for (; kb + U <= whole; kb += U) gemv_step<TX, TILED, NT, NC, U, false, false>(w, xrow, K, kb, U, acc);
    if (U == 2 && kb < whole) gemv_step<TX, TILED, NT, NC, 1, false, false>(w, xrow, K, kb, 1, acc);
  }
  if (!TILED && whole < kb1) gemv_step<TX, TILED, NT, NC, 1, false, true>(w, xrow, K, whole, 1, acc);
  // column NC * f + t of accumulator f: pick, then add the F columns of each token
  const int mine = (threadIdx.x & 15) / NC;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    v4f v = acc[i][0];
#pragma unroll
    for (int f = 1; f < F; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = mine == f ? acc[i][f][r] : v[r];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (F >= 2) v[r] += dpp_move<0x128>(v[r]);   // 8 columns round
      if constexpr (F >= 4) v[r] += dpp_move<0x124>(v[r]);   // 4 columns round
    }
    sum[i] = v;
  }
}

// The untiled layout, bf16 activations.  A tile's row is K / 2 bytes from the next, and a K block of
// it only half a cache line; a request for half a line occupies the vector cache like a whole
// one.  So a load takes eight rows x two K blocks: in the lanes of rows 0-7 the first block of
// the lane's row, in those of rows 8-15 the second block of row - 8, and a second load the same of
// rows 8-15.  The matrix instruction is given activations of both blocks at once, in different
// columns (col = t + NC * (h + 2 * i): token t, block h, operand i); of its results only rows
// 0-7 x the columns h = 0 and rows 8-15 x the columns h = 1 mean anything, and their sum is
// the eight rows' products.  More than eight tokens take two sets of columns (TG = 2).
//
// n <= U pairs of K blocks from pair p on.  WIDE (p even, U even): sixteen scale bytes per row and two pairs
// in one load.  LAST: the pair that K ends in; pieces past the end read the pair's first piece, and
// their activations are zeros.
template <int NT, int NC, int TG, int U, bool WIDE, bool LAST>
__device__ inline void rows_step(const Tiles<NT>& w, const uint16_t* const (&xrow)[TG], int64_t K, int p, int n,
                                 v4f (&acc)[NT][2][TG][8 / NC]) {
  constexpr int F = 8 / NC;                          // operands per register set
  const int lane = threadIdx.x & 63, c = lane >> 4, second = (lane >> 3) & 1;
  // this lane's piece of the pair in the codes, and in the activations
  const bool in = !LAST || (int64_t)p * 256 + 128 * second + 32 * c < K;
  const uint32_t back = in ? 0 : 4 * second + c;
  const int xh = (lane & 15) / NC % 2;
  const bool xin = !LAST || (int64_t)p * 256 + 128 * xh + 32 * c < K;
  const int xback = xin ? 0 : 128 * xh + 32 * c;
  u32x4 q[U][NT][2], wide[WIDE ? U / 2 : 1][NT][2], x[U][TG][4 / F];
  uint32_t e[WIDE ? 1 : U][NT][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int b = p + (u < n ? u : n - 1);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        const uint32_t cl = w.code_lane[i] + (z ? w.code_high[i] : 0), sl = w.scale_lane[i] + (z ? w.scale_high[i] : 0);
        q[u][i][z] = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(w.codes[i] + (int64_t)b * 128 + (cl - 16u * back)));
        if constexpr (!WIDE) e[u][i][z] = (w.scales[i] + (int64_t)b * 8)[sl + (4u * second + c - back)];
        else if (u % 2 == 0)
          wide[u / 2][i][z] = *reinterpret_cast<const u32x4_a1*>(w.scales[i] + (int64_t)(b >> 1) * 16 + sl);
      }
#pragma unroll
    for (int g = 0; g < TG; ++g)
#pragma unroll
      for (int s = 0; s < 4 / F; ++s) {
        x[u][g][s] = *reinterpret_cast<const u32x4_a2*>(xrow[g] + (int64_t)b * 256 + 8 * F * s - xback);
        if (LAST && !xin) x[u][g][s] = u32x4{0, 0, 0, 0};
      }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= n) break;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        uint32_t byte;
        if constexpr (WIDE) {
          const u32x4 s = wide[u / 2][i][z];
          byte = ((second ? s[2 * (u % 2) + 1] : s[2 * (u % 2)]) >> (8 * c)) & 0xFFu;
        } else {
          byte = e[u][i][z];
        }
        const float scale = __uint_as_float(byte << 23);
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          const bf16x8 a = dequant8(q[u][i][z][d], scale);
#pragma unroll
          for (int g = 0; g < TG; ++g)
            acc[i][z][g][d % F] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                a, __builtin_bit_cast(bf16x8, x[u][g][d / F]), acc[i][z][g][d % F], 0, 0, 0);
        }
      }
    __builtin_amdgcn_sched_barrier(0);
  }
}

// One wave's share, as gemv_run: kb0 a multiple of 4, the sums of column t in the lanes of column t.
template <int NT, int NC, int TG>
__device__ inline void rows_run(const Tiles<NT>& w, const uint16_t* const (&xrow)[TG], int64_t K, int kb0, int kb1,
                                v4f (&sum)[NT]) {
  constexpr int F = 8 / NC;
  constexpr int U = NT == 1 && TG == 1 ? 2 : 1;
  v4f acc[NT][2][TG][F];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int g = 0; g < TG; ++g)
#pragma unroll
        for (int f = 0; f < F; ++f) acc[i][z][g][f] = v4f{0, 0, 0, 0};
  const int whole = (int64_t)kb1 * 128 <= K ? kb1 / 2 : (kb1 - 1) / 2;   // pairs that K fills
  int p = kb0 / 2;
  for (; p + U <= whole; p += U) rows_step<NT, NC, TG, U, U != 1, false>(w, xrow, K, p, U, acc);
  if constexpr (U == 4) {
    if (p + 2 <= whole) rows_step<NT, NC, TG, 2, true, false>(w, xrow, K, p, 2, acc), p += 2;
  }
  if (U > 1 && p < whole) rows_step<NT, NC, TG, 1, false, false>(w, xrow, K, p, 1, acc), ++p;
  if (2 * p < kb1) rows_step<NT, NC, TG, 1, false, true>(w, xrow, K, p, 1, acc);
  // operands (columns 2 NC apart), then the two blocks (columns NC apart, rows 8 apart)
  const bool low = (threadIdx.x & 63) < 32;
  const int col = threadIdx.x & 15;
  const auto pick = [&](const v4f (&z0)[F], const v4f (&z1)[F], int r) {
    float v0 = z0[0][r], v1 = z1[0][r];
    if constexpr (F == 2) {
      v0 = col < 8 ? v0 : z0[1][r];
      v1 = col < 8 ? v1 : z1[1][r];
      v0 += dpp_move<0x128>(v0);
      v1 += dpp_move<0x128>(v1);
    }
    const float w0 = dpp_move<0x120 + NC>(v0), w1 = dpp_move<0x120 + NC>(v1);
    const uint32_t up = __builtin_amdgcn_permlane32_swap(__float_as_uint(w0), __float_as_uint(w0), false, false)[1];
    const uint32_t dn = __builtin_amdgcn_permlane32_swap(__float_as_uint(v1), __float_as_uint(v1), false, false)[0];
    return low ? v0 + __uint_as_float(up) : __uint_as_float(dn) + w1;
  };
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v = pick(acc[i][0][0], acc[i][1][0], r);
      if constexpr (TG == 2) {                       // tokens 8-15 to columns 8-15
        const float t = dpp_move<0x128>(pick(acc[i][0][1], acc[i][1][1], r));
        v = col < 8 ? v : t;
      }
      sum[i][r] = v;
    }
}

}  // namespace

template <int MODE, bool TILED, class TX, int NCMAX, int RT>
__global__ void __launch_bounds__(64 * kMaxWaves, 4) gemv_fp4_kernel(GemvArgs a) {
  constexpr int NT = MODE == kSilu ? 2 * RT : RT;    // row tiles: RT, or RT of gate and RT of up
  __shared__ Items L;
  __shared__ float part[kMaxWaves][NT][16][16];      // [wave][tile][token][row]
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, c = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16 * RT;
  const int64_t t0 = (int64_t)blockIdx.z * 16;
  const int Tn = a.T - t0 < 16 ? (int)(a.T - t0) : 16;
  const int64_t width = MODE == kSilu ? 2 * a.N : a.N;
  // the waves share the K blocks in spans of four
  const int nkb = (int)((a.K + 127) / 128), spans = (nkb + 3) / 4, waves = blockDim.x >> 6;
  const TX* x = (const TX*)a.x;
  const bool obf = a.out_bf16;

  const int items = !a.ids              ? 1
                    : Tn * a.k <= 64 ? list_few_items(L, a.ids, t0, Tn * a.k, a.k, a.G)
                                     : list_items(L, a.ids, t0, Tn, a.k, a.G);

  // The tokens of visit p0, one a column: returns their number, and in L.column[wave] which.
  auto columns = [&](int p0) -> int {
    if (!a.ids) {
      if (lane < 16) L.column[wave][lane] = (uint16_t)(lane < Tn ? lane : 0);
      return Tn;
    }
    const int j = slot_of(L, p0, col, Tn, a.k);
    const uint32_t m = (uint32_t)__ballot(lane < 16 && j >= 0);
    if (lane < 16 && j >= 0) L.column[wave][__popc(m & ((1u << lane) - 1))] = (uint16_t)(lane + 16 * j);
    return __popc(m);
  };
  constexpr bool kPairs = !TILED && sizeof(TX) == 2;
  // K blocks [kb0, kb1) of expert e for the nc tokens of L.column[wave], into sum (column t: the t-th)
  auto visit = [&](int e, int nc, int kb0, int kb1, v4f (&sum)[NT]) {
    Tiles<NT> w;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int64_t up = i >= RT ? a.N : 0, r0 = n0 + 16 * (i % RT);
      if constexpr (TILED) {
        const int64_t last = a.N / 16 - 1, nb = (r0 / 16 < last ? r0 / 16 : last) + up / 16;
        w.codes[i] = uniform_ptr(a.b + ((int64_t)e * (width / 16) + nb) * (a.K / 128) * 1024);
        w.scales[i] = uniform_ptr(a.s + ((int64_t)e * (width / 16) + nb) * ((a.K + 511) / 512) * 256);
        w.code_lane[i] = 16 * lane;
        w.scale_lane[i] = 16 * col;
      } else {
        const int64_t last = a.N - 1, base = r0 < last ? r0 : last;
        const int rows = (int)(last - base);         // rows past the end: the last one, not stored
        w.codes[i] = uniform_ptr(a.b + ((int64_t)e * width + up + base) * (a.K / 2));
        w.scales[i] = uniform_ptr(a.s + ((int64_t)e * width + up + base) * (a.K / 32));
        const uint32_t row = (uint32_t)((kPairs ? col & 7 : col) < rows ? (kPairs ? col & 7 : col) : rows);
        const uint32_t high = (uint32_t)((col & 7) + 8 < rows ? (col & 7) + 8 : rows);
        w.code_lane[i] = row * (uint32_t)(a.K / 2) + 16 * c + (kPairs ? 64 * (col >> 3) : 0);
        w.scale_lane[i] = row * (uint32_t)(a.K / 32);
        w.code_high[i] = (high - row) * (uint32_t)(a.K / 2);
        w.scale_high[i] = (high - row) * (uint32_t)(a.K / 32);
      }
    }
    if constexpr (kPairs) {
      auto go = [&](auto n, auto g) {
        constexpr int NC = decltype(n)::value, TG = decltype(g)::value;
        const TX* row[TG];
#pragma unroll
        for (int q = 0; q < TG; ++q) {
          const int t = col % NC + NC * q, h = col / NC % 2, i = col / (2 * NC);
          const int tj = L.column[wave][t < nc ? t : 0];
          const int64_t xr = a.per_slot ? (t0 + (tj & 15)) * a.k + (tj >> 4) : t0 + (tj & 15);
          row[q] = x + xr * a.ldx + 128 * h + 32 * c + 8 * i;
        }
        rows_run<NT, NC, TG>(w, row, a.K, kb0, kb1, sum);
      };
      using std::integral_constant;
      if (NCMAX == 4 || nc <= 4) go(integral_constant<int, 4>(), integral_constant<int, 1>());
      else if (nc <= 8) go(integral_constant<int, 8>(), integral_constant<int, 1>());
      else go(integral_constant<int, 8>(), integral_constant<int, 2>());
      return;
    }
    auto go = [&](auto n) {
      constexpr int NC = decltype(n)::value;
      const int t = col % NC;
      const int tj = L.column[wave][t < nc ? t : 0];
      const int64_t row = a.per_slot ? (t0 + (tj & 15)) * a.k + (tj >> 4) : t0 + (tj & 15);
      gemv_run<TX, TILED, NT, NC>(w, x + row * a.ldx + 32 * c + 8 * (col / NC), a.K, kb0, kb1, sum);
    };
    if constexpr (sizeof(TX) == 4) {
      go(std::integral_constant<int, 16>());
    } else {
      if (NCMAX == 4 || nc <= 4) go(std::integral_constant<int, 4>());
      else if (nc <= 8) go(std::integral_constant<int, 8>());
      else go(std::integral_constant<int, 16>());
    }
  };
  // the sum over the waves of one value, in wave order
  auto joined = [&](int i, int t, int r) {
    float v = part[0][i][t][r];
    for (int q = 1; q < waves; ++q) v += part[q][i][t][r];
    return v;
  };

  if constexpr (MODE == kSum) {
    // the waves split the K blocks of all visits, expert by expert, and keep their own sums in LDS
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<v4f*>(&part[wave][i][col][4 * c]) = v4f{0, 0, 0, 0};
    const int64_t units = (int64_t)items * spans;
    int64_t at = units * wave / waves;
    const int64_t end = units * (wave + 1) / waves;
    while (at < end) {
      const int it = (int)(at / spans), s0 = (int)(at - (int64_t)it * spans);
      const int s1 = (int)(end - (int64_t)it * spans < spans ? end - (int64_t)it * spans : spans);
      const int p0 = __builtin_amdgcn_readfirstlane(L.item[it]), nc = columns(p0);
      const int tj = L.column[wave][col < nc ? col : 0], t = tj & 15;
      const float g = a.w[(t0 + t) * a.k + (tj >> 4)];
      v4f sum[NT];
      visit(__builtin_amdgcn_readfirstlane(L.ids[p0]), nc, 4 * s0, 4 * s1 < nkb ? 4 * s1 : nkb, sum);
      if (col < nc) {
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          v4f* p = reinterpret_cast<v4f*>(&part[wave][i][t][4 * c]);
          v4f v = *p;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = fmaf(g, sum[i][r], v[r]);
          *p = v;
        }
      }
      at += s1 - s0;
    }
    __syncthreads();
    for (int i = tid; i < RT * 256; i += blockDim.x) {
      const int t = (i >> 4) & 15, r = i & 15;
      const int64_t n = n0 + 16 * (i >> 8) + r;
      if (t < Tn && n < a.N) put(a.out, obf, (t0 + t) * a.ldo + n, joined(i >> 8, t, r));
    }
  } else {
    const int kb0 = 4 * (int)((int64_t)spans * wave / waves), end = 4 * (int)((int64_t)spans * (wave + 1) / waves);
    const int kb1 = end < nkb ? end : nkb;
    for (int it = blockIdx.y; it < items; it += gridDim.y) {
      const int p0 = a.ids ? __builtin_amdgcn_readfirstlane(L.item[it]) : 0, nc = columns(p0);
      v4f sum[NT];
      visit(a.ids ? __builtin_amdgcn_readfirstlane(L.ids[p0]) : 0, nc, kb0, kb1, sum);
#pragma unroll
      for (int i = 0; i < NT; ++i) *reinterpret_cast<v4f*>(&part[wave][i][col][4 * c]) = sum[i];
      __syncthreads();
      for (int i = tid; i < RT * 256; i += blockDim.x) {
        const int t = (i >> 4) & 15, r = i & 15;
        const int64_t n = n0 + 16 * (i >> 8) + r;
        if (t >= nc || n >= a.N) continue;
        float v = joined(i >> 8, t, r);
        if constexpr (MODE == kSilu) v = v / (1.0f + expf(-v)) * joined(RT + (i >> 8), t, r);
        const int tj = L.column[wave][t];
        put(a.out, obf, ((t0 + (tj & 15)) * a.k + (tj >> 4)) * a.ldo + n, v);
      }
      __syncthreads();
    }
    if (a.ids && blockIdx.y == 0) {                  // slots without an expert
      for (int p = tid >> 4; p < Tn * a.k; p += blockDim.x >> 4) {
        if (L.ids[p] >= 0) continue;
        for (int r = tid & 15; r < 16 * RT; r += 16)
          if (n0 + r < a.N) put(a.out, obf, (t0 * a.k + p) * a.ldo + n0 + r, 0.0f);
      }
    }
  }
}

static constexpr int gemv_lds(int nt) { return (int)sizeof(Items) + kMaxWaves * nt * 1024; }
const KernelInfo kInfoGemvFp4 = {"gemv_fp4_kernel", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kMaxWaves, 0, 0, gemv_lds(1),
                                 gemv_lds(1), (const void*)gemv_fp4_kernel<kPlain, true, uint16_t, 16, 1>};
const KernelInfo kInfoGemvFp4Silu = {"gemv_fp4_kernel<silu>", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kMaxWaves, 0, 0,
                                     gemv_lds(2), gemv_lds(2),
                                     (const void*)gemv_fp4_kernel<kSilu, true, uint16_t, 16, 1>};
const KernelInfo kInfoGemvFp4Sum = {"gemv_fp4_kernel<sum>", "fgg_moe_gemv_fp4", 16, 16, 128, 64 * kMaxWaves, 0, 0,
                                    gemv_lds(1), gemv_lds(1), (const void*)gemv_fp4_kernel<kSum, true, uint16_t, 16, 1>};

hipError_t launch_gemv_fp4(bool tiled, int32_t G, int64_t T, int32_t k, int64_t N, int64_t K, const void* x,
                           bool x_bf16, int64_t ldx, bool per_slot, const uint8_t* b, const uint8_t* s,
                           const int32_t* ids, const float* w, bool silu, void* out, bool out_bf16, int64_t ldo,
                           int num_cus, hipStream_t st) {
  const GemvArgs a = {G, T, k, N, K, x, ldx, per_slot, b, s, ids, w, out, out_bf16, ldo};
  const int64_t pairs = (T < 16 ? T : 16) * k;
  const unsigned visits = ids && !w ? (unsigned)(pairs < G ? pairs : G) : 1;
  const int waves = !w && K <= 2048 ? 4 : kMaxWaves;   // a span of 512 K for each
  // Two row tiles a wave share the activations' loads, which is worth most of their cost from five
  // tokens on (tiled: down of 16 tokens, N 7168, 62 -> 53.5 us; 16384 x 7168, 16 tokens, 32 -> 25), as
  // long as there is a workgroup for most compute units (4096 x 7168, 128 workgroups, 11.4 -> 14.4).
  // Not with the untiled layout's paired loads (8 tokens 61 -> 65 us: registers spill).
  const int rt = tiled && x_bf16 && !silu && T > 4 && (N + 31) / 32 * visits >= num_cus * 3 / 4 ? 2 : 1;
  const dim3 grid((unsigned)((N + 16 * rt - 1) / (16 * rt)), visits, (unsigned)((T + 15) / 16));
  const KernelInfo& info = w ? kInfoGemvFp4Sum : silu ? kInfoGemvFp4Silu : kInfoGemvFp4;
  trace_launch(info, grid, "G=%d T=%lld k=%d N=%lld K=%lld %s %s->%s", (int)G, (long long)T, (int)k, (long long)N,
               (long long)K, tiled ? "tiled" : "rows", x_bf16 ? "bf16" : "fp32", out_bf16 ? "bf16" : "fp32");
  auto go = [&](auto mode, auto til, auto tx, auto nc, auto r) {
    hipLaunchKernelGGL((gemv_fp4_kernel<decltype(mode)::value, decltype(til)::value, decltype(tx), decltype(nc)::value,
                                        decltype(r)::value>), grid, dim3(64 * waves), 0, st, a);
  };
  using std::integral_constant;
  auto with_type = [&](auto mode, auto til) {
    using One = integral_constant<int, 1>;
    if (!x_bf16) return go(mode, til, float(), integral_constant<int, 16>(), One());
    if (T <= 4) return go(mode, til, uint16_t(), integral_constant<int, 4>(), One());
    if constexpr (decltype(mode)::value != kSilu && decltype(til)::value) {
      if (rt == 2) return go(mode, til, uint16_t(), integral_constant<int, 16>(), integral_constant<int, 2>());
    }
    go(mode, til, uint16_t(), integral_constant<int, 16>(), One());
  };
  auto with_mode = [&](auto til) {
    if (w) with_type(integral_constant<int, kSum>(), til);
    else if (silu) with_type(integral_constant<int, kSilu>(), til);
    else with_type(integral_constant<int, kPlain>(), til);
  };
  if (tiled) with_mode(std::true_type());
  else with_mode(std::false_type());
  return hipGetLastError();
}

}  // namespace fgg
