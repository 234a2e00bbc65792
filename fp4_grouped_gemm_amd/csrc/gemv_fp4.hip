// Few tokens times 4-bit expert weights, activations unquantized: the generation step's
// form of the experts' products.
//
//   y[t, j][n] = sum_K x[t (, j)][K] * B[e][n][K],   e = topk_ids[t][j],
//   B = E2M1 code * 2^(scale byte - 127), one scale byte per 32 along K
//
// plain (y per slot), with SiLU(gate)*up (B holds [gate | up] rows), or summed over the
// token's slots with the gate weights.
//
// Bound by the weights' bytes: every distinct expert of up to 16 tokens is read once, whatever number
// of them chose it.  Measured: gate-up of one token's 8 experts (N 2048, K 7168, tiled, 125 MB) 22.8
// us, 5.5 TB/s, of 32 experts 85.7 us, 5.8 TB/s; of 16 tokens 94.7 us, 5.2 TB/s; down of 16 tokens (N
// 7168, K 2048, 248 MB) 49 us tiled, 62 us untiled (half lines); a 4096 x 7168 matrix and one token 6.0
// us, of which a launch and two memory latencies are most.  fp32 activations cost two to four times that
// (gate-up of one token 60 us, of 16 tokens 225; down of 16 tokens, tiled, 189): instruction issue.  An E2M1 code times a power of two is a bf16
// number, so the weights go through v_cvt_scalef32_pk_bf16_fp4 (two codes and their scale per
// instruction) into the bf16 matrix instruction 16x16x32 with 16 weight rows as its rows and the tokens
// as its columns: products are exact, sums in fp32.  One 16-byte load per lane (row lane % 16, 32
// consecutive K at 32 * (lane / 16): one scale) feeds four of them; K runs through the instructions in
// that order on both operands.  fp32 activations are split into three bf16 parts (8 + 8 + 8 bits,
// exact down to bf16's smallest step, 2^-133) and take three instructions.
//
// A workgroup owns a tile of weight rows; its four, eight or sixteen waves split the K blocks (of every
// expert, in the summed form), or with little K own a tile for each one or two, and their partial sums
// are joined through LDS in a fixed order, so no result depends on the order of arrival.  Tokens are
// columns: the experts to visit are the distinct ids among the tokens' slots, found per workgroup by an
// LDS table of first occurrences; a token that names one expert twice has its second slot visited on
// its own.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_wave.hpp"

namespace fgg {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32_a1 __attribute__((aligned(1)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int kMaxWaves = 16;       // (of one workgroup)
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
  int group;             // tokens of a workgroup, at most 16
};

// The eight codes of one 32-bit word, times 2^(byte - 127), as bf16.  scale holds the byte as its exponent, which is
// all that the instruction reads: byte 0 is 2^-127 and 255 a NaN, and results below 2^-126 keep their bits (bf16 has
// them to 2^-133, and the matrix core takes them).
__device__ inline bf16x8 dequant8(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Activations of one K block for up to NC tokens (4, 8 or 16).  The matrix instruction has 16
// columns and a K block takes four of them (operand d: elements 8d .. 8d + 7 of each lane's 32).
// With few tokens the columns hold several operands at once: column F * t + i holds token t's
// operand s * F + i of register set s (F = 16 / NC operands per set), so a K block takes NC / 4
// register sets instead of four.  Instruction d multiplies set d / F into accumulator
// d % F, of which only columns F * t + d % F mean anything: those are picked at the end.
//
// Loads are made for four neighbouring lanes to share 64 bytes.  Up to four tokens have that in the
// operand order itself (a quad is one token's four operands).  In that order sixteen tokens' loads
// would touch 32 lines each, 16 bytes of 64 of them (dense 16384 x 7168: 32 us against 25): more are
// loaded row by row, 16 lanes to a token's block, and turned into operands through LDS: every wave has
// its own scratch, its LDS accesses run in order, and a row's 16-byte pieces are XORed with a key
// for which the sixteen lanes that a cycle of ds_read_b128 serves (0-3, 12-15, 20-27 and so on) hit
// sixteen different bank groups.
constexpr int kXsBytes = 16 * 256;                   // sixteen tokens' blocks
template <class TX, int NC>
struct Frag;
template <int NC>
struct Frag<uint16_t, NC> {
  static constexpr int F = 16 / NC, S = NC / 4;
  u32x4 v[S];
  // the lane's element offset in its token's row, and the token whose row that is, of register set s
  static __device__ int token(int lane, int s) { return NC == 4 ? (lane & 15) / F : 4 * s + (lane >> 4); }
  static __device__ int element(int lane) {
    return NC == 4 ? 32 * (lane >> 4) + 8 * (lane & 15 & (F - 1)) : 8 * (lane & 15);
  }
  __device__ void load(const uint16_t* const (&row)[S], int64_t at, bool in) {
#pragma unroll
    for (int s = 0; s < S; ++s) {
      v[s] = *reinterpret_cast<const u32x4_a2*>(row[s] + at);
      if (!in) v[s] = u32x4{0, 0, 0, 0};
    }
  }
  // into operand order (set s: operands s * F + i)
  __device__ void arrange(uint8_t* xs, int lane) {
    if constexpr (NC > 4) {
      const int col = lane & 15, c = lane >> 4;
      const auto key = [](int t) { return F == 1 ? (t & 3) | (t >> 3) * 8 : (t & 1) * 2 | (t >> 2) * 8; };
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int t = 4 * s + c;
        *reinterpret_cast<u32x4*>(xs + t * 256 + 16 * (col ^ key(t))) = v[s];
      }
      wave_sync();
      const int t = col / F;
#pragma unroll
      for (int s = 0; s < S; ++s)
        v[s] = *reinterpret_cast<const u32x4*>(xs + t * 256 + 16 * ((4 * c + F * s + col % F) ^ key(t)));
      wave_sync();
    }
  }
  __device__ void mul(int d, bf16x8 a, v4f (&acc)[F]) const {
    acc[d % F] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, __builtin_bit_cast(bf16x8, v[d / F]), acc[d % F], 0, 0, 0);
  }
};
template <>
struct Frag<float, 16> {
  static constexpr int F = 1, S = 1;
  u32x4 v[8];
  static __device__ int token(int lane, int) { return lane & 15; }
  static __device__ int element(int lane) { return 32 * (lane >> 4); }
  __device__ void load(const float* const (&row)[1], int64_t at, bool in) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = *reinterpret_cast<const u32x4_a4*>(row[0] + at + 4 * i);
      if (!in) v[i] = u32x4{0, 0, 0, 0};
    }
  }
  __device__ void arrange(uint8_t*, int) {}
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

// Whether more than four tokens' bf16 activations are turned into operands through LDS.
template <class TX, int NC>
constexpr bool stages_activations() { return NC > 4 && sizeof(TX) == 2; }

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
  float gate[kMaxPairs];            // gate weights (the summed form)
};

// The list of at most 64 pairs, by each wave on its own: lane p holds pair p, and each distinct expert's
// pairs are one ballot.  Every wave writes the same values to LDS and reads only what it
// wrote itself, so there is no barrier.
__device__ inline int list_few_items(Items& L, const int32_t* ids, int64_t t0, int P, int k, int G) {
  const int p = threadIdx.x & 63;
  int e = p < P ? ids[t0 * k + p] : -1;
  if (e < 0 || e >= G) e = -1;
  uint64_t same = 0;                                  // the pairs that name this pair's expert
  for (uint64_t left = __ballot(e >= 0); left;) {
    const int head = __builtin_amdgcn_readlane(e, __ffsll((unsigned long long)left) - 1);
    const uint64_t m = __ballot(e == head);
    if (e == head) same = m;
    left &= ~m;
  }
  const uint64_t before = (1ull << p) - 1, token = ~0ull << (p / k * k);   // (p / k * k <= p < 64)
  const bool again = (same & before & token) != 0;
  const bool lead = e >= 0 && (again || (same & before) == 0);
  const uint64_t m = __ballot(lead);
  if (p < P) {
    L.ids[p] = e;
    L.again[p] = (uint8_t)again;
    if (lead) L.item[__popcll(m & before)] = (uint16_t)p;
  }
  wave_sync();
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

// The weights of NT row tiles of one expert: wave-uniform pointers to each tile's first K block,
// and this lane's offsets in a block of codes (16 bytes), in a span of four blocks of scales, and
// (untiled) of the scale byte of its operand in a block.
//
// The operand of lane 16 c + r is piece c of row r.  Tiled, that is the order in memory.  Untiled, the
// 64-byte rows of a block are loaded four lanes to a row (lane 4 r + c) and moved to their lanes by
// an LDS permute, and so is a row's dword of four scale bytes per block (lane 4 r + block).
template <int NT>
struct Tiles {
  const uint8_t* codes[NT];
  const uint8_t* scales[NT];
  uint32_t code_lane[NT], scale_lane[NT], byte_lane[NT];
};

// n <= U K blocks from kb on of NT row tiles of one expert, added to acc: every load is issued
// before the first is used, and none is conditional (a load under a branch is waited for at
// the branch's end; past n the last block is read again).  WIDE (U >= 2, kb a multiple of U): the scale
// bytes of a span of four blocks in one load; a byte per block otherwise.  FULL: n is U.  LAST (U = 1):
// the block that K ends in, whose lanes past the end read the block's first piece, with zeros for
// activations.
template <class TX, bool TILED, int NT, int NC, int U, bool WIDE, bool FULL, bool LAST>
__device__ inline void gemv_step(const Tiles<NT>& w, const TX* const (&xrow)[Frag<TX, NC>::S], uint8_t* scratch,
                                 int lane, int64_t K, int kb, int n, v4f (&acc)[NT][Frag<TX, NC>::F]) {
  using X = Frag<TX, NC>;
  const int col = lane & 15, c = lane >> 4;
  const int64_t k0 = (int64_t)kb * 128;
  // (LAST) back to the block's first piece: of codes, of scale bytes, of activations
  const uint32_t cback = LAST && k0 + 32 * (lane & 3) >= K ? lane & 3 : 0;
  const uint32_t sback = LAST && k0 + 32 * c >= K ? c : 0;
  const bool xin = !LAST || k0 + X::element(lane) < K;
  const int xback = xin ? 0 : X::element(lane);
  using Scales = std::conditional_t<TILED, u32x4, uint32_t>;
  u32x4 q[U][NT];
  Scales wide[WIDE ? (U + 3) / 4 : 1][NT];
  uint32_t e[WIDE ? 1 : U][NT];
  X f[U];
  // Uniform pointers + 32-bit lane offsets (activations: lane pointers), and a block's place in the
  // step as a constant where the step is full: no address registers per load.
  const int64_t code_step = TILED ? 1024 : 64;
  const uint8_t *wb[NT], *sb[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    wb[i] = w.codes[i] + kb * code_step;
    sb[i] = w.scales[i] + (TILED ? (int64_t)(kb >> 2) * 256 : (int64_t)(WIDE ? kb & ~3 : kb) * 4);
  }
  const TX* xb[X::S];
#pragma unroll
  for (int s = 0; s < X::S; ++s) xb[s] = xrow[s] + (int64_t)kb * 128 - xback;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int b = FULL || u < n ? u : n - 1;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const auto* at = reinterpret_cast<const u32x4*>(wb[i] + (w.code_lane[i] - 16 * cback) + b * code_step);
      // Whole lines, read once: past the caches.  Untiled, a load takes half of each line and the next
      // block's load the other half, from the cache (8 experts' gate-up 35 -> 28 us).
      if constexpr (TILED) q[u][i] = __builtin_nontemporal_load(at);
      else q[u][i] = *at;
      if constexpr (!WIDE) {
        const int in_span = TILED ? ((kb & 3) + b) * 4 : b * 4;   // (tiled: the step stays in its span)
        e[u][i] = (sb[i] + (w.byte_lane[i] - sback))[in_span];
      } else if (u % 4 == 0) {
        if constexpr (TILED) wide[u / 4][i] = *reinterpret_cast<const u32x4*>(sb[i] + w.scale_lane[i]);
        else wide[u / 4][i] = *reinterpret_cast<const u32_a1*>(sb[i] + w.scale_lane[i]);
      }
    }
    f[u].load(xb, b * 128, xin);
  }
  __builtin_amdgcn_sched_barrier(0);                 // keep the loads together, ahead of their uses
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!FULL && u >= n) break;
    f[u].arrange(scratch, lane);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      u32x4 a = q[u][i];
      if constexpr (!TILED) {
#pragma unroll
        for (int d = 0; d < 4; ++d) a[d] = __builtin_amdgcn_ds_bpermute(4 * (4 * col + c), a[d]);
      }
      uint32_t byte;
      if constexpr (!WIDE) {
        byte = e[u][i];
      } else if constexpr (TILED) {
        const u32x4 s = wide[u / 4][i];
        const uint32_t four = U >= 4 ? s[u % 4] : kb & 2 ? s[(u + 2) % 4] : s[u % 4];
        byte = (four >> (8 * c)) & 0xFFu;
      } else {
        const int at = U >= 4 ? u % 4 : (kb & 2) + u;
        const uint32_t four = __builtin_amdgcn_ds_bpermute(4 * (4 * col + at), wide[u / 4][i]);
        byte = (four >> (8 * c)) & 0xFFu;
      }
      const float scale = __uint_as_float(byte << 23);
#pragma unroll
      for (int d = 0; d < 4; ++d) f[u].mul(d, dequant8(a[d], scale), acc[i]);
    }
    __builtin_amdgcn_sched_barrier(0);               // and the converted codes of one block at a time
  }
}

// One wave's share: K blocks [kb0, kb1), kb0 a multiple of 4; the sums of token t in the lanes of
// columns F t .. F t + F - 1.  xrow: the rows that this lane loads from, at its element (where there is
// no token, any: a column's sums depend on its own activations only).
template <class TX, bool TILED, int NT, int NC>
__device__ inline void gemv_run(const Tiles<NT>& w, const TX* const (&xrow)[Frag<TX, NC>::S], uint8_t* scratch,
                                int lane, int64_t K, int kb0, int kb1, v4f (&sum)[NT]) {
  constexpr int F = Frag<TX, NC>::F;
  // blocks in flight: without spilled registers (8 instead of 4, or 4 instead of 2, lost more by those
  // than it gained: down of 8 tokens, tiled, 50.5 against 57 us)
  constexpr int U = sizeof(TX) == 4 ? (NT == 1 ? 2 : 1) : NC == 16 ? (NT == 2 ? 1 : 2) : NC == 8 && NT == 2 ? 2 : 4;
  v4f acc[NT][F];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int f = 0; f < F; ++f) acc[i][f] = v4f{0, 0, 0, 0};
  const int whole = (int64_t)kb1 * 128 <= K ? kb1 : kb1 - 1;
  // (untiled, a span has its four scale bytes in every row only where K fills it)
  const int spans = TILED ? whole : (int)(K / 512) * 4 < whole ? (int)(K / 512) * 4 : whole;
  int kb = kb0;
  if constexpr (U > 1)
    for (; kb + U <= spans; kb += U) gemv_step<TX, TILED, NT, NC, U, true, true, false>(w, xrow, scratch, lane, K, kb, U, acc);
  if constexpr (U > 1) {                             // one to three blocks of a span
    if (kb < whole) gemv_step<TX, TILED, NT, NC, U, TILED, false, false>(w, xrow, scratch, lane, K, kb, whole - kb < U ? whole - kb : U, acc);
    kb += U;
  }
  for (; kb < whole; ++kb) gemv_step<TX, TILED, NT, NC, 1, false, true, false>(w, xrow, scratch, lane, K, kb, 1, acc);
  if (!TILED && whole < kb1) gemv_step<TX, TILED, NT, NC, 1, false, true, true>(w, xrow, scratch, lane, K, whole, 1, acc);
  // column F t + f of accumulator f: pick, then add the F columns of each token
  const int mine = lane & (F - 1);
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    v4f v = acc[i][0];
#pragma unroll
    for (int f = 1; f < F; ++f)
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = mine == f ? acc[i][f][r] : v[r];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      if constexpr (F >= 2) v[r] += dpp_move<0xB1>(v[r]);
      if constexpr (F >= 4) v[r] += dpp_move<0x4E>(v[r]);
    }
    sum[i] = v;
  }
}

}  // namespace

// kTileWaves of the kWaves waves share a row tile's K.
template <int MODE, bool TILED, class TX, int NCMAX, int RT, int kWaves, int kTileWaves>
__global__ void __launch_bounds__(kWaves == 16 ? 1024 : 512, 4) gemv_fp4_kernel(GemvArgs a) {
  constexpr int NT = MODE == kSilu ? 2 : RT;         // row tiles: gate and up, or RT one below the other
  __shared__ Items L;
  __shared__ __attribute__((aligned(16))) float part[kWaves][NT][16][16];   // [wave][tile][token][row]
  constexpr bool kXs = stages_activations<TX, NCMAX>();
  constexpr int kScratch = kXs ? kXsBytes : 0;       // a wave's own
  __shared__ __attribute__((aligned(16))) uint8_t scratch[kScratch ? kWaves * kScratch : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, c = lane >> 4;
  int64_t n0 = (int64_t)blockIdx.x * (16 * RT);             // first output column of the tile at work
  const int64_t t0 = (int64_t)blockIdx.z * a.group;
  const int Tn = a.T - t0 < a.group ? (int)(a.T - t0) : a.group;
  const int64_t width = MODE == kSilu ? 2 * a.N : a.N;
  // the waves share the K blocks in spans of four
  const int nkb = (int)((a.K + 127) / 128), spans = (nkb + 3) / 4;
  constexpr int waves = kWaves, tw = kTileWaves, side = waves / tw;
  const TX* x = (const TX*)a.x;
  const bool obf = a.out_bf16;

  const int items = !a.ids              ? 1
                    : Tn * a.k <= 64 ? list_few_items(L, a.ids, t0, Tn * a.k, a.k, a.G)
                                     : list_items(L, a.ids, t0, Tn, a.k, a.G);

  // The tokens of visit p0, one a column: returns their number, and in L.column[wave] which.
  auto columns = [&](int p0) -> int {
    int nc = Tn;
    wave_sync();
    if (!a.ids) {
      if (lane < 16) L.column[wave][lane] = (uint16_t)(lane < Tn ? lane : 0);
    } else {
      // a token has one slot for a visit: the four lanes of its column look for it.  A pair that is named
      // again is a visit of its own.
      const int e = L.ids[p0];
      const bool alone = L.again[p0];
      int mine = -1;
      if (alone) mine = lane == p0 / a.k ? p0 % a.k : -1;
      else if (col < Tn) {
        for (int j = c; j < a.k; j += 4)
          if (L.ids[col * a.k + j] == e && !L.again[col * a.k + j]) mine = j;
      }
      const uint64_t found = __ballot(mine >= 0);
      const uint32_t m = (uint32_t)(found | found >> 16 | found >> 32 | found >> 48) & 0xFFFFu;
      if (mine >= 0) L.column[wave][__popc(m & ((1u << col) - 1))] = (uint16_t)(col + 16 * mine);
      nc = __popc(m);
    }
    wave_sync();
    return nc;
  };
  // K blocks [kb0, kb1) of expert e for the nc tokens of L.column[wave], into sum; returns the number of
  // columns of a token (the t-th one's sums are in the lanes of column t times that)
  auto visit = [&](int e, int nc, int kb0, int kb1, v4f (&sum)[NT]) -> int {
    // (an own copy of the lane's number: what is derived from it for the three column forms is not
    // to be computed once ahead of all visits, where it would fill the registers)
    int lane = tid & 63;
    if constexpr (kXs || (NT == 2 && !TILED)) asm volatile("" : "+v"(lane));
    const int col = lane & 15, c = lane >> 4;
    Tiles<NT> w;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      // (gate and up are N rows apart, tiles of one matrix 16; a tile past the end is the last one again)
      const int64_t up = MODE == kSilu && i ? a.N : 0, r0 = n0 + (MODE == kSilu ? 0 : 16 * i);
      if constexpr (TILED) {
        const int64_t last = a.N / 16 - 1, nb = (r0 / 16 < last ? r0 / 16 : last) + up / 16;
        w.codes[i] = uniform_ptr(a.b + ((int64_t)e * (width / 16) + nb) * (a.K / 128) * 1024);
        w.scales[i] = uniform_ptr(a.s + ((int64_t)e * (width / 16) + nb) * ((a.K + 511) / 512) * 256);
        w.code_lane[i] = 16 * lane;
        w.scale_lane[i] = 16 * col;
        w.byte_lane[i] = 16 * col + c;
      } else {
        const int64_t last = a.N - 1, base = r0 < last ? r0 : last;
        const int rows = (int)(last - base < 15 ? last - base : 15);   // rows past the end: the last one, not stored
        const uint32_t row = lane >> 2 < rows ? lane >> 2 : rows, row_c = col < rows ? col : rows;
        w.codes[i] = uniform_ptr(a.b + ((int64_t)e * width + up + base) * (a.K / 2));
        w.scales[i] = uniform_ptr(a.s + ((int64_t)e * width + up + base) * (a.K / 32));
        w.code_lane[i] = row * (uint32_t)(a.K / 2) + 16 * (lane & 3);
        w.scale_lane[i] = row * (uint32_t)(a.K / 32) + 4 * (lane & 3);
        w.byte_lane[i] = row_c * (uint32_t)(a.K / 32) + c;
      }
    }
    auto go = [&](auto n) -> int {
      using X = Frag<TX, decltype(n)::value>;
      const TX* row[X::S];
#pragma unroll
      for (int s = 0; s < X::S; ++s) {
        const int t = X::token(lane, s), tj = L.column[wave][t < nc ? t : 0];
        const int64_t xr = a.per_slot ? (t0 + (tj & 15)) * a.k + (tj >> 4) : t0 + (tj & 15);
        row[s] = x + xr * a.ldx + X::element(lane);
      }
      gemv_run<TX, TILED, NT, decltype(n)::value>(w, row, scratch + wave * kScratch, lane, a.K, kb0, kb1, sum);
      return X::F;
    };
    using std::integral_constant;
    if constexpr (sizeof(TX) == 4) return go(integral_constant<int, 16>());
    else if constexpr (NCMAX == 4) return go(integral_constant<int, 4>());
    else if (nc <= 4) return go(integral_constant<int, 4>());
    else if (nc <= 8) return go(integral_constant<int, 8>());
    else return go(integral_constant<int, 16>());
  };
  // the sum over a tile's waves, from q0 on, of one value, in wave order
  auto joined = [&](int q0, int i, int t, int r) {
    float v = part[q0][i][t][r];
    for (int q = 1; q < tw; ++q) v += part[q0 + q][i][t][r];
    return v;
  };

  if constexpr (MODE == kSum) {
    // the waves split the K blocks of all visits, expert by expert, and keep their own sums in LDS
    for (int p = tid; p < Tn * a.k; p += blockDim.x) L.gate[p] = a.w[t0 * a.k + p];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NT; ++i) *reinterpret_cast<v4f*>(&part[wave][i][col][4 * c]) = v4f{0, 0, 0, 0};
    const int64_t units = (int64_t)items * spans;
    int64_t at = units * wave / waves;
    const int64_t end = units * (wave + 1) / waves;
    while (at < end) {
      const int it = (int)(at / spans), s0 = (int)(at - (int64_t)it * spans);
      const int s1 = (int)(end - (int64_t)it * spans < spans ? end - (int64_t)it * spans : spans);
      const int p0 = __builtin_amdgcn_readfirstlane(L.item[it]), nc = columns(p0);
      v4f sum[NT];
      const int f = visit(__builtin_amdgcn_readfirstlane(L.ids[p0]), nc, 4 * s0, 4 * s1 < nkb ? 4 * s1 : nkb, sum);
      if (col % f == 0 && col / f < nc) {
        const int tj = L.column[wave][col / f], t = tj & 15;
        const float g = L.gate[t * a.k + (tj >> 4)];
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
      if (t < Tn && n < a.N) put(a.out, obf, (t0 + t) * a.ldo + n, joined(0, i >> 8, t, r));
    }
  } else {
    const int sub = wave / tw, at = wave % tw;         // of the tiles side by side, and of a tile's waves
    const int kb0 = 4 * (int)((int64_t)spans * at / tw), end = 4 * (int)((int64_t)spans * (at + 1) / tw);
    const int kb1 = end < nkb ? end : nkb;
    const int64_t first = (int64_t)blockIdx.x * (16 * side), step = (int64_t)gridDim.x * (16 * side);
    for (int it = blockIdx.y; it < items; it += gridDim.y) {
      const int p0 = a.ids ? __builtin_amdgcn_readfirstlane(L.item[it]) : 0, nc = columns(p0);
      const int e = a.ids ? __builtin_amdgcn_readfirstlane(L.ids[p0]) : 0;
      for (int64_t n = first; n < a.N; n += step) {
        n0 = n + 16 * sub;
        v4f sum[NT];
        const int f = visit(e, nc, kb0, kb1, sum);
        if (col % f == 0) {
#pragma unroll
          for (int i = 0; i < NT; ++i) *reinterpret_cast<v4f*>(&part[wave][i][col / f][4 * c]) = sum[i];
        }
        __syncthreads();
        for (int i = tid; i < 256 * side; i += blockDim.x) {
          const int q0 = (i >> 8) * tw, t = (i >> 4) & 15, r = i & 15;
          const int64_t to = n + 16 * (i >> 8) + r;
          if (t >= nc || to >= a.N) continue;
          float v = joined(q0, 0, t, r);
          if constexpr (MODE == kSilu) v = v / (1.0f + expf(-v)) * joined(q0, 1, t, r);
          const int tj = L.column[wave][t];
          put(a.out, obf, ((t0 + (tj & 15)) * a.k + (tj >> 4)) * a.ldo + to, v);
        }
        __syncthreads();
      }
    }
    if (a.ids && blockIdx.y == 0) {                  // slots without an expert
      for (int p = tid >> 4; p < Tn * a.k; p += blockDim.x >> 4) {
        if (L.ids[p] >= 0) continue;
        for (int64_t n = first; n < a.N; n += step)
          for (int64_t to = n + (tid & 15); to < n + 16 * side && to < a.N; to += 16)
            put(a.out, obf, (t0 * a.k + p) * a.ldo + to, 0.0f);
      }
    }
  }
}

// The forms by what differs in their workgroups: output, row tiles of a wave, waves, waves of a tile (the others
// take tiles beside it), and whether activations are staged (the weights' layout changes neither threads nor LDS).
template <int MODE, int RT, int W, int TW, bool STAGED>
static KernelInfo gemv_form(const char* name) {
  constexpr int kLds = (int)sizeof(Items) + W * 1024 * (MODE == kSilu ? 2 : RT) + (STAGED ? W * kXsBytes : 0);
  return {name, "fgg_moe_gemv_fp4", 16 * RT * (W / TW), 16, 128, 64 * W, 0, 0, kLds, kLds,
          (const void*)gemv_fp4_kernel<MODE, true, uint16_t, STAGED ? 16 : 4, RT, W, TW>};
}
const KernelInfo kInfoGemvFp4[kGemvForms] = {
    gemv_form<kPlain, 1, 8, 8, false>("gemv_fp4_kernel<plain, 8 waves>"),
    gemv_form<kPlain, 1, 8, 8, true>("gemv_fp4_kernel<plain, 8 waves, staged>"),
    gemv_form<kPlain, 1, 4, 4, false>("gemv_fp4_kernel<plain, 4 waves>"),
    gemv_form<kPlain, 1, 4, 4, true>("gemv_fp4_kernel<plain, 4 waves, staged>"),
    gemv_form<kPlain, 1, 4, 2, false>("gemv_fp4_kernel<plain, 4 waves, 2 tiles>"),
    gemv_form<kPlain, 1, 4, 2, true>("gemv_fp4_kernel<plain, 4 waves, 2 tiles, staged>"),
    gemv_form<kPlain, 1, 4, 1, false>("gemv_fp4_kernel<plain, 4 waves, 4 tiles>"),
    gemv_form<kPlain, 1, 4, 1, true>("gemv_fp4_kernel<plain, 4 waves, 4 tiles, staged>"),
    gemv_form<kSilu, 1, 8, 8, false>("gemv_fp4_kernel<silu, 8 waves>"),
    gemv_form<kSilu, 1, 8, 8, true>("gemv_fp4_kernel<silu, 8 waves, staged>"),
    gemv_form<kSilu, 1, 4, 4, false>("gemv_fp4_kernel<silu, 4 waves>"),
    gemv_form<kSilu, 1, 4, 4, true>("gemv_fp4_kernel<silu, 4 waves, staged>"),
    gemv_form<kSilu, 1, 4, 2, false>("gemv_fp4_kernel<silu, 4 waves, 2 tiles>"),
    gemv_form<kSilu, 1, 4, 2, true>("gemv_fp4_kernel<silu, 4 waves, 2 tiles, staged>"),
    gemv_form<kSilu, 1, 4, 1, false>("gemv_fp4_kernel<silu, 4 waves, 4 tiles>"),
    gemv_form<kSilu, 1, 4, 1, true>("gemv_fp4_kernel<silu, 4 waves, 4 tiles, staged>"),
    gemv_form<kSum, 1, 8, 8, false>("gemv_fp4_kernel<sum, 8 waves>"),
    gemv_form<kSum, 1, 8, 8, true>("gemv_fp4_kernel<sum, 8 waves, staged>"),
    gemv_form<kSum, 1, 16, 16, false>("gemv_fp4_kernel<sum, 16 waves>"),
    gemv_form<kSum, 1, 16, 16, true>("gemv_fp4_kernel<sum, 16 waves, staged>"),
    gemv_form<kSum, 2, 16, 16, true>("gemv_fp4_kernel<sum, 16 waves, 2 tiles a wave, staged>"),
};
// The entry of a form above.
static constexpr int gemv_index(int mode, int rt, int waves, int tile_waves, bool staged) {
  if (rt == 2) return kGemvForms - 1;
  const int shape = mode == kSum ? waves == 16 : waves == 8 ? 0 : tile_waves == 4 ? 1 : tile_waves == 2 ? 2 : 3;
  return mode * 8 + shape * 2 + staged;
}

hipError_t launch_gemv_fp4(bool tiled, int32_t G, int64_t T, int32_t k, int64_t N, int64_t K, const void* x,
                           bool x_bf16, int64_t ldx, bool per_slot, const uint8_t* b, const uint8_t* s,
                           const int32_t* ids, const float* w, bool silu, void* out, bool out_bf16, int64_t ldo,
                           int cus, hipStream_t st) {
  // (any count may be set: at most 65535 workgroups where a rule below fills the compute units, the grid's depth)
  const int64_t num_cus = cus < 65535 ? cus : 65535;
  GemvArgs a = {G, T, k, N, K, x, ldx, per_slot, b, s, ids, w, out, out_bf16, ldo, 16};
  const int64_t pairs = (T < 16 ? T : 16) * k;
  const unsigned visits = ids && !w ? (unsigned)(pairs < G ? pairs : G) : 1;
  // The summed form with many tokens: two row tiles a wave (twice the bytes in flight, half the
  // activations' loads) and sixteen waves a workgroup, one of which fills a compute unit.  Down of
  // 16 tokens over 32 experts (N 7168, K 2048), tiled, 57.6 -> 49.3 us, of 8 tokens 46.9 -> 45.3; of one
  // token 15.3 -> 15.5; untiled 16 tokens 64.1 -> 63.4 among other calls, 8 tokens 54.7 -> 59.0.
  const int rt = w && x_bf16 && tiled && T > 4 && (N + 31) / 32 >= num_cus * 3 / 4 ? 2 : 1;
  const int64_t tiles = (N + 16 * rt - 1) / (16 * rt);
  // Waves: a span of 512 K for each, four to K 2048.  To K 4096 four with two spans each do better than eight where the
  // tiles are many (two experts of eight, N 14336, K 4096, tiled: 1 token 18.5 -> 14.6 us, 8 tokens 55.9 -> 48.5)
  // and worse where they are few (one matrix, 4096 rows: 5.1 -> 5.5).  The summed form takes sixteen where there are no
  // more tiles than compute units (N 3328, K 1152, 3 experts, 16 tokens: 12.9 -> 7.6).
  // With a span or two for four waves, two or four tiles side by side, again where the tiles are many (16 tokens, tiled:
  // 10 experts, N 7024, K 256, 16.6 -> 10.0 us, SiLU 20.6 -> 11.7; 25 experts, N 3264, K 640, 22.8 -> 17.3; where they are
  // few, 4 experts, N 320, K 256, 4.8 -> 5.5, SiLU 5.6 -> 6.7).
  const bool many = tiles * visits > 4 * num_cus;
  const bool few_spans = K <= 2048 || (K <= 4096 && many);
  const int waves = w ? (rt == 2 || tiles <= num_cus ? 16 : 8) : few_spans ? 4 : 8;
  // Tokens per workgroup.  The summed form has one workgroup per row tile, which visits every expert of its tokens in
  // turn; where the tiles are few, fewer tokens each leave it fewer activations (a K block of 16 tokens is 4 KB, of a
  // tile 1 KB) and, below four, fewer experts if the tokens choose different ones: as long as every workgroup has a
  // compute unit to itself (with two on each it loses: N 2048, 16 tokens, 26 -> 40 us).  32 experts, top-8, K 2048,
  // tiled: N 512 of 16 tokens 26.1 -> 13.6 us, N 1024 of 4 tokens 16.8 -> 10.1, N 2048 of 8 tokens 24.3 -> 21.3;
  // 10 experts, top-8, groups of two or one instead of four: 10.4 -> 11.1.  (Two row tiles a wave are for many tokens:
  // their kernel has sixteen columns.)
  if (w && x_bf16 && rt == 1)
    for (const int few : {8, 4, 2, 1})
      if (T > few && tiles * ((T + few - 1) / few) <= num_cus && (few >= 4 || G >= 2 * k)) a.group = few;
  // Tiles per workgroup: two workgroups of eight waves fill a compute unit, or four of four waves, and more of them
  // only repeat the start (the list, the first loads).  Gate-up of one token, 8 and 32 experts: 25.1 -> 24.0 and
  // 100 -> 86 us; 8 tokens 129 -> 102; with fewer workgroups the loop would cost 4 us a tile.  Of four waves
  // against two workgroups' worth of tiles: one token's 8 experts, N 2048, K 2048, SiLU, untiled 12.3 -> 10.9.
  const int tile_waves = w || !many || K > 1024 ? waves : K <= 512 ? 1 : 2;
  auto go = [&](auto mode, auto til, auto tx, auto nc) {
    constexpr int M = decltype(mode)::value, NC = decltype(nc)::value;
    constexpr bool TILED = decltype(til)::value;
    using TX = decltype(tx);
    // The grid and the block are those of the kernel that is launched, whatever led to it.
    auto launch = [&](auto row_tiles, auto nwaves, auto ntile) {
      constexpr int RT = decltype(row_tiles)::value, W = decltype(nwaves)::value, TW = decltype(ntile)::value;
      constexpr int kRows = 16 * RT * (W / TW);        // of a workgroup at a time
      const int64_t wide = (N + kRows - 1) / kRows;
      int64_t loop = w ? 1 : wide * visits / ((W == 4 ? 4 : 2) * num_cus);
      loop = loop < 1 ? 1 : loop > 4 ? 4 : loop;
      const dim3 grid((unsigned)((wide + loop - 1) / loop), visits, (unsigned)((T + a.group - 1) / a.group));
      const KernelInfo& info = kInfoGemvFp4[gemv_index(M, RT, W, TW, stages_activations<TX, NC>())];
      trace_launch(info, grid, "G=%d T=%lld k=%d N=%lld K=%lld %s %s->%s", (int)G, (long long)T, (int)k, (long long)N,
                   (long long)K, tiled ? "tiled" : "rows", x_bf16 ? "bf16" : "fp32", out_bf16 ? "bf16" : "fp32");
      hipLaunchKernelGGL((gemv_fp4_kernel<M, TILED, TX, NC, RT, W, TW>), grid, dim3(64 * W), 0, st, a);
    };
    constexpr std::integral_constant<int, 1> n1;
    constexpr std::integral_constant<int, 2> n2;
    constexpr std::integral_constant<int, 4> n4;
    constexpr std::integral_constant<int, 8> n8;
    constexpr std::integral_constant<int, 16> n16;
    if constexpr (M == kSum) {
      if constexpr (TILED && sizeof(TX) == 2 && NC == 16)
        if (rt == 2) return launch(n2, n16, n16);
      if (waves == 16) return launch(n1, n16, n16);
    } else {
      if (tile_waves == 1) return launch(n1, n4, n1);
      if (tile_waves == 2) return launch(n1, n4, n2);
      if (waves == 4) return launch(n1, n4, n4);
    }
    launch(n1, n8, n8);
  };
  using std::integral_constant;
  auto with_type = [&](auto mode, auto til) {
    if (!x_bf16) return go(mode, til, float(), integral_constant<int, 16>());
    if (T <= 4 || a.group <= 4) return go(mode, til, uint16_t(), integral_constant<int, 4>());
    go(mode, til, uint16_t(), integral_constant<int, 16>());
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
