// bf16 products of row segments with their segment's weights (gfx950): the linear layer
// of an expert layer, its two gradients, and the gated block with its gradient.
//
//   linear     y[r][n]  = sum_k x[r][k] W_g[n][k]                        r in segment g
//   gated      h = the same with W_g = [gate | up];  a = silu(h_gate) h_up
//   rows'      dx[r][k] = sum_n dy[r][n] W_g[n][k]
//   gated back da[r][i] = sum_n dy[r][n] Wd_g[n][i];  dgate = da up s (1 + gate (1 - s)),
//              dup = da gate s, a = gate s up,  s = 1 / (1 + e^-gate)
//   weights'   dW_g[n][k] = sum_r dy[r][n] x[r][k]                       over segment g
//
// All five are one tiled product C[m][n] = sum_c P[m][c] Q[n][c] whose operands lie in memory
// either with the summed index along the row ("row") or across the rows ("col"):
// linear and gated row x row, the rows' gradients row x col, the weights' gradient col x col.
//
// gfx950 mapping:
//  * v_mfma_f32_16x16x32_bf16 with the n operand first, so a lane holds four consecutive columns of
//    one row; fp32 accumulators, rounded once.
//  * three workgroup shapes, chosen by an estimate (plan_rows, plan_dw).  Large: 256 x 256 outputs, 64 deep,
//    8 waves (two per SIMD) of 128 x 64, two LDS stages of 64 KB; per 64 deep a wave reads 24 KB of LDS for
//    64 MFMAs, which is what the LDS delivers in the MFMAs' time.  8192^3: 802 us, 1.37 PFLOP/s (row x row;
//    row x col and col x col within 4 %; the library's product 681 us).  Medium: 128 x 128 by 4 waves, two workgroups per compute unit, for
//    tiles that would not fill the chip.  Small: 64 x 64, four stages, where time is the sum's latency or
//    the weights' bytes (16 rows onto 16384 columns, sum 4096: 21 us, 6.4 TB/s).
//  * stages are filled by buffer loads straight into LDS, the next one's issued before the current one is
//    computed.  A buffer descriptor's range check writes zeros for what lies outside (rows past the
//    segment, columns past the edge, the end of the sum), so ragged sizes cost no branch in the loop
//    and what lies there never enters a product.
//  * "row" tiles: LDS rows of the tile's depth, 16-byte chunks mixed by row (row_key) so that the sixteen
//    lanes that one cycle of a ds_read_b128 serves hit sixteen different chunks.  "col" tiles: LDS rows of
//    the tile's outputs for one summed index, read by ds_read_b64_tr_b16, which turns 4 x 16 blocks in the
//    read; 32-byte units mixed by row (col_key).
//  * a tile's segment is found by a scan over the segments' row counts in each wave's lanes (no table, no
//    workspace).  Workgroups are dealt to the 8 XCDs in turn, and 32 consecutive tiles (8 high, 4 wide)
//    go to one XCD, whose L2 then holds what they share.
//  * what bounds the Large shape: the matrix cores at the clock that the card holds under them, and writing:
//    without its stores the weights' gradient of 8 x 14336 x 4096 in fp32 (1.9 GB) takes 775 us instead of
//    1170 (bf16 results: 961), in every shape alike: a tile's first stages wait for the last one's stores, which share
//    their counter.  Where segments are a few tiles high, a tile at most half full of rows is a whole turn of its
//    compute unit though it does half the products.
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_segments.hpp"

namespace fgg {

namespace {

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

constexpr int kXcds = 8, kSM = 8, kChunk = 32;           // tiles of one XCD at a time: 8 high, 4 wide
constexpr uint32_t kOutside = 0x80000000u;               // offset that the range check rejects

constexpr int BK = 64;                                   // depth of a stage

// A workgroup's shape: M x N outputs by WM x WN waves, STAGES buffers.
template <int M_, int N_, int WM_, int WN_, int STAGES_>
struct Shape {
  static constexpr int M = M_, N = N_, WM = WM_, WN = WN_, kStages = STAGES_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr bool kPersistent = kWaves == 8;
  static constexpr int FI = M / WM / 16, FJ = N / WN / 16;     // a wave's 16 x 16 accumulators
  static constexpr int kPBytes = M * BK * 2, kQBytes = N * BK * 2;
  static constexpr int kQOff = kStages * kPBytes;              // LDS: P stages, then Q stages
  static constexpr int kStageBytes = kPBytes + kQBytes, kLdsBytes = kStages * kStageBytes;
  static constexpr int kPDma = kPBytes / 1024 / kWaves, kQDma = kQBytes / 1024 / kWaves;   // 1 KB loads per wave
};
using Large = Shape<256, 256, 2, 4, 2>;
using Medium = Shape<128, 128, 2, 2, 2>;
using Small = Shape<64, 64, 2, 2, 4>;
using Quarter = Shape<128, 128, 2, 4, 4>;            // of a Large tile, by its eight waves
static_assert(Quarter::kThreads == Large::kThreads && Quarter::kLdsBytes <= Large::kLdsBytes, "one workgroup");

// "row" tiles (128-byte LDS rows): the 16-byte chunk c of row r lies at chunk c ^ row_key(r), such that the sixteen
// lanes that one cycle of a ds_read_b128 serves (rows 0..3 and 12..15 of one chunk, 4..11 of the next) hit
// different chunks.
__device__ inline int row_key(int r) { return r & 7; }

enum Form { kLinear, kGated, kDx, kGatedBwd, kDw, kAdapters };
constexpr bool p_is_col(int f) { return f == kDw; }
constexpr bool q_is_col(int f) { return f == kDx || f == kGatedBwd || f == kDw; }

// The value of x, hidden from the optimizer: what is derived from it in a tile's beginning or end is computed
// there instead of being held (or spilled) across the K loop.
__device__ inline int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// N times 16 bytes per lane, from base + voff[i] into LDS at lds + 1024 i + 16 * lane; zeros where voff is kOutside.
// (The wait states after the writes of M0 and of the descriptor as in dma16; M0 is saved and restored once: with
// N loads apart, 8192 rows of 8 segments, 14336 -> 4096, took 919 us instead of 863.)
template <int N>
__device__ inline void buf_dma16(const void* base, const uint32_t* voff, uint32_t lds) {
  static_assert(N == 2 || N == 4, "loads of one asm");
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const v4i rs = {__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                  __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32) & 0xFFFF), (int)0x80000000u, 0x00020000};
  const uint32_t at = __builtin_amdgcn_readfirstlane(lds);
  uint32_t save;
#define FGG_FIRST(v) "s_mov_b32 %0, m0\n\ts_mov_b32 m0, %2\n\ts_nop 2\n\tbuffer_load_dwordx4 " v ", %1, 0 offen lds\n\t"
#define FGG_NEXT(v) "s_addk_i32 m0, 0x400\n\ts_nop 0\n\tbuffer_load_dwordx4 " v ", %1, 0 offen lds\n\t"
  if constexpr (N == 2)
    asm volatile(FGG_FIRST("%3") FGG_NEXT("%4") "s_mov_b32 m0, %0"
                 : "=&s"(save)
                 : "s"(rs), "s"(at), "v"(voff[0]), "v"(voff[1])
                 : "memory", "scc");
  else
    asm volatile(FGG_FIRST("%3") FGG_NEXT("%4") FGG_NEXT("%5") FGG_NEXT("%6") "s_mov_b32 m0, %0"
                 : "=&s"(save)
                 : "s"(rs), "s"(at), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3])
                 : "memory", "scc");
#undef FGG_FIRST
#undef FGG_NEXT
}

// "col" tiles hold W outputs a row, in 32-byte units; the key that unit numbers of row c are mixed with, such
// that the eight rows that 32 lanes read (0..3 and 8..11 from a multiple of 4) lie in different banks.
template <int W>
__device__ inline int col_key(int c) {
  return W == 64 ? ((c >> 1) & 1) | ((c >> 3) & 1) << 1 : (c & 3) | ((c >> 3) & 1) << 2;
}

// Eight consecutive summed indices of one output from a "col" tile: two 4 x 16 blocks, 4 rows apart.
template <int W>
__device__ inline v8bf tr_read(const uint8_t* p) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * W * 2));
  const v8s v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(v8bf, v);
}

}  // namespace

// (see launch_* below for what each form passes)
struct BfArgs {
  const uint16_t *p, *q;
  int64_t ldp, ldq, q_rows;            // row strides; rows of one segment's weights
  const int32_t *offsets, *counts;
  int G;
  int64_t M, m_cols, n_cols, sum;      // rows; output rows (kDw) and columns; length of the sum (not kDw)
  int n_tiles, m_tiles;                // tiles across; tiles down one segment (kDw)
  void* out;
  int64_t ldo;
  uint16_t* out2;                      // kGated: pre-activations; kGatedBwd: activation; or null
  int64_t ldo2;
  const uint16_t* h;                   // kGatedBwd: pre-activations
  int64_t ldh;
  int out_f32, accumulate;
  int chunk;                           // consecutive tiles of one XCD
  int num_cus;
  int splits;                          // kDw: parts of the sum, each with its own fp32 result
  const int32_t* ids;                  // kAdapters: the rows' adapters,
  int shift;                           // and the columns of one of them in a tile, 2^shift
};

namespace {

// Stages of a sum (0 to 2^31 - 1: rounded up in 32 bits without a sign).
__host__ __device__ constexpr int stages_of(int sum) { return (int)(((uint32_t)sum + BK - 1) / BK); }

// Part z of `splits` of the sum over a segment's rows, in whole stages.
struct Part {
  int first, rows;
};
__host__ __device__ constexpr Part part_of(int rows, int splits, int z) {
  const uint32_t per = (uint32_t)((stages_of(rows) + splits - 1) / splits) * BK;     // (2^31 at most)
  const int64_t first = (int64_t)per * z < rows ? (int64_t)per * z : rows;
  return {(int)first, (int)(rows - first < per ? rows - first : per)};
}
static_assert(part_of(INT32_MAX, 1, 0).rows == INT32_MAX && stages_of(INT32_MAX) == 1 << 25, "the longest sum");
static_assert(part_of(INT32_MAX, 32, 31).first + part_of(INT32_MAX, 32, 31).rows == INT32_MAX, "its last part");
static_assert(part_of(0, 32, 5).rows == 0 && part_of(65, 3, 1).rows == 1 && part_of(65, 3, 2).rows == 0, "short sums");

// (equal in every lane: kept in a scalar register)
__device__ inline int same(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t same(int64_t v) {
  return (int64_t)((uint64_t)(uint32_t)same((int)(v >> 32)) << 32 | (uint32_t)same((int)v));
}

// A tile: where it lies, and how long its sum is.
struct Tile {
  int64_t p_row, q_row, out_row;     // first row of P and Q (of the sum, for "col" operands), of the output
  int m0, n0, m_here, n_here, sum;   // first output row and column in the segment's result; what is left from there
  int slot[4];                       // kAdapters: the adapters side by side in the tile, -1 for none
};

__device__ inline int slot_of(const Tile& t, int i) {
  return i == 0 ? t.slot[0] : i == 1 ? t.slot[1] : i == 2 ? t.slot[2] : t.slot[3];
}

// Tiles of height BM that a segment takes (0 to 2^31 - 1 rows: rounded up without a sign).
template <int BM>
__device__ inline int tiles_down(int rows) {
  return (int)(((uint32_t)rows + BM - 1) / BM);
}

// Tiles of the whole launch (kMaxBf16Tiles at most, also where offsets fall and segments overlap).
template <int F, class S>
__device__ inline int count_tiles(const BfArgs& A) {
  if (F == kDw) return A.splits * A.G * A.m_tiles * A.n_tiles;
  if (A.offsets == nullptr) return tiles_down<S::M>((int)A.M) * A.n_tiles;
  const int lane = threadIdx.x & 63, most = (int)(kMaxBf16Tiles / A.n_tiles);
  int n = 0;
  for (int g = lane; g < A.G; g += 64) {
    n += tiles_down<S::M>(segment_of(A.offsets, A.counts, g, A.M).rows);
    if (n > most) n = most;
  }
  for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d);
  n = same(n);
  return (n < most ? n : most) * A.n_tiles;
}

// Tile t of the launch, segment by segment, in blocks 8 high; false past the last one.
template <int F, class S>
__device__ inline bool find_tile(const BfArgs& A, int t, Tile& tile) {
  constexpr int BM = S::M, BN = S::N;
  const int lane = opaque(threadIdx.x & 63);
  int g = 0, j = t, z = 0, mtg = A.m_tiles;
  Segment seg;
  if constexpr (F == kDw) {
    const int each = A.m_tiles * A.n_tiles;
    z = t / (A.G * each);
    if (z >= A.splits) return false;
    j = t - z * (A.G * each);
    g = j / each;
    j -= g * each;
    seg = A.offsets ? segment_of(A.offsets, A.counts, g, A.M) : Segment{0, (int)A.M};
  } else if (A.offsets == nullptr) {
    seg = {0, (int)A.M};
    mtg = tiles_down<BM>(seg.rows);
    if (t >= mtg * A.n_tiles) return false;
  } else {
    uint32_t before = 0;                 // (at most t; the 64 segments after it have less than 2^31 tiles)
    bool found = false;
    for (int g0 = 0; g0 < A.G; g0 += 64) {
      Segment mine = {0, 0};
      if (g0 + lane < A.G) mine = segment_of(A.offsets, A.counts, g0 + lane, A.M);
      const int tiles = tiles_down<BM>(mine.rows) * A.n_tiles;
      int upto = tiles;
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      const uint64_t hit = __ballot(before + upto > (uint32_t)t);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        g = g0 + at;
        j = t - (int)before - (__builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(tiles, at));
        seg.first = __builtin_amdgcn_readlane((int)mine.first, at);
        seg.rows = __builtin_amdgcn_readlane(mine.rows, at);
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (!found) return false;
    mtg = tiles_down<BM>(seg.rows);
  }
  const int mb = j / (kSM * A.n_tiles), k_in = j - mb * kSM * A.n_tiles;
  const int high = mtg - mb * kSM < kSM ? mtg - mb * kSM : kSM;
  const int nt = k_in / high;
  tile.m0 = (mb * kSM + k_in - nt * high) * BM;
  tile.n0 = nt * (F == kGated ? BN / 2 : BN);
  tile.n_here = (int)A.n_cols - tile.n0;
  if constexpr (F == kDw) {
    const Part part = part_of(seg.rows, A.splits, z);
    tile.sum = part.rows;
    tile.m_here = (int)A.m_cols - tile.m0;
    tile.p_row = tile.q_row = seg.first + part.first;
    tile.out_row = ((int64_t)z * A.G + g) * A.m_cols + tile.m0;
  } else {
    tile.sum = (int)A.sum;
    tile.m_here = seg.rows - tile.m0;
    tile.p_row = tile.out_row = seg.first + tile.m0;
    tile.q_row = (int64_t)g * A.q_rows + (q_is_col(F) ? 0 : tile.n0);
  }
  tile = {same(tile.p_row), same(tile.q_row), same(tile.out_row), same(tile.m0),
          same(tile.n0),    same(tile.m_here), same(tile.n_here), same(tile.sum), {}};
  return true;
}

// Quadrant `quad` of a tile twice as high and wide as S; false where it holds nothing.
template <int F, class S>
__device__ inline bool quarter(Tile& t, int quad) {
  const int down = (quad >> 1) * S::M, across = (quad & 1) * (F == kGated ? S::N / 2 : S::N);
  if (down >= t.m_here || across >= t.n_here) return false;
  t.m0 += down;
  t.m_here -= down;
  t.out_row += down;
  if (!p_is_col(F)) t.p_row += down;
  t.n0 += across;
  t.n_here -= across;
  if (!q_is_col(F)) t.q_row += across;
  return true;
}

// Tiles of shape S, one after the other, as `source` gives them (round 0, 1, ...; false: no more).  The next
// tile's first stages are loaded while the epilogue of the last one writes.
template <int F, class S, class Source>
__device__ __forceinline__ void run_tiles(const BfArgs& A, uint8_t* smem, Source source) {
  constexpr int BM = S::M, BN = S::N, FI = S::FI, FJ = S::FJ;
  const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / S::WN, wn = wave % S::WN;
  const int l16 = lane & 15, q = lane >> 4;

  // What this wave loads: 1 KB pieces of both tiles; byte offsets from P and Q, kOutside past an edge.
  // "row": a piece is 1 KB of rows of BK elements; this lane's row in it and its chunk's place in memory
  const int r_chunk = (lane % (BK / 8)) ^ row_key(lane / (BK / 8));
  // "col": a piece is 1 KB of rows of W outputs; this lane's row in it (and, in begin, its first output)
  auto c_row = [&](int W, int piece) { return piece * (512 / W) + lane / (W / 8); };
  uint32_t voff_p[S::kPDma], voff_q[S::kQDma];
  const uint16_t *P, *Q;
  int sum, nk;
  auto begin = [&](const Tile& t) {
    const int lane = opaque(threadIdx.x & 63);
    const int r_row = lane / (BK / 8), r_chunk = (lane % (BK / 8)) ^ row_key(r_row);
    auto c_row = [&](int W, int piece) { return piece * (512 / W) + lane / (W / 8); };
    auto c_col = [&](auto w_tag, int piece) {
      constexpr int W = decltype(w_tag)::value;
      const int in = lane % (W / 8);
      return ((in >> 1) ^ col_key<W>(c_row(W, piece))) * 16 + (in & 1) * 8;
    };
    sum = t.sum;
    nk = stages_of(sum);
    P = A.p + t.p_row * A.ldp + (p_is_col(F) ? t.m0 : 0);
    Q = A.q + t.q_row * A.ldq + (q_is_col(F) ? t.n0 : 0);
    // (gated: the second half of the waves loads the up rows, n_cols rows further)
    if (F == kGated && wave >= S::kWaves / 2) Q += A.n_cols * A.ldq;
#pragma unroll
    for (int i = 0; i < S::kPDma; ++i) {
      const int piece = wave * S::kPDma + i;
      if constexpr (p_is_col(F)) {
        const int c = c_col(std::integral_constant<int, BM>{}, piece);
        voff_p[i] = c < t.m_here ? (uint32_t)c_row(BM, piece) * (uint32_t)(A.ldp * 2) + c * 2 : kOutside;
      } else {
        const int row = piece * (512 / BK) + r_row;
        voff_p[i] = row < t.m_here ? (uint32_t)row * (uint32_t)(A.ldp * 2) + r_chunk * 16 : kOutside;
      }
    }
#pragma unroll
    for (int i = 0; i < S::kQDma; ++i) {
      const int piece = wave * S::kQDma + i;
      if constexpr (q_is_col(F)) {
        const int c = c_col(std::integral_constant<int, BN>{}, piece);
        voff_q[i] = c < t.n_here ? (uint32_t)c_row(BN, piece) * (uint32_t)(A.ldq * 2) + c * 2 : kOutside;
      } else {
        int row = piece * (512 / BK) + r_row;
        if (F == kGated) row &= BN / 2 - 1;  // tile rows: gate columns, then the up columns of the same index
        if constexpr (F == kAdapters) {
          const int slot = slot_of(t, piece * (512 / BK) >> A.shift);
          row &= (1 << A.shift) - 1;
          const uint32_t at = (uint32_t)(A.shift == 6 ? row : slot * (int)A.q_rows + row) * (uint32_t)(A.ldq * 2);
          voff_q[i] = slot >= 0 && row < t.n_here ? at + r_chunk * 16 : kOutside;
          continue;
        }
        voff_q[i] = row < t.n_here ? (uint32_t)row * (uint32_t)(A.ldq * 2) + r_chunk * 16 : kOutside;
      }
    }
  };
  auto issue = [&](int kb, int stage) {
    const uint16_t* p = P + (p_is_col(F) ? (int64_t)kb * BK * A.ldp : (int64_t)kb * BK);
    const uint16_t* qq = Q + (q_is_col(F) ? (int64_t)kb * BK * A.ldq : (int64_t)kb * BK);
    const int rest = sum - kb * BK;
    uint32_t vp[S::kPDma], vq[S::kQDma];
#pragma unroll
    for (int i = 0; i < S::kPDma; ++i) {
      vp[i] = voff_p[i];                   // (the sum's end: zeros)
      if (rest < BK && (p_is_col(F) ? c_row(BM, wave * S::kPDma + i) : r_chunk * 8) >= rest) vp[i] = kOutside;
    }
    buf_dma16<S::kPDma>(p, vp, lds_base + stage * S::kPBytes + wave * S::kPDma * 1024);
#pragma unroll
    for (int i = 0; i < S::kQDma; ++i) {
      vq[i] = voff_q[i];
      if (rest < BK && (q_is_col(F) ? c_row(BN, wave * S::kQDma + i) : r_chunk * 8) >= rest) vq[i] = kOutside;
    }
    buf_dma16<S::kQDma>(qq, vq, lds_base + S::kQOff + stage * S::kQBytes + wave * S::kQDma * 1024);
  };
  constexpr int kFirst = FJ == 4 ? S::kStages : S::kStages - 1;   // stages under way when a tile begins
  auto start = [&]() {
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      if (i < nk) issue(i, i);
  };

  Tile cur;
  if (same((int)source(0, cur)) == 0) return;
  begin(cur);
  start();

  // this lane's operand reads: "row": chunk 4 s + q of row l16 (+ 16 per fragment); "col": rows
  // 8 q + (l16 >> 2) (+ 4 for the second half), the fragment's 32-byte unit
  const int c_line = 8 * q + (l16 >> 2);
  auto read_p = [&](int stage, int s, int i) -> v8bf {
    const uint8_t* base = smem + stage * S::kPBytes;
    if constexpr (p_is_col(F)) {
      const uint32_t at = c_line * (BM * 2) + (l16 & 3) * 8 + (((S::WM * i + wm) ^ col_key<BM>(c_line)) << 5);
      return tr_read<BM>(base + at + s * 32 * BM * 2);
    } else {
      // (fragments go to the waves in turn, so that a part-filled tile is spread over them)
      const int at = (16 * wm + l16) * (BK * 2) + (((4 * s + q) ^ row_key(l16)) << 4);
      return *reinterpret_cast<const v8bf*>(base + at + i * (S::WM * 16 * BK * 2));
    }
  };
  auto read_q = [&](int stage, int s, int n) -> v8bf {
    const uint8_t* base = smem + S::kQOff + stage * S::kQBytes;
    if constexpr (q_is_col(F)) {
      const uint32_t at = c_line * (BN * 2) + (l16 & 3) * 8 + (((FJ * wn + n) ^ col_key<BN>(c_line)) << 5);
      return tr_read<BN>(base + at + s * 32 * BN * 2);
    } else {
      constexpr int kHalf = FJ / 2;
      const int row = (F == kGated ? 16 * kHalf : 16 * FJ) * wn + l16;
      const int further = F == kGated ? n % kHalf * 16 + n / kHalf * (BN / 2) : 16 * n;
      const int at = row * (BK * 2) + (((4 * s + q) ^ row_key(l16)) << 4);
      return *reinterpret_cast<const v8bf*>(base + at + further * (BK * 2));
    }
  };

  for (int round = 1;; ++round) {
    Tile next;
    const bool more = same((int)source(round, next)) != 0;
    v4f acc[FI][FJ];
#pragma unroll
    for (int i = 0; i < FI; ++i)
#pragma unroll
      for (int n = 0; n < FJ; ++n) acc[i][n] = v4f{0.f, 0.f, 0.f, 0.f};

    if constexpr (FJ == 4) {
      // One stage: NG groups (two 32-deep steps x row fragments) of 4 MFMAs.  A group's row fragment is read
      // two groups ahead, the column fragments of the second step during the first.  Two groups before the
      // end every fragment of the stage has been read: there the next stage's loads are awaited, the
      // waves meet, the stage kStages further goes into this stage's buffers, and the last two groups read
      // the next stage's first fragments, so that the matrix cores have work while those reads run.  The
      // order is pinned.  NI: row fragments of each wave that hold rows (a Large tile that is at most half
      // full does half the work).
      constexpr int kAhead = S::kStages - 1;
      v8bf fp[3], fq[2][4];
      auto step = [&](auto ni_tag, auto no_tag, int kb) {
        constexpr int NI = decltype(ni_tag)::value, NG = 2 * NI;
        constexpr int NO = decltype(no_tag)::value;        // kb mod 6
        constexpr int ST = NO % S::kStages, NEXT = (NO + 1) % S::kStages;
        constexpr int R = NO * NG % 3;                     // place of the stage's first row fragment in fp
        constexpr int kFirstQ = NI == 8 ? 3 : 0;           // group of the second step's first column fragment
#pragma unroll
        for (int gi = 0; gi < NG; ++gi) {
          const int s = gi / NI, i = gi % NI;
          if (gi == NG - 2) {
            __builtin_amdgcn_s_waitcnt(kLgkmZero);
            if (kb + kAhead < nk) wait_vmcnt<(kAhead - 1) * (S::kPDma + S::kQDma)>();
            else wait_vmcnt<0>();
            block_barrier();
            if (kb + S::kStages < nk) issue(kb + S::kStages, ST);
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[s][n], fp[(R + gi) % 3], acc[i][n], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            const int ahead = gi + 2;                       // (of the next stage in the last two groups)
            if (n == 0 && ahead < NG) fp[(R + ahead) % 3] = read_p(ST, ahead / NI, ahead % NI);
            if (n == 0 && ahead >= NG) fp[(R + ahead) % 3] = read_p(NEXT, 0, ahead - NG);
            if (n == 2 && gi >= kFirstQ && gi < kFirstQ + 4) fq[1][gi - kFirstQ] = read_q(ST, 1, gi - kFirstQ);
            if ((n == 1 || n == 3) && gi >= NG - 2) {
              const int k = 2 * (gi - NG + 2) + (n >> 1);
              fq[0][k] = read_q(NEXT, 0, k);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      };
      auto run = [&](auto ni_tag) {
#pragma unroll
        for (int n = 0; n < 4; ++n) fq[0][n] = read_q(0, 0, n);
        fp[0] = read_p(0, 0, 0), fp[1] = read_p(0, 0, 1);
        for (int kb = 0; kb < nk; kb += 6) {
          step(ni_tag, std::integral_constant<int, 0>{}, kb);
          if (kb + 1 < nk) step(ni_tag, std::integral_constant<int, 1>{}, kb + 1);
          if (kb + 2 < nk) step(ni_tag, std::integral_constant<int, 2>{}, kb + 2);
          if (kb + 3 < nk) step(ni_tag, std::integral_constant<int, 3>{}, kb + 3);
          if (kb + 4 < nk) step(ni_tag, std::integral_constant<int, 4>{}, kb + 4);
          if (kb + 5 < nk) step(ni_tag, std::integral_constant<int, 5>{}, kb + 5);
        }
      };
      if (nk > 0) {
        // (after the first tile the last one's stores are in the count too: all of it is awaited)
        if (nk >= S::kStages && round == 1) wait_vmcnt<kAhead * (S::kPDma + S::kQDma)>();
        else wait_vmcnt<0>();
        block_barrier();
        if (FI == 8 && cur.m_here <= BM / 2) run(std::integral_constant<int, 4>{});
        else run(std::integral_constant<int, FI>{});
      }
    } else {
      // The smaller shapes: kStages - 1 stages in flight, several workgroups on a compute unit cover each
      // other's waits.
      constexpr int kAhead = S::kStages - 1;
      auto compute = [&](int stage) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          v8bf fq[FJ], fp[FI];
#pragma unroll
          for (int n = 0; n < FJ; ++n) fq[n] = read_q(stage, s, n);
#pragma unroll
          for (int i = 0; i < FI; ++i) fp[i] = read_p(stage, s, i);
#pragma unroll
          for (int i = 0; i < FI; ++i)
#pragma unroll
            for (int n = 0; n < FJ; ++n)
              acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[n], fp[i], acc[i][n], 0, 0, 0);
        }
      };
      for (int kb = 0; kb < nk; kb += S::kStages) {
#pragma unroll
        for (int st = 0; st < S::kStages; ++st) {
          if (kb + st >= nk) break;
          // this stage has landed for every wave, and every wave has read the one before
          __builtin_amdgcn_s_waitcnt(kLgkmZero);
          if (kb + st + kAhead <= nk) wait_vmcnt<(kAhead - 1) * (S::kPDma + S::kQDma)>();
          else wait_vmcnt<0>();
          block_barrier();
          if (kb + st + kAhead < nk) issue(kb + st + kAhead, (st + kAhead) % S::kStages);
          compute(st);
        }
      }
    }

    if (more) {
      // (pinned order: the last stage's barrier has passed, every buffer is free)
      if (FJ != 4) {
        __builtin_amdgcn_s_waitcnt(kLgkmZero);
        block_barrier();
      }
      begin(next);
      start();
    }

    // Outputs.  A lane holds columns 4 q + (0..3) of each fragment for row l16; two neighbouring fragments are
    // exchanged between lanes 16 apart, so that it holds eight consecutive ones (V) of one of them.
    constexpr int kAcross = F == kGated ? FJ / 2 : FJ, V = kAcross % 2 == 0 ? 8 : 4;
    const int lane_e = opaque(lane), l16_e = lane_e & 15, q_e = lane_e >> 4;
    const int c_lane = V == 8 ? 16 * (q_e & 1) + 8 * (q_e >> 1) : 4 * q_e;
    auto gather = [&](int i, int n, float* v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (V == 8) {
          const uint32_t a = __float_as_uint(acc[i][n][e]), b = __float_as_uint(acc[i][n + 1][e]);
          const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
          v[e] = __uint_as_float(r[0]), v[4 + e] = __uint_as_float(r[1]);
        } else {
          v[e] = acc[i][n][e];
        }
      }
    };
    auto put = [&](void* base, int64_t at, const float* v) {      // V values in bf16
      uint32_t w[V / 2];
#pragma unroll
      for (int e = 0; e < V / 2; ++e) w[e] = bf16x2_rne(v[2 * e], v[2 * e + 1]);
      __builtin_memcpy(__builtin_assume_aligned((uint16_t*)base + at, 2 * V), w, 2 * V);
    };
    struct Packed {                      // V bf16 values
      uint32_t w[V / 2];
    };
    auto fetch = [&](const void* base, int64_t at) {
      Packed p;
      __builtin_memcpy(p.w, __builtin_assume_aligned((const uint16_t*)base + at, 2 * V), 2 * V);
      return p;
    };
    auto unpack = [&](const Packed& p, float* v) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = __uint_as_float(e & 1 ? p.w[e / 2] & 0xFFFF0000u : p.w[e / 2] << 16);
    };
    // gated_backward: the pre-activations of kDeep row fragments are under way, where the registers hold them (in a
    // Large tile they would spill: 538 -> 585 us for 8192 rows of 8 segments, 4096 -> 7168)
    constexpr int kDeep = F != kGatedBwd || FI == 8 ? 1 : FI < 3 ? FI : 3, kPieces = kAcross / (V / 4);
    Packed pre[kDeep][kPieces][2];
    auto fetch_pre = [&](int i) {
      const int r = 16 * (S::WM * i + wm) + l16_e;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        const int c = 16 * (kAcross * wn + k * (V / 4)) + c_lane;
        if (r < cur.m_here && c < cur.n_here) {
          const int64_t at = (cur.out_row + r) * A.ldh + cur.n0 + c;
          pre[i % kDeep][k][0] = fetch(A.h, at);
          pre[i % kDeep][k][1] = fetch(A.h, at + A.n_cols);
        }
      }
    };
    if constexpr (kDeep > 1) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) fetch_pre(i);
    }
#pragma unroll
    for (int i = 0; i < FI; ++i) {
      const int r = 16 * (S::WM * i + wm) + l16_e;
      const int64_t row = cur.out_row + r;
#pragma unroll
      for (int n = 0; n < kAcross; n += V / 4) {
        if (F != kGated && F != kGatedBwd && A.out_f32) {
          // four fp32 values are a lane's 16 bytes already
#pragma unroll
          for (int k = 0; k < V / 4; ++k) {
            const int c = 16 * (kAcross * wn + n + k) + 4 * q_e;
            if constexpr (F == kAdapters) {
              const int j = c & ((1 << A.shift) - 1), slot = slot_of(cur, 16 * (kAcross * wn + n + k) >> A.shift);
              if (r >= cur.m_here || j >= cur.n_here || slot < 0 || A.ids[row] != slot) continue;
              const v4f a = acc[i][n + k];
              float4* o = reinterpret_cast<float4*>((float*)A.out + row * A.ldo + cur.n0 + j);
              *o = make_float4(a[0], a[1], a[2], a[3]);
              continue;
            }
            if (r >= cur.m_here || c >= cur.n_here) continue;
            float4* o = reinterpret_cast<float4*>((float*)A.out + row * A.ldo + cur.n0 + c);
            const v4f a = acc[i][n + k];
            float4 w = make_float4(a[0], a[1], a[2], a[3]);
            if (F == kDw && A.accumulate) {
              const float4 old = *o;
              w.x += old.x, w.y += old.y, w.z += old.z, w.w += old.w;
            }
            *o = w;
          }
          continue;
        }
        const int c = 16 * (kAcross * wn + n) + c_lane;
        float v[V];
        gather(i, n, v);                 // (every lane takes part)
        float u[V];
        if constexpr (F == kGated) gather(i, n + FJ / 2, u);
        if (r >= cur.m_here || c >= cur.n_here) continue;
        const int64_t at = row * A.ldo + cur.n0 + c;
        if constexpr (F == kGated) {
          if (A.out2) {
            put(A.out2, row * A.ldo2 + cur.n0 + c, v);
            put(A.out2, row * A.ldo2 + cur.n0 + c + A.n_cols, u);
          }
#pragma unroll
          for (int e = 0; e < V; ++e) v[e] = v[e] * sigmoid(v[e]) * u[e];
          put(A.out, at, v);
        } else if constexpr (F == kGatedBwd) {
          float gate[V], up[V], dg[V];
          if constexpr (kDeep == 1) {
            const int64_t from = row * A.ldh + cur.n0 + c;
            pre[0][0][0] = fetch(A.h, from);
            pre[0][0][1] = fetch(A.h, from + A.n_cols);
          }
          unpack(pre[i % kDeep][kDeep == 1 ? 0 : n / (V / 4)][0], gate);
          unpack(pre[i % kDeep][kDeep == 1 ? 0 : n / (V / 4)][1], up);
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float s = sigmoid(gate[e]), silu = gate[e] * s;
            dg[e] = v[e] * up[e] * fmaf(silu, 1.0f - s, s);
            v[e] *= silu;
            up[e] *= silu;
          }
          put(A.out, at, dg);
          put(A.out, at + A.n_cols, v);
          if (A.out2) put(A.out2, row * A.ldo2 + cur.n0 + c, up);
        } else {
          if (F == kDw && A.accumulate) {
            float old[V];
            unpack(fetch(A.out, at), old);
#pragma unroll
            for (int e = 0; e < V; ++e) v[e] += old[e];
          }
          put(A.out, at, v);
        }
      }
      if constexpr (kDeep > 1) {
        if (i + kDeep < FI) fetch_pre(i + kDeep);
      }
    }

    if (!more) break;
    cur = next;
  }
}

}  // namespace

// Large: one workgroup per compute unit takes tile after tile; where the last round would leave half of them
// without one, its tiles go in quarters.  The other shapes: one tile per workgroup, two workgroups per compute unit.
template <int F, class S>
__global__ void __launch_bounds__(S::kThreads, 2) gemm_bf16_kernel(const BfArgs A) {
  __shared__ __align__(16) uint8_t smem[S::kLdsBytes];
  const int b = blockIdx.x;
  auto tile_at = [&](int round) {
    const int turn = b / kXcds + round * (int)(gridDim.x / kXcds);
    return (turn / A.chunk * kXcds + b % kXcds) * A.chunk + turn % A.chunk;
  };
  if constexpr (S::kPersistent) {
    const int total = count_tiles<F, S>(A), rest = total % (int)gridDim.x;
    const bool cut = 2 * rest <= (int)gridDim.x;
    const int whole = cut ? total - rest : total;
    run_tiles<F, S>(A, smem, [&](int round, Tile& t) {
      const int at = tile_at(round);
      return at < whole && find_tile<F, S>(A, at, t);
    });
    if (!cut) return;
    // (the quarters of a tile on one XCD; one that holds nothing is an empty turn)
    const int mine = b % kXcds * (int)(gridDim.x / kXcds) + b / kXcds;
    for (int i = mine; i < 4 * rest; i += gridDim.x) {
      run_tiles<F, Quarter>(A, smem, [&](int round, Tile& t) {
        return round == 0 && find_tile<F, S>(A, whole + i / 4, t) && quarter<F, Quarter>(t, i & 3);
      });
      __builtin_amdgcn_s_waitcnt(kLgkmZero);
      block_barrier();
    }
  } else {
    run_tiles<F, S>(A, smem, [&](int round, Tile& t) { return round == 0 && find_tile<F, S>(A, tile_at(0), t); });
  }
}

// The first product of the adapters of many tokens (see lora.hip): x A^T of a tile of 64 tokens over each adapter among
// them, of which a token takes its own: part[chunk][t][j] in fp32.  Up to four adapters lie side by side in a tile of
// 64 columns, 2^shift of them each (8192 tokens of 64 adapters in any order, rank 16, 1024 -> 1024: 98 us, one adapter
// a tile 148, with the second product 5 us faster than it is now); of more than 64 ranks two workgroups take half each where the chip is not full (651 tokens of 8 runs,
// rank 128, 456 -> 664: 17 us, both halves in one 28).
__global__ void __launch_bounds__(Small::kThreads, 2)
lora_tiles_kernel(const uint16_t* __restrict__ x, int64_t ldx, const int32_t* __restrict__ ids,
                  const uint16_t* __restrict__ a, int64_t T, int L, int r, int64_t K, int chunk, int shift,
                  float* part) {
  __shared__ __align__(16) uint8_t smem[Small::kLdsBytes];
  const int lane = threadIdx.x & 63;
  const int64_t t0 = (int64_t)blockIdx.x * Small::M, k0 = (int64_t)blockIdx.y * chunk;
  BfArgs A{};
  A.p = x + k0, A.ldp = ldx, A.q = a + k0, A.ldq = K, A.q_rows = r;
  A.out = part + (int64_t)blockIdx.y * T * r, A.ldo = r, A.out_f32 = 1;
  A.ids = ids, A.shift = shift;
  const int sum = (int)(K - k0 < chunk ? K - k0 : chunk), here = (int)(T - t0 < Small::M ? T - t0 : Small::M);
  int id = lane < here ? ids[t0 + lane] : -1;
  if (id >= L) id = -1;
  uint64_t left = __ballot(id >= 0);
  int slot[4] = {-1, -1, -1, -1}, n0 = r;
  run_tiles<kAdapters, Small>(A, smem, [&](int, Tile& t) {
    if (n0 >= r) {                       // the next adapters
      if (!left) return false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        slot[i] = -1;
        if (i << shift >= Small::N || !left) continue;
        slot[i] = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
        left &= ~__ballot(id == slot[i]);
      }
      n0 = Small::N * blockIdx.z;
    }
    t = {t0,     shift == 6 ? (int64_t)slot[0] * r + n0 : 0, t0, 0, n0, here, r - n0, sum,
         {slot[0], slot[1], slot[2], slot[3]}};
    n0 += Small::N * gridDim.z;
    return true;
  });
}

const KernelInfo kInfoLoraTiles = {"lora_tiles_kernel", "fgg_lora_add", Small::M, Small::N, BK, Small::kThreads,
                                   Small::kStages, Small::kStageBytes, 0, Small::kLdsBytes,
                                   (const void*)lora_tiles_kernel};

hipError_t launch_lora_tiles(int64_t T, int32_t L, int32_t r, int64_t K, const uint16_t* x, int64_t ldx,
                             const int32_t* ids, const uint16_t* a, int chunk, int chunks, float* part, hipStream_t st) {
  const int64_t tiles = (T + Small::M - 1) / Small::M;
  const dim3 grid((unsigned)tiles, (unsigned)chunks, r > Small::N && tiles * chunks < 256 ? 2 : 1);
  // (side by side, adapters are 32-bit byte offsets from the first)
  const int shift = r > 32 || (int64_t)L * r * K >= 1 << 30 ? 6 : r > 16 ? 5 : 4;
  trace_launch(kInfoLoraTiles, grid, "T=%lld L=%d r=%d K=%lld", (long long)T, L, r, (long long)K);
  hipLaunchKernelGGL(lora_tiles_kernel, grid, dim3(Small::kThreads), 0, st, x, ldx, ids, a, T, L, r, K, chunk, shift,
                     part);
  return hipGetLastError();
}

#define FGG_BF16_INFO(name, entry, form, S) \
  {"gemm_bf16_kernel<" name "," #S ">", entry, S::M, S::N, BK, S::kThreads, S::kStages, S::kStageBytes, 0, \
   S::kLdsBytes, (const void*)gemm_bf16_kernel<form, S>}
#define FGG_BF16_SHAPES(name, entry, form) \
  FGG_BF16_INFO(name, entry, form, Large), FGG_BF16_INFO(name, entry, form, Medium), \
      FGG_BF16_INFO(name, entry, form, Small)
const KernelInfo kInfoGemmBf16[kGemmBf16Forms] = {
    FGG_BF16_SHAPES("linear", "fgg_grouped_linear", kLinear),
    FGG_BF16_SHAPES("gated", "fgg_grouped_gated", kGated),
    FGG_BF16_SHAPES("dx", "fgg_grouped_linear_backward_input", kDx),
    FGG_BF16_SHAPES("gated_backward", "fgg_grouped_gated_backward", kGatedBwd),
    FGG_BF16_SHAPES("dw", "fgg_grouped_linear_backward_weight", kDw),
};
#undef FGG_BF16_SHAPES
#undef FGG_BF16_INFO

namespace {

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles that can exist: with offsets a segment may begin and end anywhere, so each may have a partial tile.
int64_t row_tiles(const int32_t* offsets, int32_t G, int64_t M, int height) {
  return up(M, height) + (offsets ? (G < M ? G : M) : 0);
}

template <int F, class S>
int64_t tiles_of(const BfArgs& a) {
  const int64_t across = up(a.n_cols, F == kGated ? S::N / 2 : S::N);
  return across * (F == kDw ? a.G * up(a.m_cols, S::M) : row_tiles(a.offsets, a.G, a.M, S::M));
}

template <int F, class S>
hipError_t launch_shape(BfArgs a, int index, hipStream_t st) {
  a.n_tiles = (int)up(a.n_cols, F == kGated ? S::N / 2 : S::N);
  a.m_tiles = F == kDw ? (int)up(a.m_cols, S::M) : 0;
  const int64_t tiles = tiles_of<F, S>(a) * a.splits;
  // tiles of one XCD side by side; with few tiles, an eighth of them.  Large: a workgroup per compute unit.
  int64_t most = kChunk;
  if (S::kPersistent && a.num_cus / kXcds < kChunk) most = a.num_cus < kXcds ? 1 : a.num_cus / kXcds;
  a.chunk = (int)(tiles >= kXcds * most ? most : up(tiles, kXcds));
  const int64_t round = (int64_t)kXcds * a.chunk;
  const dim3 grid((unsigned)(S::kPersistent ? round : up(tiles, round) * round));
  trace_launch(kInfoGemmBf16[3 * F + index], grid, "G=%d M=%lld columns=%lld sum=%lld%s", a.G, (long long)a.M,
               (long long)a.n_cols, (long long)(F == kDw ? a.M : a.sum), a.counts ? " counts" : "");
  hipLaunchKernelGGL((gemm_bf16_kernel<F, S>), grid, dim3(S::kThreads), 0, st, a);
  return hipGetLastError();
}

// The shape whose estimated time is least.  A tile takes its stages (64 deep) one after the other; measured, in
// microseconds a stage (Large / Medium / Small): 1.16 / 0.58 to 0.9 / 0.27 where a compute unit has one workgroup
// (Medium loads one stage ahead and waits for cold operands), 1.5 / 0.95 / 0.37 to 0.42 for a round of what it
// holds (1 / 2 / 2 workgroups) when the chip is full; plus 10 / 4 / 2 to begin and end each.  E.g. linear, one
// segment: 2048^3 50 / 25 / 32 us, 4096 x 2048 x 2048 53 / 36 / 55, 8192^3 791 / 943 / 1520, 256 x 4096 x 4096
// 87 / 41 / 20.  The estimates are for 256 compute units also where the caller leaves fewer to the Large grid: the
// parts of a sum, and with them the workspace and the result's bits, stay the same.
struct Plan {
  int shape, splits;   // 0 Large, 1 Medium, 2 Small; parts of the sum
};

double shape_us(int shape, double tiles, double stages, bool alike) {
  constexpr double kCus = 256.0;
  constexpr double one[3] = {1.16, 0.72, 0.27}, full[3] = {1.5, 0.95, 0.40}, ends[3] = {10.0, 4.0, 2.0};
  constexpr double ragged[3] = {0.3, 0.9, 0.9};        // of a round, lost to uneven segments
  const double slots = shape == 0 ? kCus : 2 * kCus;
  if (tiles <= kCus)
    return stages * (one[shape] + (shape == 0 ? (full[0] - one[0]) * tiles / kCus : 0.0)) + ends[shape] + 1.0;
  double rounds = tiles / slots;
  if (!alike) {
    rounds += ragged[shape];
  } else {
    const double whole = (double)(int64_t)rounds, rest = rounds - whole;
    // (Large: a last round of quarters)
    rounds = whole + (rest == 0.0 ? 0.0 : shape == 0 && rest <= 0.25 ? 0.4 : shape == 0 && rest <= 0.5 ? 0.8 : 1.0);
  }
  if (rounds < 1.0) rounds = 1.0;
  return rounds * (stages * full[shape] + ends[shape]);
}

// Whether a launch of so many tiles of this shape is a grid (Large takes any number with a workgroup per compute unit).
bool fits_grid(int shape, int64_t tiles) { return shape == 0 || tiles <= kMaxBf16Grid; }

// Rows' forms: segments are taken to be alike, with half a tile of each lost at its end.
Plan plan_rows(const Segments& s, int64_t cols, int64_t sum, bool gated) {
  constexpr int kSide[3] = {256, 128, 64};
  Plan best = {0, 1};
  double least = 1e30;
  for (int i = 0; i < 3; ++i) {
    const int64_t across = up(cols, gated ? kSide[i] / 2 : kSide[i]);
    if (!fits_grid(i, row_tiles(s.offsets, s.G, s.M, kSide[i]) * across)) break;
    double down = (double)up(s.M, kSide[i]);
    if (s.G > 1) {
      const double live = (double)(s.G < s.M ? s.G : s.M);
      down = (double)s.M / kSide[i] + 0.5 * live;
      if (down < live) down = live;
    }
    const double us = shape_us(i, down * (double)across, (double)up(sum, 64), s.G == 1);
    if (us < least) least = us, best.shape = i;
  }
  return best;
}

// Weights' gradient: few results with a long sum are cut into parts, whose fp32 results (written and read at
// about 4 bytes a picosecond) a second kernel adds: 30000 rows onto 1024 x 1160, 588 us in one part.
Plan plan_dw(int32_t G, int64_t M, int64_t N, int64_t K) {
  constexpr int kSide[3] = {256, 128, 64};
  Plan best = {0, 1};
  double least = 1e30;
  const double each = (double)up(up(M, G), 64);
  for (int i = 0; i < 3; ++i) {
    if (!fits_grid(i, G * up(N, kSide[i]) * up(K, kSide[i]))) break;
    const double tiles = (double)G * (double)up(N, kSide[i]) * (double)up(K, kSide[i]);
    for (int z = 1; z <= 32; ++z) {
      const double stages = (double)(int64_t)((each + z - 1) / z);
      if (z > 1 && (stages < 4 || tiles * z > 1024)) break;
      const double us = shape_us(i, tiles * z, stages, true) + (z > 1 ? 4.0 + (double)z * G * N * K * 8 / 4e6 : 0.0);
      if (us < least) least = us, best = {i, z};
    }
  }
  return best;
}

template <int F>
hipError_t launch(const BfArgs& a, int shape, hipStream_t st) {
  if (shape == 0) return launch_shape<F, Large>(a, 0, st);
  if (shape == 1) return launch_shape<F, Medium>(a, 1, st);
  return launch_shape<F, Small>(a, 2, st);
}

// out (+)= the parts' sums, in their order; four elements a thread.
template <bool F32, bool ADD>
__global__ void __launch_bounds__(256) dw_join_kernel(const float4* __restrict__ part, int splits, int64_t quads,
                                                      void* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  float4 s = part[i];
  for (int z = 1; z < splits; ++z) {
    const float4 p = part[z * quads + i];
    s.x += p.x, s.y += p.y, s.z += p.z, s.w += p.w;
  }
  if constexpr (F32) {
    float4* o = (float4*)out + i;
    if constexpr (ADD) {
      const float4 old = *o;
      s.x += old.x, s.y += old.y, s.z += old.z, s.w += old.w;
    }
    *o = s;
  } else {
    uint2* o = (uint2*)out + i;
    if constexpr (ADD) {
      const uint2 old = *o;
      s.x += __uint_as_float(old.x << 16), s.y += __uint_as_float(old.x & 0xFFFF0000u);
      s.z += __uint_as_float(old.y << 16), s.w += __uint_as_float(old.y & 0xFFFF0000u);
    }
    *o = make_uint2(bf16x2_rne(s.x, s.y), bf16x2_rne(s.z, s.w));
  }
}

// Few rows take the few-row kernel where the smallest tiles would leave half the chip without one: they then wait
// out one tile's whole sum, which the few-row kernel shares between eight waves.  Its rows cost more the more there
// are of a segment: 16 on average where the tiles are 128, to 32 where they are 64 and fewer.  Few-row / tiles, us, rows
// spread evenly: one row 7168 -> 4096 12.6 / 32, 32 rows 21.7 / 32; 16 segments 2048 -> 512, 4 rows each 8.6 / 12.3,
// 16 11.3 / 12.4, 32 15.3 / 12.5; 4 segments 4096 -> 2048, 16 rows each 19.4 / 21.0, 24 22.7 / 21.5.  How the rows are
// spread is not known here: with all of them in one segment, passes of 64 run side by side, and 256 rows bound what
// that costs (16 segments 2048 -> 512, 64 rows 12.0 / 11.8, 128 12.4 / 12.0, 256 21 / 12.2; 512 rows 40 / 12.3).
bool few_rows(const Segments& s, int64_t cols, bool gated) {
  const int64_t live = s.G < s.M ? s.G : s.M, tiles = live * up(cols, gated ? Small::N / 2 : Small::N);
  return s.M <= kFewRows && s.M <= 32 * live && tiles <= 128 && s.M * tiles <= 2048 * live;
}

}  // namespace

const KernelInfo kInfoDwJoin[4] = {
    {"dw_join_kernel<bf16>", "fgg_grouped_linear_backward_weight", 0, 0, 0, 256, 0, 0, 0, 0,
     (const void*)dw_join_kernel<false, false>},
    {"dw_join_kernel<bf16,add>", "fgg_grouped_linear_backward_weight", 0, 0, 0, 256, 0, 0, 0, 0,
     (const void*)dw_join_kernel<false, true>},
    {"dw_join_kernel<f32>", "fgg_grouped_linear_backward_weight", 0, 0, 0, 256, 0, 0, 0, 0,
     (const void*)dw_join_kernel<true, false>},
    {"dw_join_kernel<f32,add>", "fgg_grouped_linear_backward_weight", 0, 0, 0, 256, 0, 0, 0, 0,
     (const void*)dw_join_kernel<true, true>},
};

int64_t gemm_bf16_tiles(const int32_t* offsets, int32_t G, int64_t M, int64_t cols, bool gated) {
  return row_tiles(offsets, G, M, Large::M) * up(cols, gated ? Large::N / 2 : Large::N);
}

int64_t gemm_bf16_dw_tiles(int32_t G, int64_t N, int64_t K) { return (int64_t)G * up(N, Large::M) * up(K, Large::N); }

size_t gemm_bf16_dw_workspace(int32_t G, int64_t M, int64_t N, int64_t K) {
  if (M == 0 || N == 0 || K == 0) return 0;
  const int splits = plan_dw(G, M, N, K).splits;
  return splits > 1 ? (size_t)splits * (size_t)G * (size_t)N * (size_t)K * 4 : 0;
}

hipError_t launch_grouped_linear(const Segments& s, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                                 const uint16_t* w, void* y, bool y_f32, int64_t ldy, hipStream_t st) {
  BfArgs a{};
  a.splits = 1;
  a.p = x, a.ldp = ldx, a.q = w, a.ldq = K, a.q_rows = N;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M, a.num_cus = s.num_cus;
  a.n_cols = N, a.sum = K, a.out = y, a.ldo = ldy, a.out_f32 = y_f32;
  if (few_rows(s, N, false))
    return launch_rows_bf16(s, false, N, K, x, ldx, w, y, y_f32, ldy, nullptr, 0, st);
  return launch<kLinear>(a, plan_rows(s, N, K, false).shape, st);
}

hipError_t launch_grouped_gated(const Segments& s, int64_t I, int64_t K, const uint16_t* x, int64_t ldx,
                                const uint16_t* w, uint16_t* act, int64_t lda, uint16_t* h, int64_t ldh,
                                hipStream_t st) {
  BfArgs a{};
  a.splits = 1;
  a.p = x, a.ldp = ldx, a.q = w, a.ldq = K, a.q_rows = 2 * I;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M, a.num_cus = s.num_cus;
  a.n_cols = I, a.sum = K, a.out = act, a.ldo = lda, a.out2 = h, a.ldo2 = ldh;
  if (few_rows(s, I, true))
    return launch_rows_bf16(s, true, I, K, x, ldx, w, act, false, lda, h, ldh, st);
  return launch<kGated>(a, plan_rows(s, I, K, true).shape, st);
}

hipError_t launch_grouped_dx(const Segments& s, int64_t N, int64_t K, const uint16_t* dy, int64_t lddy,
                             const uint16_t* w, void* dx, bool dx_f32, int64_t lddx, hipStream_t st) {
  BfArgs a{};
  a.splits = 1;
  a.p = dy, a.ldp = lddy, a.q = w, a.ldq = K, a.q_rows = N;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M, a.num_cus = s.num_cus;
  a.n_cols = K, a.sum = N, a.out = dx, a.ldo = lddx, a.out_f32 = dx_f32;
  return launch<kDx>(a, plan_rows(s, K, N, false).shape, st);
}

hipError_t launch_grouped_gated_backward(const Segments& s, int64_t I, int64_t N, const uint16_t* dy, int64_t lddy,
                                         const uint16_t* w_down, const uint16_t* h, int64_t ldh, uint16_t* dh,
                                         int64_t lddh, uint16_t* act, int64_t lda, hipStream_t st) {
  BfArgs a{};
  a.splits = 1;
  a.p = dy, a.ldp = lddy, a.q = w_down, a.ldq = I, a.q_rows = N;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M, a.num_cus = s.num_cus;
  a.n_cols = I, a.sum = N, a.out = dh, a.ldo = lddh, a.out2 = act, a.ldo2 = lda, a.h = h, a.ldh = ldh;
  return launch<kGatedBwd>(a, plan_rows(s, I, N, false).shape, st);
}

hipError_t launch_grouped_dw(const Segments& s, int64_t N, int64_t K, const uint16_t* dy, int64_t lddy,
                             const uint16_t* x, int64_t ldx, void* dw, bool dw_f32, bool accumulate, float* ws,
                             hipStream_t st) {
  const Plan p = plan_dw(s.G, s.M, N, K);
  BfArgs a{};
  a.p = dy, a.ldp = lddy, a.q = x, a.ldq = ldx;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M, a.num_cus = s.num_cus;
  a.m_cols = N, a.n_cols = K, a.ldo = K, a.splits = p.splits;
  if (p.splits == 1) {
    a.out = dw, a.out_f32 = dw_f32, a.accumulate = accumulate;
    return launch<kDw>(a, p.shape, st);
  }
  a.out = ws, a.out_f32 = 1;
  const hipError_t e = launch<kDw>(a, p.shape, st);
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)s.G * N * K / 4;
  const dim3 grid((unsigned)up(quads, 256));
  trace_launch(kInfoDwJoin[(dw_f32 ? 2 : 0) + (accumulate ? 1 : 0)], grid, "G=%d N=%lld K=%lld parts=%d", s.G,
               (long long)N, (long long)K, p.splits);
  auto join = [&](auto* kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, st, (const float4*)ws, p.splits, quads, dw);
  };
  if (dw_f32) accumulate ? join(dw_join_kernel<true, true>) : join(dw_join_kernel<true, false>);
  else accumulate ? join(dw_join_kernel<false, true>) : join(dw_join_kernel<false, false>);
  return hipGetLastError();
}

}  // namespace fgg
