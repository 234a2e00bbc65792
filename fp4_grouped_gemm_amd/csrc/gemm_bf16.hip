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
//  * workgroup tile 256 x 256, 64 deep: 8 waves (two per SIMD) of 128 x 64 outputs, 8 x 4
//    accumulators of v_mfma_f32_16x16x32_bf16.  The n operand is the instruction's first, so a
//    lane holds four consecutive columns of one row.
//  * two LDS stages of 64 KB filled by buffer loads straight into LDS, the next one's issued
//    before the current one is computed.  A buffer descriptor's range check writes zeros for
//    what lies outside (rows past the segment, columns past the edge, the end of the sum), so
//    ragged sizes cost no branch in the loop and what lies there never enters a product.
//  * "row" tiles: 128-byte LDS rows, 16-byte chunk c of row r at chunk c ^ (r & 7): the sixteen
//    lanes that one cycle of a ds_read_b128 serves hit sixteen different chunks.
//  * "col" tiles: LDS rows of 256 outputs for one summed index, read by ds_read_b64_tr_b16, which
//    turns 4 x 16 blocks in the read; 32-byte unit u of row c at u ^ (c & 3 | (c >> 3 & 1) << 2).
//  * one workgroup per tile; a tile's segment is found by a scan over the segments' row counts
//    in each wave's lanes (no table, no workspace).  Workgroups are dealt to the 8 XCDs in turn,
//    and 32 consecutive tiles (8 high, 4 wide) go to one XCD, whose L2 then holds what they share.
#include <type_traits>

#include "fgg_device.hpp"
#include "fgg_internal.hpp"

namespace fgg {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));

constexpr int BM = 256, BN = 256, BK = 64;
constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kTileBytes = 256 * BK * 2;                 // one operand of one stage: 32 KB
constexpr int kStageBytes = 2 * kTileBytes;
constexpr int kQOff = 2 * kTileBytes;                    // LDS: P stage 0, 1, Q stage 0, 1
constexpr int kLdsBytes = 2 * kStageBytes;
constexpr int kDma = kTileBytes / 1024 / kWaves;         // 1 KB loads per wave, operand and stage
constexpr int kXcds = 8, kSM = 8, kChunk = 32;           // tiles of one XCD at a time: 8 high, 4 wide
constexpr uint32_t kOutside = 0x80000000u;               // offset that the range check rejects

enum Form { kLinear, kGated, kDx, kGatedBwd, kDw };
constexpr bool p_is_col(int f) { return f == kDw; }
constexpr bool q_is_col(int f) { return f == kDx || f == kGatedBwd || f == kDw; }

// 16 bytes per lane from base + voff into LDS at lds + 16 * lane; zeros where voff is kOutside.
__device__ inline void buf_dma16(const void* base, uint32_t voff, uint32_t lds) {
  const uint64_t b = (uint64_t)(uintptr_t)base;
  const v4i rs = {__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                  __builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32) & 0xFFFF), (int)0x80000000u, 0x00020000};
  uint32_t save;
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %3\n\t"
      "buffer_load_dwordx4 %1, %2, 0 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(save)
      : "v"(voff), "s"(rs), "s"(lds)
      : "memory");
}

// Eight consecutive summed indices of one output from a "col" tile: two 4 x 16 blocks, 4 rows apart.
__device__ inline v8bf tr_read(const uint8_t* p) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p));
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * 512));
  const v8s v = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  return __builtin_bit_cast(v8bf, v);
}

// 1 / (1 + e^-g) by the hardware's base-2 exponential and reciprocal: within |g| 2^-23 of the
// value for g < 0 (the product's rounding), far inside the bf16 rounding that follows; an
// overflowing e^-g gives 0, NaN stays NaN.
__device__ inline float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

struct Segment {
  int64_t first;   // its first row
  int rows;        // its rows (never past M)
};

// Segment g, from the caller's arrays, kept inside [0, M) whatever they hold.
__device__ inline Segment segment_of(const int32_t* offsets, const int32_t* counts, int g, int64_t M) {
  int64_t s = offsets[g], e = offsets[g + 1];
  s = s < 0 ? 0 : s > M ? M : s;
  if (counts) {
    const int64_t c = counts[g];
    if (c < e - s) e = s + c;
  }
  e = e > M ? M : e;
  return {s, e > s ? (int)(e - s) : 0};
}

}  // namespace

// (see launch_* below for what each form passes)
struct BfArgs {
  const uint16_t *p, *q;
  int64_t ldp, ldq, q_group;           // row strides; elements of one segment's weights
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
};

template <int F>
__global__ void __launch_bounds__(kThreads, 1) gemm_bf16_kernel(const BfArgs A) {
  __shared__ __align__(16) uint8_t smem[kLdsBytes];
  const uint32_t lds_base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave >> 2, wn = wave & 3;
  const int l16 = lane & 15, q = lane >> 4;

  // the tile of this workgroup
  const int b = blockIdx.x;
  const int turn = b / kXcds;
  const int t = (turn / A.chunk * kXcds + b % kXcds) * A.chunk + turn % A.chunk;
  int g = 0, j = t, mtg = A.m_tiles;
  Segment seg;
  if constexpr (F == kDw) {
    g = t / (A.m_tiles * A.n_tiles);
    if (g >= A.G) return;
    j = t - g * (A.m_tiles * A.n_tiles);
    seg = A.offsets ? segment_of(A.offsets, A.counts, g, A.M) : Segment{0, (int)A.M};
  } else if (A.offsets == nullptr) {
    seg = {0, (int)A.M};
    mtg = (int)((A.M + BM - 1) / BM);
    if (t >= mtg * A.n_tiles) return;
  } else {
    int before = 0;
    bool found = false;
    for (int g0 = 0; g0 < A.G; g0 += 64) {
      Segment mine = {0, 0};
      if (g0 + lane < A.G) mine = segment_of(A.offsets, A.counts, g0 + lane, A.M);
      const int tiles = (mine.rows + BM - 1) / BM * A.n_tiles;
      int upto = tiles;
      for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(upto, d);
        if (lane >= d) upto += v;
      }
      const uint64_t hit = __ballot(before + upto > t);
      if (hit) {
        const int at = __builtin_ctzll(hit);
        g = g0 + at;
        j = t - (before + __builtin_amdgcn_readlane(upto, at) - __builtin_amdgcn_readlane(tiles, at));
        seg.first = __builtin_amdgcn_readlane((int)mine.first, at);
        seg.rows = __builtin_amdgcn_readlane(mine.rows, at);
        found = true;
        break;
      }
      before += __builtin_amdgcn_readlane(upto, 63);
    }
    if (!found) return;
    mtg = (seg.rows + BM - 1) / BM;
  }
  const int mb = j / (kSM * A.n_tiles), k_in = j - mb * kSM * A.n_tiles;
  const int high = mtg - mb * kSM < kSM ? mtg - mb * kSM : kSM;
  const int m0 = (mb * kSM + k_in % high) * BM, nt = k_in / high;
  const int n0 = nt * (F == kGated ? BN / 2 : BN);
  // output rows and columns from here on, and the length of the sum
  const int m_here = F == kDw ? (int)A.m_cols - m0 : seg.rows - m0;
  const int n_here = (int)A.n_cols - n0;
  const int sum = F == kDw ? seg.rows : (int)A.sum;
  const int nk = (sum + BK - 1) / BK;

  const uint16_t* P = A.p + seg.first * A.ldp + (F == kDw ? (int64_t)m0 : (int64_t)m0 * A.ldp);
  const uint16_t* Q;
  if constexpr (F == kDw) Q = A.q + seg.first * A.ldq + n0;
  else if constexpr (q_is_col(F)) Q = A.q + (int64_t)g * A.q_group + n0;
  else Q = A.q + (int64_t)g * A.q_group + (int64_t)n0 * A.ldq;

  // what this wave loads: 1 KB pieces of both tiles; byte offsets from P and Q, kOutside past an edge
  uint32_t voff_p[kDma], voff_q[kDma];
  const int r_row = lane >> 3, r_chunk = (lane & 7) ^ r_row;                  // "row": 8 rows a piece
#pragma unroll
  for (int i = 0; i < kDma; ++i) {
    const int piece = wave * kDma + i;
    const int c_row = 2 * piece + (lane >> 5);                                // "col": 2 rows a piece
    const int c_col = ((((lane & 31) >> 1) ^ ((c_row & 3) | ((c_row >> 3) & 1) << 2)) << 4) + (lane & 1) * 8;
    if constexpr (p_is_col(F)) {
      voff_p[i] = c_col < m_here ? (uint32_t)c_row * (uint32_t)(A.ldp * 2) + c_col * 2 : kOutside;
    } else {
      const int row = piece * 8 + r_row;
      voff_p[i] = row < m_here ? (uint32_t)row * (uint32_t)(A.ldp * 2) + r_chunk * 16 : kOutside;
    }
    if constexpr (q_is_col(F)) {
      voff_q[i] = c_col < n_here ? (uint32_t)c_row * (uint32_t)(A.ldq * 2) + c_col * 2 : kOutside;
    } else {
      const int row = piece * 8 + r_row;
      if constexpr (F == kGated) {     // tile rows 0..127: gate columns, 128..255: the up columns of the same index
        voff_q[i] = (row & 127) < n_here ? (uint32_t)(row & 127) * (uint32_t)(A.ldq * 2) + r_chunk * 16 : kOutside;
      } else {
        voff_q[i] = row < n_here ? (uint32_t)row * (uint32_t)(A.ldq * 2) + r_chunk * 16 : kOutside;
      }
    }
  }
  // (gated: waves 4..7 load the up rows, n_cols rows further)
  const uint16_t* Qw = F == kGated && wave >= 4 ? Q + A.n_cols * A.ldq : Q;
  auto issue = [&](int kb, int stage) {
    const uint16_t* p = P + (p_is_col(F) ? (int64_t)kb * BK * A.ldp : (int64_t)kb * BK);
    const uint16_t* qq = Qw + (q_is_col(F) ? (int64_t)kb * BK * A.ldq : (int64_t)kb * BK);
    const int rest = sum - kb * BK;
    const uint32_t lds = lds_base + stage * kTileBytes + wave * kDma * 1024;
#pragma unroll
    for (int i = 0; i < kDma; ++i) {
      const int c_row = 2 * (wave * kDma + i) + (lane >> 5);
      uint32_t vp = voff_p[i], vq = voff_q[i];
      if (rest < BK) {                 // the end of the sum: zeros
        if ((p_is_col(F) ? c_row : r_chunk * 8) >= rest) vp = kOutside;
        if ((q_is_col(F) ? c_row : r_chunk * 8) >= rest) vq = kOutside;
      }
      buf_dma16(p, vp, lds + i * 1024);
      buf_dma16(qq, vq, lds + kQOff + i * 1024);
    }
  };

  // this lane's operand reads: "row": chunk 4 s + q of row l16 (+ 16 per fragment); "col": rows
  // 8 q + (l16 >> 2) (+ 4 for the second half), the fragment's 32-byte unit
  const int c_key = ((l16 >> 2) & 3) | (q & 1) << 2;
  const uint32_t c_lane = (8 * q + (l16 >> 2)) * 512 + (l16 & 3) * 8;
  auto read_p = [&](int stage, int s, int i) -> v8bf {
    const uint8_t* base = smem + stage * kTileBytes;
    if constexpr (p_is_col(F)) {
      return tr_read(base + (c_lane + wm * 256 + ((i ^ c_key) << 5)) + s * 32 * 512);
    } else {
      const int row = wm * 128 + l16;
      return *reinterpret_cast<const v8bf*>(base + (row * 128 + (((4 * s + q) ^ (row & 7)) << 4)) + i * 2048);
    }
  };
  auto read_q = [&](int stage, int s, int n) -> v8bf {
    const uint8_t* base = smem + kQOff + stage * kTileBytes;
    if constexpr (q_is_col(F)) {
      return tr_read(base + (c_lane + (((4 * wn + n) ^ c_key) << 5)) + s * 32 * 512);
    } else {
      const int row = (F == kGated ? 32 : 64) * wn + l16;
      const int further = F == kGated ? (n & 1) * 16 + (n >> 1) * 128 : 16 * n;
      return *reinterpret_cast<const v8bf*>(base + (row * 128 + (((4 * s + q) ^ (row & 7)) << 4)) + further * 128);
    }
  };

  v4f acc[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int n = 0; n < 4; ++n) acc[i][n] = v4f{0.f, 0.f, 0.f, 0.f};

  // One stage: 16 groups (two halves of the depth, 8 row fragments) of 4 MFMAs.  A group's row
  // fragment is read two groups ahead, the column fragments of the second half during the first.
  // At group 14 every fragment of the stage has been read: there the next stage's loads are
  // awaited, the waves meet, the stage after next goes into this stage's buffers, and the last
  // two groups read the next stage's first fragments, so that the matrix cores have work while
  // those reads run.  The order is pinned.
  v8bf fp[3], fq[2][4];
  auto step = [&](auto st_tag, auto off_tag, int kb) {
    constexpr int ST = decltype(st_tag)::value;
    constexpr int R = decltype(off_tag)::value;          // place of the stage's first row fragment in fp
#pragma unroll
    for (int gi = 0; gi < 16; ++gi) {
      const int s = gi >> 3, i = gi & 7;
      if (gi == 14) {
        __builtin_amdgcn_s_waitcnt(kLgkmZero);
        wait_vmcnt<0>();
        block_barrier();
        if (kb + 2 < nk) issue(kb + 2, ST);
      }
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        acc[i][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fq[s][n], fp[(R + gi) % 3], acc[i][n], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
        if (n == 0) {
          const int ahead = gi + 2;                       // (of the next stage from group 14 on)
          fp[(R + ahead) % 3] = ahead < 16 ? read_p(ST, ahead >> 3, ahead & 7) : read_p(ST ^ 1, 0, ahead - 16);
        }
        if (n == 2 && gi >= 3 && gi < 7) fq[1][gi - 3] = read_q(ST, 1, gi - 3);
        if ((n == 1 || n == 3) && gi >= 14) fq[0][2 * (gi - 14) + (n >> 1)] = read_q(ST ^ 1, 0, 2 * (gi - 14) + (n >> 1));
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  if (nk > 0) {
    issue(0, 0);
    wait_vmcnt<0>();
    block_barrier();
    if (nk > 1) issue(1, 1);
#pragma unroll
    for (int n = 0; n < 4; ++n) fq[0][n] = read_q(0, 0, n);
    fp[0] = read_p(0, 0, 0), fp[1] = read_p(0, 0, 1);
    // (16 fragments a stage and three places: the first one's place moves on by one)
    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    using I2 = std::integral_constant<int, 2>;
    for (int kb = 0; kb < nk; kb += 6) {
      step(I0{}, I0{}, kb);
      if (kb + 1 < nk) step(I1{}, I1{}, kb + 1);
      if (kb + 2 < nk) step(I0{}, I2{}, kb + 2);
      if (kb + 3 < nk) step(I1{}, I0{}, kb + 3);
      if (kb + 4 < nk) step(I0{}, I1{}, kb + 4);
      if (kb + 5 < nk) step(I1{}, I2{}, kb + 5);
    }
  }

  // outputs: lane holds columns 4 q + (0..3) of each fragment for row l16
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = wm * 128 + 16 * i + l16;
    if (r >= m_here) continue;
    const int64_t row = (F == kDw ? (int64_t)g * A.m_cols : seg.first) + m0 + r;
    if constexpr (F == kGated) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int c = 32 * wn + 16 * n + 4 * q;
        if (c >= n_here) continue;
        float a[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gate = acc[i][n][e];
          a[e] = gate * sigmoid(gate) * acc[i][n + 2][e];
        }
        *reinterpret_cast<uint2*>((uint16_t*)A.out + row * A.ldo + n0 + c) =
            make_uint2(bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3]));
        if (A.out2) {
          uint16_t* hrow = A.out2 + row * A.ldo2 + n0 + c;
          const v4f u = acc[i][n], v = acc[i][n + 2];
          *reinterpret_cast<uint2*>(hrow) = make_uint2(bf16x2_rne(u[0], u[1]), bf16x2_rne(u[2], u[3]));
          *reinterpret_cast<uint2*>(hrow + A.n_cols) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int c = wn * 64 + 16 * n + 4 * q;
        if (c >= n_here) continue;
        v4f v = acc[i][n];
        if constexpr (F == kGatedBwd) {
          const uint16_t* hrow = A.h + row * A.ldh + n0 + c;
          const uint2 gw = *reinterpret_cast<const uint2*>(hrow);
          const uint2 uw = *reinterpret_cast<const uint2*>(hrow + A.n_cols);
          const uint32_t gs[2] = {gw.x, gw.y}, us[2] = {uw.x, uw.y};
          float dg[4], du[4], a[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float gate = __uint_as_float((e & 1) ? gs[e >> 1] & 0xFFFF0000u : gs[e >> 1] << 16);
            const float up = __uint_as_float((e & 1) ? us[e >> 1] & 0xFFFF0000u : us[e >> 1] << 16);
            const float s = sigmoid(gate);
            const float silu = gate * s;
            dg[e] = v[e] * up * fmaf(silu, 1.0f - s, s);
            du[e] = v[e] * silu;
            a[e] = silu * up;
          }
          uint16_t* drow = (uint16_t*)A.out + row * A.ldo + n0 + c;
          *reinterpret_cast<uint2*>(drow) = make_uint2(bf16x2_rne(dg[0], dg[1]), bf16x2_rne(dg[2], dg[3]));
          *reinterpret_cast<uint2*>(drow + A.n_cols) = make_uint2(bf16x2_rne(du[0], du[1]), bf16x2_rne(du[2], du[3]));
          if (A.out2)
            *reinterpret_cast<uint2*>(A.out2 + row * A.ldo2 + n0 + c) =
                make_uint2(bf16x2_rne(a[0], a[1]), bf16x2_rne(a[2], a[3]));
        } else if (A.out_f32) {
          float4* o = reinterpret_cast<float4*>((float*)A.out + row * A.ldo + n0 + c);
          if (F == kDw && A.accumulate) {
            const float4 old = *o;
            v[0] += old.x, v[1] += old.y, v[2] += old.z, v[3] += old.w;
          }
          *o = make_float4(v[0], v[1], v[2], v[3]);
        } else {
          uint2* o = reinterpret_cast<uint2*>((uint16_t*)A.out + row * A.ldo + n0 + c);
          if (F == kDw && A.accumulate) {
            const uint2 old = *o;
            v[0] += __uint_as_float(old.x << 16), v[1] += __uint_as_float(old.x & 0xFFFF0000u);
            v[2] += __uint_as_float(old.y << 16), v[3] += __uint_as_float(old.y & 0xFFFF0000u);
          }
          *o = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
        }
      }
    }
  }
}

#define FGG_BF16_INFO(name, entry, form) \
  {"gemm_bf16_kernel<" name ">", entry, BM, BN, BK, kThreads, 2, kStageBytes, 0, kLdsBytes, \
   (const void*)gemm_bf16_kernel<form>}
const KernelInfo kInfoGemmBf16[kGemmBf16Forms] = {
    FGG_BF16_INFO("linear", "fgg_grouped_linear", kLinear),
    FGG_BF16_INFO("gated", "fgg_grouped_gated", kGated),
    FGG_BF16_INFO("dx", "fgg_grouped_linear_backward_input", kDx),
    FGG_BF16_INFO("gated_backward", "fgg_grouped_gated_backward", kGatedBwd),
    FGG_BF16_INFO("dw", "fgg_grouped_linear_backward_weight", kDw),
};
#undef FGG_BF16_INFO

namespace {

// Tiles that can exist: with offsets a segment may begin and end anywhere, so each may have a partial tile.
int64_t row_tiles(const int32_t* offsets, int32_t G, int64_t M) {
  const int64_t whole = (M + BM - 1) / BM;
  return offsets ? whole + (G < M ? G : M) : whole;
}

template <int F>
hipError_t launch(BfArgs a, int64_t m_tiles, int64_t tiles, hipStream_t st) {
  if (tiles == 0) return hipSuccess;
  a.m_tiles = (int)m_tiles;
  a.n_tiles = (int)((a.n_cols + (F == kGated ? BN / 2 : BN) - 1) / (F == kGated ? BN / 2 : BN));
  // tiles of one XCD side by side; with few tiles, an eighth of them
  a.chunk = tiles >= kXcds * kChunk ? kChunk : (int)((tiles + kXcds - 1) / kXcds);
  const int64_t round = (int64_t)kXcds * a.chunk;
  const dim3 grid((unsigned)((tiles + round - 1) / round * round));
  trace_launch(kInfoGemmBf16[F], grid, "G=%d M=%lld columns=%lld sum=%lld%s", a.G, (long long)a.M,
               (long long)a.n_cols, (long long)(F == kDw ? a.M : a.sum), a.counts ? " counts" : "");
  hipLaunchKernelGGL(gemm_bf16_kernel<F>, grid, dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

int64_t col_tiles(int64_t cols, int width) { return (cols + width - 1) / width; }

}  // namespace

int64_t gemm_bf16_tiles(const int32_t* offsets, int32_t G, int64_t M, int64_t cols, bool gated) {
  return row_tiles(offsets, G, M) * col_tiles(cols, gated ? BN / 2 : BN);
}

int64_t gemm_bf16_dw_tiles(int32_t G, int64_t N, int64_t K) { return (int64_t)G * col_tiles(N, BM) * col_tiles(K, BN); }

hipError_t launch_grouped_linear(const Segments& s, int64_t N, int64_t K, const uint16_t* x, int64_t ldx,
                                 const uint16_t* w, void* y, bool y_f32, int64_t ldy, hipStream_t st) {
  BfArgs a{};
  a.p = x, a.ldp = ldx, a.q = w, a.ldq = K, a.q_group = N * K;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M;
  a.n_cols = N, a.sum = K, a.out = y, a.ldo = ldy, a.out_f32 = y_f32;
  return launch<kLinear>(a, 0, gemm_bf16_tiles(s.offsets, s.G, s.M, N, false), st);
}

hipError_t launch_grouped_gated(const Segments& s, int64_t I, int64_t K, const uint16_t* x, int64_t ldx,
                                const uint16_t* w, uint16_t* act, int64_t lda, uint16_t* h, int64_t ldh,
                                hipStream_t st) {
  BfArgs a{};
  a.p = x, a.ldp = ldx, a.q = w, a.ldq = K, a.q_group = 2 * I * K;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M;
  a.n_cols = I, a.sum = K, a.out = act, a.ldo = lda, a.out2 = h, a.ldo2 = ldh;
  return launch<kGated>(a, 0, gemm_bf16_tiles(s.offsets, s.G, s.M, I, true), st);
}

hipError_t launch_grouped_dx(const Segments& s, int64_t N, int64_t K, const uint16_t* dy, int64_t lddy,
                             const uint16_t* w, void* dx, bool dx_f32, int64_t lddx, hipStream_t st) {
  BfArgs a{};
  a.p = dy, a.ldp = lddy, a.q = w, a.ldq = K, a.q_group = N * K;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M;
  a.n_cols = K, a.sum = N, a.out = dx, a.ldo = lddx, a.out_f32 = dx_f32;
  return launch<kDx>(a, 0, gemm_bf16_tiles(s.offsets, s.G, s.M, K, false), st);
}

hipError_t launch_grouped_gated_backward(const Segments& s, int64_t I, int64_t N, const uint16_t* dy, int64_t lddy,
                                         const uint16_t* w_down, const uint16_t* h, int64_t ldh, uint16_t* dh,
                                         int64_t lddh, uint16_t* act, int64_t lda, hipStream_t st) {
  BfArgs a{};
  a.p = dy, a.ldp = lddy, a.q = w_down, a.ldq = I, a.q_group = N * I;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M;
  a.n_cols = I, a.sum = N, a.out = dh, a.ldo = lddh, a.out2 = act, a.ldo2 = lda, a.h = h, a.ldh = ldh;
  return launch<kGatedBwd>(a, 0, gemm_bf16_tiles(s.offsets, s.G, s.M, I, false), st);
}

hipError_t launch_grouped_dw(const Segments& s, int64_t N, int64_t K, const uint16_t* dy, int64_t lddy,
                             const uint16_t* x, int64_t ldx, void* dw, bool dw_f32, bool accumulate, hipStream_t st) {
  BfArgs a{};
  a.p = dy, a.ldp = lddy, a.q = x, a.ldq = ldx;
  a.offsets = s.offsets, a.counts = s.counts, a.G = s.G, a.M = s.M;
  a.m_cols = N, a.n_cols = K, a.out = dw, a.ldo = K, a.out_f32 = dw_f32, a.accumulate = accumulate;
  return launch<kDw>(a, col_tiles(N, BM), gemm_bf16_dw_tiles(s.G, N, K), st);
}

}  // namespace fgg
