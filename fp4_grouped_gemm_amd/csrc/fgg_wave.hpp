// Cross-lane helpers shared by the router, the row kernels and the few-token products (gfx950 only).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fgg {

struct OpMax {
  template <class T>
  __device__ T operator()(T a, T b) const { return a > b ? a : b; }
};
struct OpFMax {   // fmaxf: a NaN operand is ignored
  __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct OpAdd {
  template <class T>
  __device__ T operator()(T a, T b) const { return a + b; }
};

template <int CTRL, class T>
__device__ inline T dpp_move(T v) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "32- or 64-bit values");
  if constexpr (sizeof(T) == 4) {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, true);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(T, ((uint64_t)hi << 32) | lo);
  }
}

// The value of the lane 16 (or 32) away, given in both copies: first holds the even
// (lower) rows' values everywhere, second the odd (upper) rows'.
template <int W, class T, class Op>
__device__ inline T swap_reduce(T v, Op op) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    if constexpr (W == 16) {
      const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      return op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
    } else {
      const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
      return op(__builtin_bit_cast(T, (uint32_t)r[0]), __builtin_bit_cast(T, (uint32_t)r[1]));
    }
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t l0, l1, h0, h1;
    if constexpr (W == 16) {
      const auto l = __builtin_amdgcn_permlane16_swap((uint32_t)u, (uint32_t)u, false, false);
      const auto h = __builtin_amdgcn_permlane16_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
      l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
    } else {
      const auto l = __builtin_amdgcn_permlane32_swap((uint32_t)u, (uint32_t)u, false, false);
      const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)(u >> 32), (uint32_t)(u >> 32), false, false);
      l0 = l[0], l1 = l[1], h0 = h[0], h1 = h[1];
    }
    return op(__builtin_bit_cast(T, ((uint64_t)h0 << 32) | l0), __builtin_bit_cast(T, ((uint64_t)h1 << 32) | l1));
  }
}

// Between LDS accesses of one wave that pass values from lane to lane: the hardware runs them in
// order, and this keeps the compiler from moving one across (no instruction, no wait).
__device__ inline void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Reduction over aligned groups of GW lanes (16, 32 or 64), the result in every lane.
// Data-parallel moves inside the 16-lane rows (quad swaps, then mirrors of 8 and 16
// lanes) and the row swaps of gfx950 above them: no LDS permute.  Both halves of each
// exchange are combined by the same commutative operation, so every lane of a group
// holds the same bits, whatever the group's place in the wave.
template <int GW, class T, class Op>
__device__ inline T group_reduce(T v, Op op) {
  static_assert(GW == 16 || GW == 32 || GW == 64, "group width");
  v = op(v, dpp_move<0xB1>(v));    // lane ^ 1
  v = op(v, dpp_move<0x4E>(v));    // lane ^ 2
  v = op(v, dpp_move<0x141>(v));   // mirror of 8 lanes
  v = op(v, dpp_move<0x140>(v));   // mirror of 16 lanes
  if constexpr (GW >= 32) v = swap_reduce<16>(v, op);
  if constexpr (GW >= 64) v = swap_reduce<32>(v, op);
  return v;
}

}  // namespace fgg
