// What the bf16 products of row segments share (gfx950 only).
#pragma once

#include <type_traits>

#include "fgg_device.hpp"

namespace fgg {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

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
  if (counts) {
    const int64_t c = counts[g];
    if (c < e - s) e = s + c;
  }
  s = s < 0 ? 0 : s > M ? M : s;
  e = e > M ? M : e;
  return {s, e > s ? (int)(e - s) : 0};
}

}  // namespace fgg
