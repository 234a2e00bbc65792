// What the bf16 products of row segments share (gfx950 only).
#pragma once

#include <type_traits>

#include "fgg_device.hpp"

namespace fgg {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));

// 1 / (1 + e^-g) by the hardware's base-2 exponential and reciprocal.  Relative error at most about (1.3 |g| + 5)
// 2^-24 down to g = -87: g log2(e) is off by 1.3 2^-24 of itself (the constant's and the product's roundings), which
// the exponential turns into 1.3 |g| 2^-24 of its value; exponential and reciprocal add an ulp (two 2^-24) each and
// the sum its rounding.  That is 2^-18.4 at |g| = 32, far inside the bf16 rounding that follows.  Below -87, where the
// value is under 2^-126, the result is 0; NaN stays NaN.
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
