// The router of a mixture-of-experts layer: from each token's logits over the experts
// to its k expert ids and gate weights, and the gradient of the logits.
//
//   s_e   = softmax(l)_e  or  sigmoid(l_e)
//   key_e = l_e without a selection bias (both gates grow with l), s_e + b_e with one
//   ids   = the k largest keys in decreasing order, ties to the lower expert
//   w_j   = scale * s_{ids j}          or, renormalized,   scale * s_{ids j} / sum_m s_{ids m}
//
// One group of lanes (16, 32 or 64, the smallest that has a lane for every expert up to
// 64) owns a token and holds its logits in registers, experts EPL * lane .. in order;
// a wave takes 64 / GW tokens.  Selection: k rounds of a group-wide maximum over 32-bit
// keys in integer order.  What depends on every expert (the softmax's normalizer) is
// computed only when it is asked for: the renormalized softmax is the softmax of the k
// chosen logits.
//
// Bound by instruction issue, not by memory: one token is one wave's few hundred vector
// instructions.  8192 tokens x 256 experts, bf16, top-8 (4.7 MB, 1 us at a large copy's rate):
// 7.5 us; with a search and two reductions a round 10.1 (a round is one reduction, the tie being the first lane of
// a ballot, and a queue step); 16384 x 384 fp32 16.0 us, 19.6 with a search over eight.  Gradient, 16384 x 160
// fp32, top-6 (21.8 MB): 8.7 us (12.8 with gathered scores and element-wise loads, 10.4 without the
// row of LDS).  One token: 3.2 us, a launch.
//
// With a bias the keys are sums of rounded scores, and two experts whose keys differ by
// less than the rounding of 32 bits would be ordered by it.  The experts are chosen in 32 bits, and a wave in
// which some token has two of its first k + 1 keys closer than those roundings forms its keys in 64 bits (the sigmoid
// or exponential of every logit in double) and chooses again.  16384 x 384 fp32, top-8, sigmoid: 23.2 us, with all keys
// in 64 bits 35.6 (48.2 with the library's exponential and reductions of 64-bit keys).
#include "fgg_device.hpp"
#include "fgg_internal.hpp"
#include "fgg_wave.hpp"

namespace fgg {

namespace {

constexpr float kInf = __builtin_inff();

__device__ inline float load_one(const float* p) { return *p; }
__device__ inline float load_one(const uint16_t* p) { return bf16_to_f32(*p); }

// Experts [e, e + EPL) of a row, -inf from E on; and the same elements stored.  Whole groups move as
// vectors of the element's alignment (this part's vector memory takes any).  A load has no branch around it (the
// row's last EPL experts are read instead of what is behind the row, E >= EPL), so several stay in flight; its
// elements are put in place after it.
template <int EPL, class T>
struct Experts {
  typedef T Vec __attribute__((ext_vector_type(EPL), aligned(sizeof(T))));
  Vec v;
  __device__ void load(const T* row, int e, int E) {
    const int at = e + EPL <= E ? e : E - EPL;
    v = *reinterpret_cast<const Vec*>(row + at);
  }
  __device__ void get(int e, int E, float (&x)[EPL]) const {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (sizeof(T) == 2) x[i] = bf16_to_f32(v[i]);
      else x[i] = v[i];
    }
    if (e + EPL > E) {
      const int down = e + EPL - E;                   // (EPL and more: none is in the row)
#pragma unroll
      for (int d = 1; d < EPL; d *= 2)
        if (down & d) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) x[i] = i + d < EPL ? x[i + d < EPL ? i + d : i] : -kInf;
        }
#pragma unroll
      for (int i = 0; i < EPL; ++i) x[i] = e + i < E ? x[i] : -kInf;
    }
  }
};
template <class T>
struct Experts<1, T> {
  T v;
  __device__ void load(const T* row, int e, int E) { v = row[e < E ? e : E - 1]; }
  __device__ void get(int e, int E, float (&x)[1]) const {
    float f;
    if constexpr (sizeof(T) == 2) f = bf16_to_f32(v);
    else f = v;
    x[0] = e < E ? f : -kInf;
  }
};
template <int EPL>
__device__ inline void store_experts(float* row, int e, int E, const float (&x)[EPL]) {
  typedef float Vec __attribute__((ext_vector_type(EPL), aligned(4)));
  if (EPL > 1 && e + EPL <= E) {
    Vec v;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = x[i];
    *reinterpret_cast<Vec*>(row + e) = v;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e + i < E) row[e + i] = x[i];
  }
}
template <int EPL>
__device__ inline void store_experts(uint16_t* row, int e, int E, const float (&x)[EPL]) {
  typedef uint16_t Vec __attribute__((ext_vector_type(EPL), aligned(2)));
  if (EPL > 1 && e + EPL <= E) {
    Vec v;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = bf16_bits_rne(x[i]);
    *reinterpret_cast<Vec*>(row + e) = v;
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (e + i < E) row[e + i] = bf16_bits_rne(x[i]);
  }
}

// Floating order as unsigned order; 0 is below every number's key (the key of -inf is
// 0x007FFFFF) and stands for "cannot be chosen".  Signed zeros are made equal first.
__device__ inline uint32_t order_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ inline float order_value(uint32_t k) {
  return __uint_as_float(k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ inline uint64_t order_key(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// sigma(v) * e^-m for m <= 0 and v <= max(m, 0): the scale e^-m keeps the sum of the
// chosen scores away from zero when every chosen logit is far below zero.
__device__ inline float sigmoid_scaled(float v, float m) {
  if (v >= 0.0f) return 1.0f / (1.0f + expf(-v));
  return expf(v - m) / (1.0f + expf(v));
}

// e^(x - m) for x <= m, as e^-g with g = m - x held to 200 (e^-200 is 0 in fp32; -inf and the
// difference of far logits end there).
__device__ inline float exp_below(float x, float m) { return exp_neg(fminf(m - x, 200.0f)); }

// e^x in 64 bits for x <= 0 (a NaN stays one): x = n ln 2 + r with |r| <= ln 2 / 2, and Taylor's polynomial to
// r^13 / 13! (the next term is 4e-18).  Below -750 all is 0.
__device__ inline double exp64_nonpos(double x) {
  x = x < -750.0 ? -750.0 : x;
  const double n = __builtin_rint(x * 1.4426950408889634074);
  double r = fma(n, -0.69314718055994530942, x);
  r = fma(n, -2.3190468138462996e-17, r);             // (ln 2 beyond its first 53 bits)
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// The sigmoid in 64 bits: e^-|x| is at most 1, so nothing overflows; the reciprocal of 1 + e^-|x|, in [1/2, 1],
// is the hardware's estimate with two Newton steps.
__device__ inline double sigmoid64(float x) {
  const double e = exp64_nonpos(-(double)fabsf(x)), a = 1.0 + e;
  double y = __builtin_amdgcn_rcp(a);
  y = fma(fma(-a, y, 1.0), y, y);
  y = fma(fma(-a, y, 1.0), y, y);
  return x < 0.0f ? e * y : y;
}

// The group's lane `src` (0 <= src < GW, the same in the group) of v.
template <int GW>
__device__ inline int group_lane(int v, int src) {
  if constexpr (GW == 64) return __builtin_amdgcn_readlane(v, src);
  return __shfl(v, src, GW);
}

// Gate weights of the chosen experts: lane j of a group holds slot j's logit v (on:
// the slot holds an expert).  m_all, sum_all: the softmax's maximum and normalizer over
// all experts (read only for the softmax without renormalization).
template <int GW>
__device__ inline float gate_weight(float v, bool on, bool sigmoid, bool renorm, float m_all, float sum_all) {
  float num;
  if (sigmoid) {
    const float top = renorm ? group_reduce<GW>(on ? v : -kInf, OpFMax()) : 0.0f;
    num = on ? sigmoid_scaled(v, fminf(top, 0.0f)) : 0.0f;
    if (!renorm) return num;
  } else if (renorm) {
    const float top = group_reduce<GW>(on ? v : -kInf, OpFMax());
    num = on ? exp_below(v, top) : 0.0f;
  } else {
    return on ? exp_below(v, m_all) / sum_all : 0.0f;
  }
  const float sum = group_reduce<GW>(num, OpAdd());
  return on ? num / sum : 0.0f;
}

// The k largest keys of a group, in `rounds` >= k rounds: lane j gets round j's key (of 64-bit keys the upper half,
// 0 only where the whole is) and expert, -1 where none is left.  A lane's experts are sorted once, in queues of up to
// four (equal keys keep their order), the places of a queue in the bytes of one word; the lane's candidate is the
// largest head, and the lane that gave the largest of all moves that queue up.  Queues and lanes hold ascending
// experts, so of equal keys the first is the lower expert.  Consumes the keys.
template <int GW, int EPL, class Key>
__device__ inline void select_largest(Key (&key)[EPL], int rounds, int gl, int& my_id, uint32_t& my_key) {
  constexpr int Q = EPL < 4 ? EPL : 4, NQ = EPL / Q;
  uint32_t at[NQ];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    uint32_t p[Q];
#pragma unroll
    for (int i = 0; i < Q; ++i) p[i] = q * Q + i;
#pragma unroll
    for (int end = Q - 1; end > 0; --end)
#pragma unroll
      for (int i = 0; i < end; ++i) {
        Key &ka = key[q * Q + i], &kb = key[q * Q + i + 1];
        const bool swap = kb > ka;
        const Key hi = swap ? kb : ka, lo = swap ? ka : kb;
        const uint32_t phi = swap ? p[i + 1] : p[i], plo = swap ? p[i] : p[i + 1];
        ka = hi, kb = lo, p[i] = phi, p[i + 1] = plo;
      }
    at[q] = p[0];
#pragma unroll
    for (int i = 1; i < Q; ++i) at[q] |= p[i] << (8 * i);
  }
  const int base = (threadIdx.x & 63) & ~(GW - 1);    // the group's first lane
  my_id = -1, my_key = 0;
  for (int j = 0; j < rounds; ++j) {
    Key best = key[0];
    uint32_t place = at[0];
    int bq = 0;
#pragma unroll
    for (int q = 1; q < NQ; ++q)
      if (key[q * Q] > best) best = key[q * Q], place = at[q], bq = q;
    uint32_t top;
    uint64_t heads;
    if constexpr (sizeof(Key) == 8) {
      const uint32_t hi = (uint32_t)(best >> 32);
      top = group_reduce<GW>(hi, OpMax());
      heads = __ballot(hi == top);
      if (__popcll(heads) > 64 / GW) {                // some group has equal upper halves
        const uint32_t lo = hi == top ? (uint32_t)best : 0u;
        const uint32_t top_lo = group_reduce<GW>(lo, OpMax());
        heads = __ballot(hi == top && lo == top_lo);
      }
    } else {
      top = group_reduce<GW>(best, OpMax());
      heads = __ballot(best == top);
    }
    int src, e;
    if constexpr (GW == 64) {
      src = __ffsll((unsigned long long)heads) - 1;
      e = EPL == 1 ? src : src * EPL + (__builtin_amdgcn_readlane((int)place, src) & 0xFF);
    } else {
      src = __ffs((uint32_t)(heads >> base) & (uint32_t)((1ull << GW) - 1)) - 1;
      e = src;                                        // (one expert per lane)
    }
    if (gl == j && top != 0) my_id = e, my_key = top;
    if (gl == src) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (q == bq) {
#pragma unroll
          for (int i = 0; i < Q; ++i) key[q * Q + i] = i + 1 < Q ? key[q * Q + (i + 1 < Q ? i + 1 : i)] : 0;
          at[q] >>= 8;
        }
      }
    }
  }
}

}  // namespace

template <class TI, int GW, int EPL, bool BIAS>
__global__ void __launch_bounds__(256) route_kernel(const TI* __restrict__ logits, int64_t T, int E, int64_t ld, int k,
                                                    bool sigmoid, const float* __restrict__ bias, bool renorm,
                                                    float scale, int32_t* __restrict__ ids, float* __restrict__ w) {
  const int lane = threadIdx.x & 63, gl = lane & (GW - 1);
  const int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / GW) + lane / GW;
  const bool live = t < T;
  const TI* row = logits + (live ? t : 0) * ld;
  float x[EPL], add[EPL];
  int bad = 0;                                        // a NaN in the row (or +inf under a softmax)
  Experts<EPL, TI> in;
  Experts<EPL, float> in_bias;
  in.load(row, gl * EPL, E);
  if constexpr (BIAS) in_bias.load(bias, gl * EPL, E);
  in.get(gl * EPL, E, x);
  if constexpr (BIAS) in_bias.get(gl * EPL, E, add);
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    bad |= __builtin_amdgcn_classf(x[i], sigmoid ? 0x003 : 0x203);   // NaN (and +inf)
  }
  bad = group_reduce<GW>(bad, OpMax());

  // the softmax's maximum and normalizer, where something depends on every expert
  float m_all = -kInf, sum_all = 0.0f, s[EPL];
  if (!sigmoid && (BIAS || !renorm)) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) m_all = fmaxf(m_all, x[i]);
    m_all = group_reduce<GW>(m_all, OpFMax());
#pragma unroll
    for (int i = 0; i < EPL; ++i) sum_all += s[i] = exp_below(x[i], m_all);
    sum_all = group_reduce<GW>(sum_all, OpAdd());
    const float inv = __builtin_amdgcn_rcpf(sum_all);
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] *= inv;
  } else if (BIAS) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x[i] * -1.44269504f));
  }

  int my_id;
  uint32_t my_key, key[EPL];
  if constexpr (BIAS) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const float c = s[i] + add[i];
      key[i] = (x[i] > -kInf && c > -kInf) ? order_key(c) : 0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = x[i] > -kInf ? order_key(x[i]) : 0;
  }
  if constexpr (BIAS) {
    // One more round than k, where a lane is left for it, shows what the last was chosen over.  A 32-bit key is off
    // by at most 2^-21 (sigmoid: a few roundings of a number up to 1, and of x, worth |x| s (1 - s) < 1/4 of one) or
    // 2^-18 of the largest score (softmax: the sum's 22 roundings), and 2^-23 of itself: an order with gaps of twice
    // that is the order of the exact keys.
    select_largest<GW, EPL>(key, k < GW ? k + 1 : k, gl, my_id, my_key);
    const uint32_t next = __shfl_down(my_key, 1, GW);
    const float v = order_value(my_key);
    const float apart = (sigmoid ? 0x1p-19f : 0x1p-17f * __builtin_amdgcn_rcpf(sum_all)) + fabsf(v) * 0x1p-21f;
    const bool close = gl == GW - 1 ? E > GW : next != 0 && !(v - order_value(next) > apart);
    const bool again = bad || (gl < k && my_key != 0 && close);
    if (__any(again)) {
      uint64_t key64[EPL];
      double sum = 0.0, d[EPL];
      if (sigmoid) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] = sigmoid64(x[i]);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          d[i] = x[i] > -kInf ? exp64_nonpos((double)x[i] - (double)m_all) : 0.0;
          sum += d[i];
        }
        // a row with NaN or +inf has no scores: by the bias alone
        sum = group_reduce<GW>(sum, OpAdd());
        const double inv = bad ? 0.0 : 1.0 / sum;
#pragma unroll
        for (int i = 0; i < EPL; ++i) d[i] *= inv;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const double c = (d[i] == d[i] ? d[i] : 0.0) + (double)add[i];   // (d of a +inf is a NaN)
        key64[i] = (x[i] > -kInf && c > -(double)kInf) ? order_key(c) : 0;
      }
      select_largest<GW, EPL>(key64, k, gl, my_id, my_key);
    }
    if (gl >= k) my_id = -1;
  } else {
    select_largest<GW, EPL>(key, k, gl, my_id, my_key);
  }
  float my_v = BIAS ? 0.0f : order_value(my_key);
  if (BIAS && my_id >= 0) my_v = load_one(row + my_id);           // (in the cache: the row was just read)
  const bool on = my_id >= 0;
  float g = gate_weight<GW>(my_v, on, sigmoid, renorm, m_all, sum_all) * scale;
  if (bad) g = __builtin_nanf("");
  if (live && gl < k) {
    ids[t * k + gl] = my_id;
    w[t * k + gl] = on ? g : 0.0f;
  }
}

// Gradient of the logits from the gradient of the gate weights.  With u_j = scale * dw_j:
//   softmax:               dl_e = s_e (sum_{j: id_j = e} u_j - sum_j u_j s_{id_j})
//   softmax, renormalized: dl_e = sum_{j: id_j = e} p_j (u_j - sum_m u_m p_m),  p = softmax of the chosen logits
//   sigmoid:               dl_e = sum_{j: id_j = e} u_j s_j (1 - s_j)
//   sigmoid, renormalized: dl_e = sum_{j: id_j = e} p_j (1 - s_j)(u_j - sum_m u_m p_m),  p_j = s_j / sum_m s_m
// Only the first reads every logit; the others read the chosen ones and write the row.
template <class TI, int GW, int EPL>
__global__ void __launch_bounds__(256) route_backward_kernel(const TI* __restrict__ logits, int64_t T, int E,
                                                             int64_t ld, int k, bool sigmoid, bool renorm, float scale,
                                                             const int32_t* __restrict__ ids,
                                                             const float* __restrict__ dw, TI* __restrict__ dlogits,
                                                             int64_t ldd) {
  const int lane = threadIdx.x & 63, gl = lane & (GW - 1);
  const int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * (64 / GW) + lane / GW;
  const bool live = t < T;
  const TI* row = logits + (live ? t : 0) * ld;
  int id = -1;
  float u = 0.0f, v = -kInf;
  if (live && gl < k) {
    id = ids[t * k + gl];
    u = scale * dw[t * k + gl];
  }
  const bool whole = !sigmoid && !renorm;
  const bool on = id >= 0 && id < E;
  if (!on) id = -1, u = 0.0f;
  if (!whole && on) v = load_one(row + id);
  if (v != v) u = v;                                  // (a maximum and a clamped difference drop a NaN)
  float d = u;
  if (!whole) {
    const float p = gate_weight<GW>(v, on && v != -kInf, sigmoid, renorm, 0.0f, 1.0f);
    const float mean = renorm ? group_reduce<GW>(on ? u * p : 0.0f, OpAdd()) : 0.0f;
    d = p * (u - mean);
    if (sigmoid && on) d *= v >= 0.0f ? expf(-v) / (1.0f + expf(-v)) : 1.0f / (1.0f + expf(v));   // 1 - sigma(v)
  }
  // d_j to expert id_j.  Over 32 experts through a row of LDS of each wave's own, where no id stands twice in a token
  // (every lane that wrote its number at its expert finds it there): 16384 x 160 10.4 -> 8.7 us, 16384 x 384 of
  // bf16 15.1 -> 10.5.  Slot by slot otherwise (16384 x 32 4.3 us
  // slot by slot, 4.2 through LDS; one token 3.1 us either way).
  float out[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
  bool placed = false;
  if constexpr (GW == 64) {
    __shared__ __attribute__((aligned(16))) float rows[4][64 * EPL];
    float* own = rows[threadIdx.x >> 6];
    int found = lane;
    if (on) *reinterpret_cast<volatile int*>(own + id) = lane;
    wave_sync();
    if (on) found = *reinterpret_cast<volatile int*>(own + id);
    placed = __all(found == lane);
    if (placed) {
      constexpr int V = EPL < 4 ? EPL : 4;
      typedef float Vec __attribute__((ext_vector_type(V)));
      wave_sync();
#pragma unroll
      for (int i = 0; i < EPL; i += V) *reinterpret_cast<Vec*>(own + lane * EPL + i) = Vec(0.0f);
      wave_sync();
      if (on) own[id] = d;
      wave_sync();
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] = own[lane * EPL + i];
    }
  }
  if (!placed) {
    for (int j = 0; j < k; ++j) {
      const int mine = group_lane<GW>(id, j) - gl * EPL;
      const float dj = __int_as_float(group_lane<GW>(__float_as_int(d), j));
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] += mine == i ? dj : 0.0f;
    }
  }
  if (whole) {
    float x[EPL], m = -kInf, sum = 0.0f, dot = 0.0f;
    bool bad = false;
    Experts<EPL, TI> in;
    in.load(row, gl * EPL, E);
    in.get(gl * EPL, E, x);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      m = fmaxf(m, x[i]);
      bad |= __builtin_amdgcn_classf(x[i], 0x203);    // NaN, +inf
    }
    m = group_reduce<GW>(m, OpFMax());
    const bool none = m == -kInf;                     // a row without any expert: all zero
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      x[i] = exp_below(x[i], m);
      sum += x[i];
      dot = fmaf(out[i], x[i], dot);
    }
    if (bad) sum = __builtin_nanf("");
    sum = group_reduce<GW>(sum, OpAdd());
    const float inv = none ? 0.0f : 1.0f / sum;
    dot = group_reduce<GW>(dot, OpAdd()) * inv;
#pragma unroll
    for (int i = 0; i < EPL; ++i) out[i] = x[i] * inv * (out[i] - dot);
    if (none) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) out[i] = 0.0f;
    }
  }
  if (live) store_experts<EPL>(dlogits + t * ldd, gl * EPL, E, out);
}

const KernelInfo kInfoRoute = {"route_kernel", "fgg_moe_route", 0, 0, 0, 256, 0, 0, 0, 0,
                               (const void*)route_kernel<float, 64, 4, false>};
// The gradient's forms, by lanes of a token and experts of a lane: four waves' rows of LDS over 32 experts.
template <int GW, int EPL>
static KernelInfo backward_form(const char* name) {
  constexpr int kLds = GW == 64 ? 4 * 64 * EPL * 4 : 0;
  return {name, "fgg_moe_route_backward", 0, 0, 0, 256, 0, 0, kLds, kLds,
          (const void*)route_backward_kernel<float, GW, EPL>};
}
const KernelInfo kInfoRouteBackward[kRouteBackwardForms] = {
    backward_form<16, 1>("route_backward_kernel<16 lanes>"),
    backward_form<32, 1>("route_backward_kernel<32 lanes>"),
    backward_form<64, 1>("route_backward_kernel<64 lanes>"),
    backward_form<64, 2>("route_backward_kernel<64 lanes x 2>"),
    backward_form<64, 4>("route_backward_kernel<64 lanes x 4>"),
    backward_form<64, 8>("route_backward_kernel<64 lanes x 8>"),
    backward_form<64, 16>("route_backward_kernel<64 lanes x 16>"),
};

// Calls f(group width, experts per lane) as compile-time constants: the smallest that hold E.
template <class F>
static void with_shape(int E, F f) {
  using std::integral_constant;
  if (E <= 16) f(integral_constant<int, 16>(), integral_constant<int, 1>());
  else if (E <= 32) f(integral_constant<int, 32>(), integral_constant<int, 1>());
  else if (E <= 64) f(integral_constant<int, 64>(), integral_constant<int, 1>());
  else if (E <= 128) f(integral_constant<int, 64>(), integral_constant<int, 2>());
  else if (E <= 256) f(integral_constant<int, 64>(), integral_constant<int, 4>());
  else if (E <= 512) f(integral_constant<int, 64>(), integral_constant<int, 8>());
  else f(integral_constant<int, 64>(), integral_constant<int, 16>());
}

static int64_t route_blocks(int64_t T, int E) {
  const int per_block = 4 * (E <= 16 ? 4 : E <= 32 ? 2 : 1);
  return (T + per_block - 1) / per_block;
}

hipError_t launch_route(const void* logits, bool bf16, int64_t T, int32_t E, int64_t ld, int32_t k, bool sigmoid,
                        const float* bias, bool renorm, float scale, int32_t* ids, float* w, hipStream_t st) {
  const dim3 grid((unsigned)route_blocks(T, E));
  trace_launch(kInfoRoute, grid, "T=%lld E=%d k=%d %s %s%s%s", (long long)T, (int)E, (int)k, bf16 ? "bf16" : "fp32",
               sigmoid ? "sigmoid" : "softmax", bias ? " bias" : "", renorm ? " renorm" : "");
  with_shape(E, [&](auto gw, auto epl) {
    constexpr int GW = decltype(gw)::value, EPL = decltype(epl)::value;
    auto go = [&](auto* in) {
      using TI = std::remove_cv_t<std::remove_pointer_t<decltype(in)>>;
      if (bias)
        hipLaunchKernelGGL((route_kernel<TI, GW, EPL, true>), grid, dim3(256), 0, st, in, T, (int)E, ld, (int)k,
                           sigmoid, bias, renorm, scale, ids, w);
      else
        hipLaunchKernelGGL((route_kernel<TI, GW, EPL, false>), grid, dim3(256), 0, st, in, T, (int)E, ld, (int)k,
                           sigmoid, bias, renorm, scale, ids, w);
    };
    if (bf16) go((const uint16_t*)logits);
    else go((const float*)logits);
  });
  return hipGetLastError();
}

hipError_t launch_route_backward(const void* logits, bool bf16, int64_t T, int32_t E, int64_t ld, int32_t k,
                                 bool sigmoid, bool renorm, float scale, const int32_t* ids, const float* dw,
                                 void* dlogits, int64_t ldd, hipStream_t st) {
  const dim3 grid((unsigned)route_blocks(T, E));
  with_shape(E, [&](auto gw, auto epl) {
    constexpr int GW = decltype(gw)::value, EPL = decltype(epl)::value;
    constexpr int kForm = GW == 16 ? 0 : GW == 32 ? 1 : EPL == 1 ? 2 : EPL == 2 ? 3 : EPL == 4 ? 4 : EPL == 8 ? 5 : 6;
    trace_launch(kInfoRouteBackward[kForm], grid, "T=%lld E=%d k=%d %s %s%s", (long long)T, (int)E, (int)k,
                 bf16 ? "bf16" : "fp32", sigmoid ? "sigmoid" : "softmax", renorm ? " renorm" : "");
    if (bf16)
      hipLaunchKernelGGL((route_backward_kernel<uint16_t, GW, EPL>), grid, dim3(256), 0, st, (const uint16_t*)logits,
                         T, (int)E, ld, (int)k, sigmoid, renorm, scale, ids, dw, (uint16_t*)dlogits, ldd);
    else
      hipLaunchKernelGGL((route_backward_kernel<float, GW, EPL>), grid, dim3(256), 0, st, (const float*)logits, T,
                         (int)E, ld, (int)k, sigmoid, renorm, scale, ids, dw, (float*)dlogits, ldd);
  });
  return hipGetLastError();
}

}  // namespace fgg
