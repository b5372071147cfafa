// score_stats.cuh -- the softmax statistics of a row of logits, as the score
// call keeps them.
//
// For logits z and a temperature T the statistics of a set of entries are
//   m = max z,   S = sum e^((z - m) / T),   U = sum (z - m) e^((z - m) / T),
// from which, over the whole vocabulary,
//   log-sum-exp of z / T = m / T + log S
//   log p of entry v     = (z_v - m) / T - log S
//   entropy              = log S - (U / S) / T
// (with log p_v as above, -sum p log p = log S - sum p_v (z_v - m) / T). Both
// terms of the entropy are non-negative, so nothing cancels, and z itself
// never enters an exponential or a product: only differences from the maximum.
//
// Every sum runs in an order fixed by the vocabulary index alone:
//   * 32 consecutive entries share their exact maximum; the two halves of 16
//     are summed in ascending order from zero and added;
//   * four such groups make a 128-entry half ((0 . 1) . (2 . 3)), two halves
//     a 256-entry tile, and the tiles of a row combine in the 128-leaf tree of
//     the log-prob call (head_kernels.cuh).
// The projection kernels that feed it (vocabulary on the lanes, or hidden
// rows on the lanes) follow this order, so a row's results are the same bits
// on either.
#pragma once
#include <cmath>
#include <cstdint>
#include "ptx.cuh"

namespace detlm {

constexpr float kLog2eScore = 1.4426950408889634f;
constexpr float kVeryLow = -3.0e38f;

struct Stat { float m, S, U; };   // an empty set is {-inf, 0, 0}

// max that returns NaN when either side is NaN
__device__ __forceinline__ float fmax_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// One entry into the sums relative to `mm` (the group's maximum, or kVeryLow
// when the group has none). c = log2(e) / T. A logit of -inf counts as zero at
// any temperature (its difference is clamped where it meets e = 0, so that the
// product stays finite); a NaN stays one.
__device__ __forceinline__ void stat_add(float z, float mm, float c, float& S, float& U) {
  const float t = __fsub_rn(z, mm);
  const float e = exp2_approx(__fmul_rn(t, c));
  S = __fadd_rn(S, e);
  U = __fmaf_rn(fmax_nan(t, kVeryLow), e, U);
}

// Union of two disjoint sets; commutative bit for bit. An empty side (S = 0)
// leaves the other as it is.
__device__ __forceinline__ Stat stat_merge(const Stat& a, const Stat& b, float c) {
  const bool sw = a.m < b.m;
  const Stat hi = sw ? b : a, lo = sw ? a : b;
  if (lo.S == 0.0f) return hi;
  const float far = lo.m == hi.m ? 0.0f : __fsub_rn(lo.m, hi.m);
  const float e = exp2_approx(__fmul_rn(far, c));
  // the scaled sum first: for a far lower side it is zero before d, which is
  // kept finite, meets it
  const float d = fmax_nan(far, kVeryLow);
  const float s = __fmul_rn(lo.S, e);
  return Stat{hi.m, __fadd_rn(hi.S, s), __fadd_rn(hi.U, __fmaf_rn(s, d, __fmul_rn(lo.U, e)))};
}

__device__ __forceinline__ Stat shfl_xor(const Stat& x, int b) {
  return Stat{__shfl_xor_sync(0xffffffffu, x.m, b), __shfl_xor_sync(0xffffffffu, x.S, b),
              __shfl_xor_sync(0xffffffffu, x.U, b)};
}

// 32 entries held by one thread, whose maximum m is known (entries `valid`
// and up do not exist).
template <bool RAGGED>
__device__ __forceinline__ Stat stat32(const float (&z0)[16], const float (&z1)[16], float m,
                                       float c, int valid) {
  const float mm = fmaxf(m, kVeryLow);
  float S0 = 0.0f, U0 = 0.0f, S1 = 0.0f, U1 = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (!RAGGED || i < valid) stat_add(z0[i], mm, c, S0, U0);
    if (!RAGGED || 16 + i < valid) stat_add(z1[i], mm, c, S1, U1);
  }
  return Stat{m, __fadd_rn(S0, S1), __fadd_rn(U0, U1)};
}

// Order-preserving 32-bit keys of logits (larger value, larger unsigned key;
// the two zeros share one). Key 0 is below every value, -inf included, and
// marks "no value".
__device__ __forceinline__ uint32_t score_key(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float score_unkey(uint32_t k) {
  if (k == 0u) return -INFINITY;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

}  // namespace detlm
