// silu(g) u and its gradient in fp32, right over the whole range of the
// operands: with s = 1 / (1 + exp(-g))
//   h = g s u,  dh/du = g s,  dh/dg = u s (1 + g (1 - s)).
// For g above kLowGate s is a normal number (2e-35 at least). Below, s is
// exp(g) to fp32's last bit, and exp(g) leaves fp32's normal numbers at -87.3
// and is zero from -104 on, where a large u or dh still makes the results
// normal. There exp(g) is kept as two factors exp(g / 2), normal down to
// g = -174 (and subnormal, with bits to spare for what results remain, to
// -206), and the products are ordered so that none of their parts leaves the
// range unless the result does.
#pragma once

#include "common.cuh"

namespace moe {

constexpr float kLowGate = -80.0f;

// The special function unit's exponential of base 2, subnormal results kept.
__device__ __forceinline__ float ex2_approx_sub(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// s = 1 / (1 + exp(-g)) and c = 1 - s, for g >= kLowGate or NaN (which stays
// NaN in both). FAST, for outputs of 16 bits: by the special function unit's
// exponential and reciprocal. Their error, at most (|g| + 4) 2^-23 of s, is
// below a thirtieth of half a step of the outputs, and the IEEE forms (20
// instructions more per element) would bound the kernels in place of HBM.
// 1 - s is formed as exp(-|g|) s or s itself, without the cancellation at
// large |g|.
template <bool FAST>
__device__ __forceinline__ void sigmoid_pair(float g, float& s, float& c) {
  const float a = fabsf(g);   // exp(-|g|) is in (0, 1]: no overflow on either side
  const float e = FAST ? ex2_approx(-1.4426950408889634f * a) : expf(-a);
  const float r = FAST ? rcp_approx(1.0f + e) : 1.0f / (1.0f + e);
  const float er = e * r;
  s = g < 0.0f ? er : r;
  c = g < 0.0f ? r : er;
}

// exp(g / 2) for g < kLowGate.
template <bool FAST>
__device__ __forceinline__ float half_exp(float g) {
  return FAST ? ex2_approx_sub(0.72134752044448170f * g) : expf(0.5f * g);
}

// silu(g) u. Below kLowGate |g| exp(g / 2) is less than 1, so its product
// with u cannot overflow, and where that is subnormal the result is zero.
template <bool FAST>
__device__ __forceinline__ float silu_mul(float g, float u) {
  if (g < kLowGate) {
    const float e = half_exp<FAST>(g);
    return g * e * u * e;
  }
  float s, c;
  sigmoid_pair<FAST>(g, s, c);
  return g * s * u;
}

// d u e1 e2 with |e1|, e2 <= 1: the larger of d and u first (it meets e1, so
// nothing overflows), then e2 where that is at least 1, else the smaller one.
// Each part that is subnormal is then followed by factors of at most 1, or
// the result is smaller still.
__device__ __forceinline__ float mul_ordered(float d, float u, float e1, float e2) {
  const bool swap = fabsf(d) < fabsf(u);
  const float hi = swap ? u : d, lo = swap ? d : u;
  const float t = hi * e1;
  return fabsf(t) >= 1.0f ? t * e2 * lo : t * lo * e2;
}

// d u s (1 + g (1 - s)), the gate's gradient, also where d u alone is beyond
// fp32.
template <bool FAST>
__device__ __forceinline__ float dgate_mul(float g, float u, float d) {
  if (g < kLowGate) {   // 1 - s is 1 in fp32
    const float e = half_exp<FAST>(g);
    return mul_ordered(d, u, (1.0f + g) * e, e);
  }
  float s, c;
  sigmoid_pair<FAST>(g, s, c);
  // the slope is 1.1 at most: halved, and the result doubled
  return 2.0f * mul_ordered(d, u, 0.5f * (s + g * s * c), 1.0f);
}

}  // namespace moe
