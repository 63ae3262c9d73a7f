// Activations of the gated feed-forward block and their slopes, in fp32.  Internal to libswimba.
//   silu(g) = g s, slope s (1 + g (1 - s)) with s = sigmoid(g);  gelu(g) = g c, slope c + g n with c and n the
//   normal distribution's cumulative and density at g.
#pragma once
#include "block_common.cuh"

namespace swimba {

// The normal distribution's cumulative at g, and e = exp(-g^2 / 2).  The small half is formed as such: 1 + erf(g / sqrt 2)
// cancels for negative g, in fp32 by 3e-4 of the result at g = -4, 4e-2 at -5 and all of it from -5.6 on, where bf16 and
// fp32 still hold it.  kFull: by erfc.  Otherwise the tail at a = |g| is e t P(t), t = 1 / (1 + 0.362 a), with P fitted to
// the tail over e t on 0 <= a <= 13.5 (e is 0 beyond) for the least relative error, 2^-19.9 as evaluated; with the
// exponent's roundings, 2 u g^2, well inside a 16-bit type's own.  GELU at 8192 x 768 x 2048 bf16, forward and
// gradients: 75.8 and 154 us by erf, 83.7 and 180 by erfc, 73.5 and 148 so; in fp32 at 2048 x 768 x 2048 the gradients
// take 317 us by erf and 335 by erfc.
template <bool kFull>
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  if (kFull) {
    e = expf(-0.5f * g * g);
    return 0.5f * erfcf(g * -0.70710678f);
  }
  e = exp_fast(-0.5f * g * g);
  const float t = rcp_fast(fmaf(fabsf(g), 0.362f, 1.f));
  float p = fmaf(0.0480388403f, t, -0.180348486f);
  p = fmaf(p, t, 0.177071273f);
  p = fmaf(p, t, 0.0285236277f);
  p = fmaf(p, t, 0.139540434f);
  p = fmaf(p, t, 0.14266938f);
  p = fmaf(p, t, 0.144505292f);
  const float tail = e * t * p;
  return g >= 0.f ? 1.f - tail : tail;
}

// kFull: with the accurate exponential and quotient, for fp32 results; 16-bit ones hide the approximations' 2 ulp.
template <int kAct, bool kFull>
__device__ __forceinline__ float act_both(float g, float& slope) {
  if (kAct == SWIMBA_SILU) {
    float s, q;
    if (kFull) {
      const float e = expf(-fabsf(g)), small = e / (1.f + e), large = 1.f / (1.f + e);
      s = g >= 0.f ? large : small;
      q = g >= 0.f ? small : large;
    } else {
      gate_pair(g, s, q);
    }
    slope = s * fmaf(g, q, 1.f);
    return g * s;
  }
  float e;
  const float c = normal_cdf<kFull>(g, e);
  slope = fmaf(g, 0.39894228f * e, c);
  return g * c;
}

// The value alone: silu's quotient is 0 where exp(-g) overflows.
template <int kAct, bool kFull>
__device__ __forceinline__ float act_value(float g) {
  if (kAct == SWIMBA_SILU) return kFull ? g / (1.f + expf(-g)) : g * rcp_fast(1.f + exp_fast(-g));
  float e;
  return g * normal_cdf<kFull>(g, e);
}

}  // namespace swimba
