// Activations of the gated feed-forward block and their slopes, in fp32.  Internal to libswimba.
//   silu(g) = g s, slope s (1 + g (1 - s)) with s = sigmoid(g);  gelu(g) = g c, slope c + g n with c and n the
//   normal distribution's cumulative and density at g.
#pragma once
#include "block_common.cuh"

namespace swimba {

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
  const float c = 0.5f * (1.f + erff(g * 0.70710678f));
  slope = fmaf(g, 0.39894228f * (kFull ? expf(-0.5f * g * g) : exp_fast(-0.5f * g * g)), c);
  return g * c;
}

// The value alone: silu's quotient is 0 where exp(-g) overflows.
template <int kAct, bool kFull>
__device__ __forceinline__ float act_value(float g) {
  if (kAct == SWIMBA_SILU) return kFull ? g / (1.f + expf(-g)) : g * rcp_fast(1.f + exp_fast(-g));
  return g * (0.5f * (1.f + erff(g * 0.70710678f)));
}

}  // namespace swimba
