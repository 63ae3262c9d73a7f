// Activations of the gated feed-forward block and their slopes, in fp32.  Internal to libswimba.
//   silu(g) = g s, slope s (1 + g (1 - s)) with s = sigmoid(g);  gelu(g) = g c, slope c + g n with c and n the
//   normal distribution's cumulative and density at g.
#pragma once
#include "block_common.cuh"

namespace swimba {

template <int kAct>
__device__ __forceinline__ float act_both(float g, float& slope) {
  if (kAct == SWIMBA_SILU) {
    float s, q;
    gate_pair(g, s, q);
    slope = s * fmaf(g, q, 1.f);
    return g * s;
  }
  const float c = 0.5f * (1.f + erff(g * 0.70710678f));
  slope = fmaf(g, 0.39894228f * exp_fast(-0.5f * g * g), c);
  return g * c;
}

// The value alone: silu's quotient is 0 where exp(-g) overflows.
template <int kAct>
__device__ __forceinline__ float act_value(float g) {
  if (kAct == SWIMBA_SILU) return g * rcp_fast(1.f + exp_fast(-g));
  return g * (0.5f * (1.f + erff(g * 0.70710678f)));
}

}  // namespace swimba
