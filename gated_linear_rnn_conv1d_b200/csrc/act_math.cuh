// The gated feed-forward block's activations, act(g) = g·s(g): s = Φ (the exact GeLU) or s = σ
// (SiLU), with the derivative s(g) + g·s'(g).
#pragma once
#include <cuda_runtime.h>

#include "gate_math.cuh"

namespace rglru {

constexpr int kActGelu = 0, kActSilu = 1;

// s(g), and for kSlope the derivative of g·s(g). Float32 throughout, one or two special-function
// operations beside the exponential (erff takes a branch and twice the instructions).
// Φ(−|g|) = erfc(|g|/√2)/2 by Abramowitz & Stegun, Handbook of Mathematical Functions, 7.1.26:
// erfc(z) = (a₁t + … + a₅t⁵) e^{−z²}, t = 1/(1 + pz), to 1.5e-7 absolute; the exponential is
// the density's, so the derivative Φ(g) + g·φ(g) needs no other.
template <int ACT, bool kSlope>
__device__ __forceinline__ float act_gate(float g, float& slope) {
  if constexpr (ACT == kActGelu) {
    const float t = rcp_approx(fmaf(fabsf(g), 0.3275911f * 0.70710678118654752f, 1.0f));
    const float e = ex2_approx(g * g * (-0.5f * kLog2e));
    float p = fmaf(t, 1.061405429f, -1.453152027f);
    p = fmaf(p, t, 1.421413741f);
    p = fmaf(p, t, -0.284496736f);
    p = fmaf(p, t, 0.254829592f);
    const float q = 0.5f * p * t * e;  // Φ(−|g|)
    const float s = g > 0.0f ? 1.0f - q : q;
    if constexpr (kSlope) slope = fmaf(g * 0.39894228040143268f, e, s);
    return s;
  } else {
    const float s = rcp_approx(1.0f + ex2_approx(-g * kLog2e));
    if constexpr (kSlope) slope = s * fmaf(g, 1.0f - s, 1.0f);
    return s;
  }
}

}  // namespace rglru
