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

// The same for two values in packed float32 arithmetic (half the instructions): s(g), and the
// derivative of g·s(g).
template <int ACT, bool kSlope>
__device__ __forceinline__ float2 act_gate2(float2 g, float2& slope) {
  const float2 one = make_float2(1.0f, 1.0f);
  if constexpr (ACT == kActGelu) {
    const float2 den = __ffma2_rn(make_float2(fabsf(g.x), fabsf(g.y)),
                                  make_float2(0.3275911f * 0.70710678118654752f, 0.3275911f * 0.70710678118654752f), one);
    const float2 t = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    const float2 z = __fmul2_rn(__fmul2_rn(g, g), make_float2(-0.5f * kLog2e, -0.5f * kLog2e));
    const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
    // the coefficients halved: q = erfc(|g|/√2)/2
    constexpr float a1 = 0.5f * 0.254829592f, a2 = 0.5f * -0.284496736f, a3 = 0.5f * 1.421413741f,
                    a4 = 0.5f * -1.453152027f, a5 = 0.5f * 1.061405429f;
    float2 p = __ffma2_rn(t, make_float2(a5, a5), make_float2(a4, a4));
    p = __ffma2_rn(p, t, make_float2(a3, a3));
    p = __ffma2_rn(p, t, make_float2(a2, a2));
    p = __ffma2_rn(p, t, make_float2(a1, a1));
    const float2 q = __fmul2_rn(__fmul2_rn(p, t), e);
    const float2 s = make_float2(g.x > 0.0f ? 1.0f - q.x : q.x, g.y > 0.0f ? 1.0f - q.y : q.y);
    if constexpr (kSlope)
      slope = __ffma2_rn(__fmul2_rn(g, make_float2(0.39894228040143268f, 0.39894228040143268f)), e, s);
    return s;
  } else {
    const float2 z = __fmul2_rn(g, make_float2(-kLog2e, -kLog2e));
    const float2 den = __fadd2_rn(make_float2(ex2_approx(z.x), ex2_approx(z.y)), one);
    const float2 s = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    if constexpr (kSlope)
      slope = __fmul2_rn(s, __ffma2_rn(g, __fadd2_rn(one, make_float2(-s.x, -s.y)), one));
    return s;
  }
}

}  // namespace rglru
