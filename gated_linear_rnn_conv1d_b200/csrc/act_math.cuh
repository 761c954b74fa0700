// The gated feed-forward block's activations, act(g) = g·s(g): s = Φ (the exact GeLU) or s = σ
// (SiLU), with the derivative s(g) + g·s'(g).
#pragma once
#include <cuda_runtime.h>

#include "gate_math.cuh"

namespace rglru {

constexpr int kActGelu = 0, kActSilu = 1;

// s(g), and for kSlope the derivative of g·s(g). Float32 throughout, one or two special-function
// operations beside the exponential (erff takes a branch and twice the instructions).
// Φ(−|g|) = t·(c₀ + c₁t + … + c₅t⁵)·e^{−g²/2}, t = 1/(1 + p|g|): the form of Abramowitz & Stegun, Handbook of
// Mathematical Functions, 7.1.26, whose own coefficients hold 0.75e-7 in Φ but lose the tail (0.1 % of Φ at g = −4.5, 1 %
// at −8, 3 % at −12, against bf16's half step of 0.4 %). With one coefficient more these were fitted here (a linear
// program over 0 ≤ |g| ≤ 13.5 and p) to an error of at most 0.7e-7 and of at most 7.3e-5 of Φ, so that the tail too is
// right to a fiftieth of a half step. The exponential is the density's, so the derivative Φ(g) + g·φ(g) needs no other.
// (Below −13.2 it is flushed to zero: act(g) is then below bf16's smallest normal number.)
constexpr float kPhiP = 0.291f;
constexpr float kPhi0 = 0.11720908f, kPhi1 = 0.10186288f, kPhi2 = 0.17663312f, kPhi3 = -0.08683966f, kPhi4 = 0.27935827f,
                kPhi5 = -0.08822372f;

template <int ACT, bool kSlope>
__device__ __forceinline__ float act_gate(float g, float& slope) {
  if constexpr (ACT == kActGelu) {
    const float t = rcp_approx(fmaf(fabsf(g), kPhiP, 1.0f));
    const float e = ex2_approx(g * g * (-0.5f * kLog2e));
    float p = fmaf(t, kPhi5, kPhi4);
    p = fmaf(p, t, kPhi3);
    p = fmaf(p, t, kPhi2);
    p = fmaf(p, t, kPhi1);
    p = fmaf(p, t, kPhi0);
    const float q = p * t * e;  // Φ(−|g|)
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
    const float2 den = __ffma2_rn(make_float2(fabsf(g.x), fabsf(g.y)), make_float2(kPhiP, kPhiP), one);
    const float2 t = make_float2(rcp_approx(den.x), rcp_approx(den.y));
    const float2 z = __fmul2_rn(__fmul2_rn(g, g), make_float2(-0.5f * kLog2e, -0.5f * kLog2e));
    const float2 e = make_float2(ex2_approx(z.x), ex2_approx(z.y));
    float2 p = __ffma2_rn(t, make_float2(kPhi5, kPhi5), make_float2(kPhi4, kPhi4));
    p = __ffma2_rn(p, t, make_float2(kPhi3, kPhi3));
    p = __ffma2_rn(p, t, make_float2(kPhi2, kPhi2));
    p = __ffma2_rn(p, t, make_float2(kPhi1, kPhi1));
    p = __ffma2_rn(p, t, make_float2(kPhi0, kPhi0));
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
