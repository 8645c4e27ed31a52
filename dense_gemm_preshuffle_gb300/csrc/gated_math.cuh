// The activation of the gated products and its slope, in fp32:
//   ReLU  max(v, 0)                      slope 1 for v > 0, else 0
//   SiLU  v s, s = 1 / (1 + e^-v)        slope s (1 + v (1 - s))
//   GELU  v P, P = (1 + erf(v/sqrt 2))/2 slope P + v e^(-v^2/2) / sqrt(2 pi)
// GELU's P goes through q = erfc(|v| / sqrt 2) by Abramowitz and Stegun,
// Handbook of Mathematical Functions, formula 7.1.26 (|error| <= 1.5e-7), as
// in epilogue.cuh.
#pragma once
#include "../../include/gemm_preshuffle.h"

namespace gp {

struct ActSlope {
  float value, slope;
};

template <int ACT>
__device__ __forceinline__ ActSlope act_slope(float v) {
  if constexpr (ACT == GP_ACT_RELU) {
    // a NaN stays one: v > 0 is false for it, so it is selected explicitly
    return {v > 0.0f ? v : (v != v ? v : 0.0f), v > 0.0f ? 1.0f : 0.0f};
  } else if constexpr (ACT == GP_ACT_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-v));  // e^-v = inf gives 0
    return {v * s, s * fmaf(v, 1.0f - s, 1.0f)};
  } else {
    const float z = fabsf(v) * 0.70710678118654752f;
    const float t = __fdividef(1.0f, fmaf(0.3275911f, z, 1.0f));
    const float e = __expf(-z * z);
    float poly = fmaf(t, 1.061405429f, -1.453152027f);
    poly = fmaf(t, poly, 1.421413741f);
    poly = fmaf(t, poly, -0.284496736f);
    poly = fmaf(t, poly, 0.254829592f);
    const float half_q = 0.5f * t * poly * e;
    const float p = v >= 0.0f ? 1.0f - half_q : half_q;
    return {v * p, fmaf(v * 0.39894228040143268f, e, p)};
  }
}

template <int ACT>
__device__ __forceinline__ float act_value(float v) {
  return act_slope<ACT>(v).value;
}

}  // namespace gp
