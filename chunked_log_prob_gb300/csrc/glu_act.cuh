// The activations of the gated feed-forward block and their derivatives, in fp32.
#pragma once

#include "grpo_gb300.h"
#include "row_ops.cuh"

namespace grpo {

// 1 / (1 + e^-x): 0 and 1 at the ends (e^-x overflows to infinity, whose
// reciprocal is 0). Off by a few units of 2^-23, far below a 16-bit output's rounding.
__device__ __forceinline__ float logistic(float x) {
  return __fdividef(1.f, 1.f + __expf(-x));
}

// act(g), and its derivative where SLOPE.
template <int ACT, bool SLOPE>
__device__ __forceinline__ float activate(float g, float& slope) {
  if constexpr (ACT == GRPO_ACT_SILU) {
    const float s = logistic(g);
    if (SLOPE) slope = s * (1.f + g * (1.f - s));
    return g * s;
  } else if constexpr (ACT == GRPO_ACT_GELU) {
    // Phi(g) by erfc, which keeps its precision in the left tail.
    const float phi = 0.5f * erfcf(-0.70710678118654752f * g);
    if (SLOPE) slope = phi + g * 0.39894228040143268f * __expf(-0.5f * g * g);
    return g * phi;
  } else if constexpr (ACT == GRPO_ACT_GELU_TANH) {
    // 0.5 (1 + tanh z) = logistic(2 z), z = c (g + k g^3).
    constexpr float c2 = 1.5957691216057308f, k = 0.044715f;
    const float s = logistic(c2 * g * (1.f + k * g * g));
    if (SLOPE) {
      // s (1 - s) is 0 far out, where g^2 may not be finite.
      const float b = fminf(fmaxf(g, -30.f), 30.f);
      slope = s + b * s * (1.f - s) * c2 * (1.f + 3.f * k * b * b);
    }
    return g * s;
  } else {
    if (SLOPE) slope = g > 0.f ? 1.f : 0.f;
    return g > 0.f ? g : (g == g ? 0.f : g);
  }
}

// f(std::integral_constant-like tag) for the run-time activation.
template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  switch (act) {
    case GRPO_ACT_SILU: f(ActTag<GRPO_ACT_SILU>()); break;
    case GRPO_ACT_GELU: f(ActTag<GRPO_ACT_GELU>()); break;
    case GRPO_ACT_GELU_TANH: f(ActTag<GRPO_ACT_GELU_TANH>()); break;
    default: f(ActTag<GRPO_ACT_RELU>()); break;
  }
}

}  // namespace grpo
