// Activations and their slopes in float32:
//   relu z [z > 0];  gelu z Phi(z);  gelu_tanh z sigma(2 sqrt(2 / pi) (z + 0.044715 z^3));
//   silu z sigma(z)
// All but relu are z times a probability that is formed without a difference: Phi as
// erfc(-z / sqrt 2) / 2 and sigma(a) as 1 / (1 + exp(-a)), so that what is left far below
// zero keeps its relative accuracy. gelu_tanh is that sigma, since (1 + tanh a) / 2 =
// sigma(2 a).
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/flce.h"

namespace flce {
namespace {

struct Activated {
  float y, slope;
};

// FAST (results rounded to bf16): by the hardware's exponential and reciprocal, a few 2^-22
// of the value for arguments to 80 in size, instead of their correctly rounded forms.
template <bool FAST>
__device__ __forceinline__ float sigma(float a) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(a * -1.44269504f));
  return 1.f / (1.f + expf(-a));
}

template <int ACT, bool FAST>
__device__ __forceinline__ Activated activate(float z) {
  if constexpr (ACT == FLCE_ACT_RELU) {
    return z > 0.f ? Activated{z, 1.f} : Activated{z != z ? z : 0.f, 0.f};
  } else if constexpr (ACT == FLCE_ACT_GELU) {
    const float P = 0.5f * erfcf(z * -0.70710678f);
    return {z * P, fmaf(z * 0.39894228f, expf(-0.5f * z * z), P)};
  } else if constexpr (ACT == FLCE_ACT_GELU_TANH) {
    constexpr float k = 1.5957691216f, c = 0.044715f;         // 2 sqrt(2 / pi)
    const float zz = z * z, s = sigma<FAST>(k * z * fmaf(c, zz, 1.f));
    return {z * s, fmaf(z * s * (1.f - s), k * fmaf(3.f * c, zz, 1.f), s)};
  } else if constexpr (ACT == FLCE_ACT_SILU) {
    const float s = sigma<FAST>(z);
    return {z * s, s * fmaf(z, 1.f - s, 1.f)};
  } else {
    return {z, 1.f};
  }
}

// run(the activation's integral constant)
template <class F>
auto with_activation(int act, F&& run) {
  switch (act) {
    case FLCE_ACT_RELU: return run(std::integral_constant<int, FLCE_ACT_RELU>{});
    case FLCE_ACT_GELU: return run(std::integral_constant<int, FLCE_ACT_GELU>{});
    case FLCE_ACT_GELU_TANH: return run(std::integral_constant<int, FLCE_ACT_GELU_TANH>{});
    case FLCE_ACT_SILU: return run(std::integral_constant<int, FLCE_ACT_SILU>{});
    default: return run(std::integral_constant<int, FLCE_ACT_NONE>{});
  }
}

}  // namespace
}  // namespace flce
