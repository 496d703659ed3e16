// Activations and their slopes in float32:
//   relu z [z > 0];  gelu z Phi(z);  gelu_tanh z sigma(2 sqrt(2 / pi) (z + 0.044715 z^3));
//   silu z sigma(z)
// All but relu are z times a probability that is formed without a difference that cancels:
// sigma(a) as 1 / (1 + exp(-a)), and Phi(-a), a >= 0, as exp(-a^2 / 2) G(a), so that what is
// left far below zero keeps its relative accuracy. gelu_tanh is that sigma, since (1 +
// tanh a) / 2 = sigma(2 a).
//
// G(a) = Phi(-a) exp(a^2 / 2) falls from 1/2 like 1 / a; it is a polynomial of degree 8 in
// t = 1 / (1 + 0.3 a), fitted here by weighted least squares to the scaled complementary
// error function in 64 bits: off by 5.8e-8 of the value for a in [0, 14], 3.5e-7 with its
// float32 roundings (exp(-98) ends float32's range). Two library functions instead, erfc and
// exp, took a third of a 2048 x 1024 x 1024 forward.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/flce.h"

namespace flce {
namespace {

struct Activated {
  float y, slope;
};

// FAST (results rounded to bf16): by the hardware's exponential and reciprocal, off by about
// (2 + |a| / 4) 2^-22 of the value, most of it the exponent's rounding; otherwise by expf and a
// division (silu over a from -80 to 80: at most 3.2 2^-24 of the value).
template <bool FAST>
__device__ __forceinline__ float sigma(float a) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(a * -1.44269504f));
  return 1.f / (1.f + expf(-a));
}

// exp(-a^2 / 2), h = a^2 rounded; what that rounding left is a first-order factor.
template <bool FAST>
__device__ __forceinline__ float gauss(float a, float h) {
  if constexpr (FAST) return __builtin_amdgcn_exp2f(h * -0.72134752f);
  const float e = expf(-0.5f * h);
  return h < 1e30f ? fmaf(e, -0.5f * fmaf(a, a, -h), e) : e;
}

template <int ACT, bool FAST>
__device__ __forceinline__ Activated activate(float z) {
  if constexpr (ACT == FLCE_ACT_RELU) {
    return z > 0.f ? Activated{z, 1.f} : Activated{z != z ? z : 0.f, 0.f};
  } else if constexpr (ACT == FLCE_ACT_GELU) {
    const float a = fabsf(z), h = a * a, E = gauss<FAST>(a, h);
    const float t = FAST ? __builtin_amdgcn_rcpf(fmaf(0.3f, a, 1.f)) : 1.f / fmaf(0.3f, a, 1.f);
    float G = 0.0383785382f;
    G = fmaf(G, t, -0.16916726f);
    G = fmaf(G, t, 0.228662318f);
    G = fmaf(G, t, -0.0765088679f);
    G = fmaf(G, t, 0.142537051f);
    G = fmaf(G, t, 0.0946829284f);
    G = fmaf(G, t, 0.121920479f);
    G = fmaf(G, t, 0.119487672f);
    G = fmaf(G, t, 7.16975861e-06f);
    const float Q = G * E, P = z < 0.f ? Q : 1.f - Q;
    return {z * P, fmaf(z * 0.39894228f, E, P)};
  } else if constexpr (ACT == FLCE_ACT_GELU_TANH) {
    constexpr float k = 1.5957691216f, c = 0.044715f;         // 2 sqrt(2 / pi)
    // an infinite square would make the slope 0 times infinity; sigma is 0 or 1 long before
    const float zz = fminf(z * z, 1e20f), s = sigma<FAST>(k * z * fmaf(c, zz, 1.f));
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
__host__ __device__ __forceinline__ auto with_activation(int act, F&& run) {
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
