// Reductions across the lanes of a wave with data-parallel primitives and the
// gfx950 lane swaps: vector instructions, no trip through LDS. Every lane of the
// group gets the same bits.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace flce {
namespace {

template <int CTRL, class T>
__device__ __forceinline__ T dpp_move(T x) {
  static_assert(sizeof(T) == 4, "one register");
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_bit_cast(
      T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
#else
  return x;
#endif
}

constexpr int kDppXor1 = 0xB1, kDppXor2 = 0x4E;              // within 4 lanes
constexpr int kDppDown = 0x100;      // + n: from the lane n further on, 0 past the 16
constexpr int kDppHalfMirror = 0x141, kDppMirror = 0x140;    // reversed within 8, 16 lanes

// op over the TPT (a power of two up to 16) adjacent lanes of a group.
template <int TPT, class T, class Op>
__device__ __forceinline__ T group_all(T x, Op op) {
  static_assert(TPT == 1 || TPT == 2 || TPT == 4 || TPT == 8 || TPT == 16, "within a row");
  if constexpr (TPT >= 2) x = op(x, dpp_move<kDppXor1>(x));
  if constexpr (TPT >= 4) x = op(x, dpp_move<kDppXor2>(x));
  if constexpr (TPT >= 8) x = op(x, dpp_move<kDppHalfMirror>(x));
  if constexpr (TPT >= 16) x = op(x, dpp_move<kDppMirror>(x));
  return x;
}

// op over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
template <class T, class Op>
__device__ __forceinline__ T rows_all(T x, Op op) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = op(__builtin_bit_cast(T, uint32_t(a[0])), __builtin_bit_cast(T, uint32_t(a[1])));
  const auto v = __builtin_bit_cast(uint32_t, x);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  x = op(__builtin_bit_cast(T, uint32_t(b[0])), __builtin_bit_cast(T, uint32_t(b[1])));
#endif
  return x;
}

// op over the two lanes l, l ^ 16.
template <class T, class Op>
__device__ __forceinline__ T pair_rows(T x, Op op) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto u = __builtin_bit_cast(uint32_t, x);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  x = op(__builtin_bit_cast(T, uint32_t(a[0])), __builtin_bit_cast(T, uint32_t(a[1])));
#endif
  return x;
}

// op over the wave.
template <class T, class Op>
__device__ __forceinline__ T wave_all(T x, Op op) {
  return rows_all(group_all<16>(x, op), op);
}

struct AddOp {
  template <class T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};
struct MinOp {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a < b ? a : b; }
};

}  // namespace
}  // namespace flce
