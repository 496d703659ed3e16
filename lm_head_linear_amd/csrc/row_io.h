// Rows of bf16 or float32 values moved in 16-byte chunks at any element
// alignment (global loads and stores of gfx950 need none), as float32 in
// registers.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace flce {
namespace {

typedef __attribute__((ext_vector_type(4))) uint32_t row_u32x4;
typedef row_u32x4 __attribute__((aligned(2))) row_u32x4_any;
typedef uint16_t Bf16Bits;                          // a bf16 value in memory

// Values per 16-byte chunk of T (Bf16Bits or float).
template <class T>
constexpr int kPerChunk = 16 / int(sizeof(T));

__device__ __forceinline__ float to_f32(Bf16Bits b) { return __uint_as_float(uint32_t(b) << 16); }
__device__ __forceinline__ float to_f32(float x) { return x; }

// Rounded to nearest even (v_cvt_pk_bf16_f32), or as it is.
template <class T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ Bf16Bits from_f32<Bf16Bits>(float x) {
  return __builtin_bit_cast(uint16_t, __bf16(x));
}
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }

template <class T>
__device__ __forceinline__ void unpack_chunk(const row_u32x4& v, float (&f)[kPerChunk<T>]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = __uint_as_float(v[e]);
  }
}

template <class T>
__device__ __forceinline__ row_u32x4 pack_chunk(const float (&f)[kPerChunk<T>]) {
  row_u32x4 v;
  if constexpr (sizeof(T) == 2) {
    typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bf16x2 p = {__bf16(f[2 * e]), __bf16(f[2 * e + 1])};
      v[e] = __builtin_bit_cast(uint32_t, p);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(f[e]);
  }
  return v;
}

__device__ __forceinline__ row_u32x4 load_raw(const void* p) {
  return *static_cast<const row_u32x4_any*>(p);
}

// Elements [c, c + kPerChunk) of a row of n elements: zero past the end.
template <class T>
__device__ __forceinline__ void load_chunk(const T* row, int64_t c, int64_t n,
                                           float (&f)[kPerChunk<T>]) {
  constexpr int E = kPerChunk<T>;
  if (c + E <= n) {
    unpack_chunk<T>(load_raw(row + c), f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = c + e < n ? to_f32(row[c + e]) : 0.f;
  }
}

// The same in two steps for rows of whole chunks (n a multiple of a chunk): the load, without
// a condition that would have it waited for before the next one is issued, and the values.
template <class T>
__device__ __forceinline__ row_u32x4 load_whole(const T* row, int64_t c, int64_t n) {
  return load_raw(row + (c < n ? c : 0));
}
template <class T>
__device__ __forceinline__ void unpack_whole(const row_u32x4& v, int64_t c, int64_t n,
                                             float (&f)[kPerChunk<T>]) {
  unpack_chunk<T>(c < n ? v : row_u32x4{0u, 0u, 0u, 0u}, f);
}

template <class T>
__device__ __forceinline__ void store_chunk(T* row, int64_t c, int64_t n,
                                            const float (&f)[kPerChunk<T>]) {
  constexpr int E = kPerChunk<T>;
  if (c + E <= n) {
    *reinterpret_cast<row_u32x4_any*>(row + c) = pack_chunk<T>(f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e < n) row[c + e] = from_f32<T>(f[e]);
  }
}

}  // namespace
}  // namespace flce
