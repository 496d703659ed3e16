// Dropout's mask: ten rounds of the counter-based generator Philox 4x32 (J. Salmon,
// M. Moraes, R. Dror, D. Shaw: "Parallel random numbers: as easy as 1, 2, 3", SC 2011).
// The key is the seed, the counter (column / 8, row, offset): one call gives 128 bits,
// 16 for each of eight columns of a row. A value is kept where its 16 bits are at least
// round(65536 p). Nothing is stored: the backward forms the same mask again.
//
// 16 bits an element, and not 32, so that a call serves the eight values of a 16-byte
// chunk of bf16: its 20 products of 32 bits run at a quarter of the vector rate, and with
// a call for every four values they, not memory, would bound a row's pass.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ops_plan.h"
#include "row_io.h"

namespace flce {
namespace {

struct Mask8 {
  uint32_t w[4];               // columns 2 i and 2 i + 1 of the block in the halves of w[i]
};

// The state a thread keeps: the key, and the offset with the device's step added.
struct DropKey {
  uint32_t k0, k1, o0, o1;
};
__device__ __forceinline__ DropKey drop_key(const DropSpec& d) {
  const uint64_t o = d.offset + (d.step ? uint64_t(*d.step) : 0);
  return DropKey{uint32_t(d.seed), uint32_t(d.seed >> 32), uint32_t(o), uint32_t(o >> 32)};
}

__device__ __forceinline__ Mask8 drop_bits(const DropKey& k, uint32_t row, uint32_t block) {
  uint32_t a = block, b = row, c = k.o0, d = k.o1, k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = uint64_t(a) * 0xD2511F53u, q = uint64_t(c) * 0xCD9E8D57u;
    a = uint32_t(q >> 32) ^ b ^ k0;
    b = uint32_t(q);
    c = uint32_t(p >> 32) ^ d ^ k1;
    d = uint32_t(p);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Mask8{{a, b, c, d}};
}

// Whether value e of the chunk that starts at column c (a whole chunk's multiple) stays.
__device__ __forceinline__ bool drop_keeps(const Mask8& m, int e, uint32_t threshold) {
  const uint32_t w = m.w[e >> 1];
  return ((e & 1) ? w >> 16 : w & 0xffffu) >= threshold;
}

// The mask of E (4 or 8) values from column c of a row, the first in bits 0 .. 15 of w[0].
template <int E>
__device__ __forceinline__ Mask8 drop_chunk(const DropKey& k, int64_t row, int64_t c) {
  Mask8 m = drop_bits(k, uint32_t(row), uint32_t(c >> 3));
  if (E == 4 && (c & 4)) {
    m.w[0] = m.w[2];
    m.w[1] = m.w[3];
  }
  return m;
}

}  // namespace
}  // namespace flce
