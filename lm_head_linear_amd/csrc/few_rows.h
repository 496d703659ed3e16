// Products of few tokens with a wide matrix W [V][H] of bf16 rows, W read once: the head of
// a decoding step.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gemm_bf16.h"

namespace flce {
namespace {

// ---- few tokens -----------------------------------------------------------------------
// A workgroup: 64 RB vocabulary rows, 16 RB of them a wave, and 16 NT tokens. A lane
// loads 16 bytes of W's row l % 16 at k = 8 (l / 16): the matrix instruction's operand
// as it is, no LDS. The h of a 128-k chunk is shared by the waves through LDS, two
// chunks in turn. Both come kAheadK chunks early, so that several KiB of W per wave
// are under way all the time. The loads of whole chunks have no condition (past the
// last one it is loaded again): a branch around a load makes the compiler wait for
// it as if the other way had been taken. The part of a chunk at the end of a row that
// is no multiple of 128 is read first, element by element where it leaves the row.
//
// Bound by reading W. Every workgroup reads all of h from L2 as well, so more than 32
// tokens take two row blocks a wave (us with one and two, W of 131072 x 4096: 1 token
// 211 and 226, 32 tokens 224 and 233, 64 tokens 254 and 241, 128 tokens 296 and 262;
// 48 tokens, 256000 x 3584: 451 and 411). Non-temporal loads of W are slower (48
// tokens: 533): the two halves of a 128-byte line come by two loads.
constexpr int kChunkK = 128;                       // k per chunk: four matrix steps
constexpr int kHld = kChunkK + 8;                  // elements of a token's chunk in LDS

// Eight elements of a row at p. ALIGN: bytes that every row starts at a multiple of:
// 16, 4 or 2. Odd rows of a 2-byte aligned matrix are read as aligned words and
// shifted: the element behind p + 7 is read with them.
template <int ALIGN>
__device__ __forceinline__ bf16x8 load_k8(const uint16_t* p) {
  typedef u32x4 __attribute__((aligned(4))) u32x4_word;
  if constexpr (ALIGN == 16) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p));
  } else if constexpr (ALIGN == 4) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4_word*>(p));
  } else {
    const bool odd = (reinterpret_cast<uintptr_t>(p) & 2) != 0;
    const uint16_t* q = odd ? p - 1 : p;
    const u32x4 v = *reinterpret_cast<const u32x4_word*>(q);
    const uint32_t e = *reinterpret_cast<const uint32_t*>(odd ? q + 8 : q + 6);
    const uint32_t sh = odd ? 16 : 0;
    return __builtin_bit_cast(bf16x8, u32x4{__builtin_amdgcn_alignbit(v[1], v[0], sh),
                                            __builtin_amdgcn_alignbit(v[2], v[1], sh),
                                            __builtin_amdgcn_alignbit(v[3], v[2], sh),
                                            __builtin_amdgcn_alignbit(e, v[3], sh)});
  }
}
// The same at k of a row of H elements, zero past it.
template <int ALIGN>
__device__ __forceinline__ bf16x8 load_k8_end(const uint16_t* row, int64_t k, int64_t H) {
  typedef __attribute__((ext_vector_type(8))) uint16_t u16x8;
  if (ALIGN != 2 && k + 8 <= H) return load_k8<ALIGN>(row + k);
  u16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = k + e < H ? row[k + e] : uint16_t(0);
  return __builtin_bit_cast(bf16x8, v);
}

template <int NT, int RB>
union FewSmem {
  uint16_t h[2][16 * NT][kHld];
  float z[16 * NT][64 * RB + 4];
};
// Lanes of a token in the epilogues of such a tile (48 tokens: whole waves idle).
template <int NT>
constexpr int kFewLanes = NT == 3 ? 4 : 256 / (16 * NT);

// The tile's products in sm.z: 64 RB rows from v0 of the V rows of W, tokens 0 .. N - 1 of h
// (rows ldh apart; W's are dense).
template <int NT, int ALIGN, int RB>
__device__ __forceinline__ void few_logits(const uint16_t* __restrict__ h, int64_t ldh,
                                           const uint16_t* __restrict__ W, int64_t N, int64_t H,
                                           int64_t V, int64_t v0, FewSmem<NT, RB>& sm) {
  constexpr int kAheadK = NT == 8 ? 1 : NT >= 3 ? 2 : 3, R = kAheadK + 1;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 15, kg = (lane >> 4) * 8;
  const uint16_t* wrow[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t v = v0 + i * 64 + w * 16 + r;
    wrow[i] = W + (v < V ? v : V - 1) * H;
  }
  // h: load p of a thread is 16 bytes of token 16 p + tid / 16 at k = 8 (tid % 16)
  const int hr = tid >> 4, hk = (tid & 15) * 8;
  const uint16_t* hrow[NT];
#pragma unroll
  for (int p = 0; p < NT; ++p) hrow[p] = h + (16 * p + hr < N ? 16 * p + hr : N - 1) * ldh;
  bf16x8 a[R][4][RB], b[R][NT];
  auto load = [&](bf16x8 (&fa)[4][RB], bf16x8 (&fb)[NT], int64_t k0) {
#pragma unroll
    for (int p = 0; p < NT; ++p) fb[p] = load_k8<ALIGN>(hrow[p] + k0 + hk);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) fa[s][i] = load_k8<ALIGN>(wrow[i] + k0 + s * 32 + kg);
  };
  auto keep = [&](const bf16x8 (&fb)[NT], int half) {
#pragma unroll
    for (int p = 0; p < NT; ++p) *reinterpret_cast<bf16x8*>(&sm.h[half][16 * p + hr][hk]) = fb[p];
  };
  f32x4 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const bf16x8 (&fa)[4][RB], int half) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const bf16x8 f = *reinterpret_cast<const bf16x8*>(&sm.h[half][16 * j + r][s * 32 + kg]);
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][i], f, acc[i][j], 0, 0, 0);
      }
  };
  const int64_t full = H / kChunkK, end = full * kChunkK;
  auto chunk_k = [&](int64_t c) { return (c < full ? c : full - 1) * kChunkK; };
  if (end < H) {                                   // the end of the rows
    bf16x8 ea[4][RB], eb[NT];
#pragma unroll
    for (int p = 0; p < NT; ++p) eb[p] = load_k8_end<ALIGN>(hrow[p], end + hk, H);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) ea[s][i] = load_k8_end<ALIGN>(wrow[i], end + s * 32 + kg, H);
    keep(eb, 1);
    __syncthreads();
    multiply(ea, 1);
  }
  if (full > 0) {
#pragma unroll
    for (int u = 0; u < kAheadK; ++u) load(a[u], b[u], chunk_k(u));
    keep(b[0], 0);
    __syncthreads();
    for (int64_t c0 = 0; c0 < full; c0 += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        load(a[(u + kAheadK) % R], b[(u + kAheadK) % R], chunk_k(c0 + u + kAheadK));
        const int half = int(c0 + u) & 1;
        if (c0 + u < full) multiply(a[u], half);
        keep(b[(u + 1) % R], half ^ 1);
        __syncthreads();
      }
    }
  }
  __syncthreads();
  // acc[i][j][e]: row 64 i + 16 w + 4 (lane / 16) + e, token 16 j + lane % 16
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(&sm.z[16 * j + r][64 * i + 16 * w + (lane >> 4) * 4]) = acc[i][j];
  __syncthreads();
}

// run(token blocks, row blocks a wave) of the variant for N tokens (up to 128).
template <class F>
void with_few(int64_t N, F&& run) {
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (N <= 16) run(One{}, One{});
  else if (N <= 32) run(Two{}, One{});
  else if (N <= 48) run(std::integral_constant<int, 3>{}, Two{});
  else if (N <= 64) run(std::integral_constant<int, 4>{}, Two{});
  else run(std::integral_constant<int, 8>{}, Two{});
}

}  // namespace
}  // namespace flce
