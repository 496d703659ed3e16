// A matrix product on CDNA4 matrix cores (gfx950) for rows of any length, stride and
// alignment, bf16 or float32: C[m][n] = sum_k B(m, k) A(n, k) in float32, tiles of 128 x
// 128. The head's product (gemm_bf16.h) takes 256 x 256 tiles of aligned bf16 rows; this
// one serves what that does not: float32, odd rows, and outputs of too few such tiles.
//
// A's rows are C's columns, so that a lane of the matrix instruction's result holds four
// consecutive columns of one row of C: bias, residual and output move 8 or 16 bytes a lane
// without a trip through LDS.
//
// Each operand is stored with k contiguous ([rows][k], form N) or with its rows contiguous
// ([k][rows], form T). A stage holds 128 bytes of k a row (64 bf16, 32 float32), two in
// turn; the loads of the next one are under way while one is multiplied. A lane reads 16
// bytes of k of a row at a time: eight bf16 feed one v_mfma_f32_16x16x32_bf16, four float32
// four v_mfma_f32_16x16x4_f32, both operands in the same order of k.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm_index.h"
#include "row_io.h"

namespace flce {
namespace {
namespace small {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;

constexpr int kTile = 128, kThreads = 256;
constexpr int kStageBytes = kTile * 128;           // one operand, one stage
// k of a stage, and of a 16-byte chunk.
template <class T>
constexpr int kStageK = 128 / int(sizeof(T));

// An operand: rows x K elements, ld between stored rows.
template <class T>
struct Operand {
  const T* p;
  int64_t ld, rows;
};

// LDS byte of 16-byte chunk c (of 8) of row r, form N: swizzled so that the 16 rows of a
// fragment read lie in different banks.
__device__ __forceinline__ int lds_n(int r, int c) { return (r * 8 + (c ^ ((r >> 1) & 7))) * 16; }
// LDS byte of columns [col, col + 16 / sizeof(T)) of k-row k, form T.
template <class T>
__device__ __forceinline__ int lds_t(int k, int col) {
  if constexpr (sizeof(T) == 2) {
    // as the head's transposed tiles, rows of 256 bytes (gemm_index.h)
    return (k * 16 + ((col >> 3) ^ gemm::swz_t(k))) * 16 + ((col >> 2) & 1) * 8;
  } else {
    // a fragment read takes 16 columns of four k-rows 4 apart: 16 banks each
    return k * 512 + (col ^ (((k >> 2) & 3) << 4)) * 4;
  }
}

// The loads of a thread: chunk i (of 4) of an operand's stage.
template <class T, int FORM>
struct Loads {
  static constexpr int E = kPerChunk<T>;
  const T* at[4];
  int lds[4];
  int64_t step;                                    // elements between stages
  int row[4], k[4];                                // tile row (column) and stage k of chunk i
  __device__ __forceinline__ Loads(const Operand<T>& o, int64_t r0, int tid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int id = tid + kThreads * i;
      if constexpr (FORM == 0) {
        row[i] = id >> 3;
        k[i] = (id & 7) * E;
        const int64_t r = r0 + row[i] < o.rows ? r0 + row[i] : o.rows - 1;
        at[i] = o.p + r * o.ld + k[i];
        lds[i] = lds_n(row[i], id & 7);
      } else {
        constexpr int kPerRow = kTile / E;
        k[i] = id / kPerRow;
        row[i] = (id % kPerRow) * E;
        const int64_t c = r0 + row[i] < o.rows ? r0 + row[i] : 0;
        at[i] = o.p + int64_t(k[i]) * o.ld + c;
        lds[i] = lds_t<T>(k[i], row[i]);
      }
    }
    step = FORM == 0 ? kStageK<T> : int64_t(kStageK<T>) * o.ld;
  }
  __device__ __forceinline__ void load(row_u32x4 (&v)[4], int64_t stage) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = load_raw(at[i] + stage * step);
  }
  // The stage from k0, whose k (and, form T, columns) past the end are zero.
  __device__ __forceinline__ void load_end(row_u32x4 (&v)[4], const Operand<T>& o, int64_t r0,
                                           int64_t k0, int64_t K) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float f[E];
      const int64_t kk = k0 + k[i], r = r0 + row[i];
      if constexpr (FORM == 0) load_chunk(o.p + (r < o.rows ? r : o.rows - 1) * o.ld, kk, K, f);
      else load_chunk(o.p + (kk < K ? kk : K - 1) * o.ld, r, kk < K ? o.rows : 0, f);
      v[i] = pack_chunk<T>(f);
    }
  }
  __device__ __forceinline__ void store(char* stage, const row_u32x4 (&v)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<row_u32x4*>(stage + lds[i]) = v[i];
  }
};

// 16 bytes of k (part p of two: chunk 4 p + lane / 16) of rows row_base + lane % 16.
template <class T, int FORM>
__device__ __forceinline__ row_u32x4 read_frag(const char* stage, int row_base, int p, int lane) {
  const int i = lane & 15, g = lane >> 4;
  if constexpr (FORM == 0) {
    return *reinterpret_cast<const row_u32x4*>(stage + lds_n(row_base + i, 4 * p + g));
  } else if constexpr (sizeof(T) == 2) {
    typedef __attribute__((ext_vector_type(4))) short s16x4;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    typedef __attribute__((ext_vector_type(8))) short s16x8;
    s16x4 h[2] = {};
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int r = 0; r < 2; ++r)
      h[r] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(stage + lds_t<T>(32 * p + 8 * g + 4 * r + (i >> 2), row_base + 4 * (i & 3))));
#endif
    const s16x8 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(row_u32x4, v);
  } else {
    row_u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = *reinterpret_cast<const uint32_t*>(stage + lds_t<T>(16 * p + 4 * g + e, row_base + i));
    return v;
  }
}

// A wave's 64 x 64 part: acc[i][j][e] is column 16 i + 4 (lane / 16) + e, row 16 j + lane % 16.
typedef f32x4 Acc[4][4];

template <class T, int FA, int FB>
__device__ __forceinline__ void multiply(Acc& acc, const char* sa, const char* sb, int wa, int wb,
                                         int lane) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    row_u32x4 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i] = read_frag<T, FA>(sa, wa + 16 * i, p, lane);
      fb[i] = read_frag<T, FB>(sb, wb + 16 * i, p, lane);
    }
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, fa[i]), __builtin_bit_cast(bf16x8, fb[j]), acc[i][j], 0,
              0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __uint_as_float(fa[i][e]), __uint_as_float(fb[j][e]), acc[i][j], 0, 0, 0);
    }
#endif
  }
}

// The tile at column a0, row b0 over k of [0, K).
template <class T, int FA, int FB>
__device__ __forceinline__ void tile(Acc& acc, const Operand<T>& A, const Operand<T>& B, int64_t a0,
                                     int64_t b0, int64_t K, char* smem) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int wa = (w & 1) * 64, wb = (w >> 1) * 64;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const Loads<T, FA> la(A, a0, tid);
  const Loads<T, FB> lb(B, b0, tid);
  auto st_a = [&](int64_t s) { return smem + (s & 1) * 2 * kStageBytes; };
  auto st_b = [&](int64_t s) { return smem + (s & 1) * 2 * kStageBytes + kStageBytes; };
  // Whole stages are loaded without conditions. A form T chunk at the end of a row may
  // run up to 7 elements into the rows behind it (columns that are not stored): the last 8
  // k-rows are then left to the masked loads.
  const bool over = (FA == 1 && A.rows % kPerChunk<T> != 0) || (FB == 1 && B.rows % kPerChunk<T> != 0);
  const int64_t safe = over ? (K > 8 ? K - 8 : 0) : K;
  const int64_t full = safe / kStageK<T>;
  row_u32x4 va[4], vb[4];
  for (int64_t k0 = full * kStageK<T>; k0 < K; k0 += kStageK<T>) {      // once or twice
    la.load_end(va, A, a0, k0, K);
    lb.load_end(vb, B, b0, k0, K);
    la.store(st_a(1), va);
    lb.store(st_b(1), vb);
    __syncthreads();
    multiply<T, FA, FB>(acc, st_a(1), st_b(1), wa, wb, lane);
    __syncthreads();
  }
  if (full > 0) {
    la.load(va, 0);
    lb.load(vb, 0);
    la.store(st_a(0), va);
    lb.store(st_b(0), vb);
    __syncthreads();
    for (int64_t s = 0; s < full; ++s) {
      const int64_t next = s + 1 < full ? s + 1 : s;                   // the last one again
      la.load(va, next);
      lb.load(vb, next);
      multiply<T, FA, FB>(acc, st_a(s), st_b(s), wa, wb, lane);
      la.store(st_a(s + 1), va);
      lb.store(st_b(s + 1), vb);
      __syncthreads();
    }
  }
}

// f(column, row, four values of consecutive columns) for a lane's part of the tile.
template <class F>
__device__ __forceinline__ void for_acc(const Acc& acc, int64_t a0, int64_t b0, F f) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c0 = a0 + (w & 1) * 64 + 4 * (lane >> 4), r0 = b0 + (w >> 1) * 64 + (lane & 15);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) f(c0 + 16 * i, r0 + 16 * j, acc[i][j]);
}

}  // namespace small
}  // namespace
}  // namespace flce
