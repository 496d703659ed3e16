// A matrix product on CDNA4 matrix cores (gfx950) for rows of any length, stride and
// alignment, bf16 or float32: C[m][n] = sum_k B(m, k) A(n, k) in float32, tiles of TS x TS
// (128, or 64 where those leave CUs without work, and 32 of float32, whose matrix
// instruction is sixteen times slower than its loads are short). The head's product
// (gemm_bf16.h) takes 256 x 256 tiles of aligned bf16 rows; this one serves what that does
// not: float32, odd rows, and outputs of too few such tiles.
//
// A's rows are C's columns, so that a lane of the matrix instruction's result holds four
// consecutive columns of one row of C: bias, residual and output move 8 or 16 bytes a lane
// without a trip through LDS.
//
// Each operand is stored with k contiguous ([rows][k], form N) or with its rows contiguous
// ([k][rows], form T). A stage holds 128 bytes of k a row (64 bf16, 32 float32). A tile has
// few waves to hide a load behind, so several stages are under way at once: where every row
// starts at a multiple of 16 bytes (DIRECT) stages are loaded straight into LDS, four in turn,
// or three of the smaller tiles, of which another workgroup then fits beside (gradients of
// 2048 x 1024 x 1024: 20 us, with four 23, with two 24); otherwise two stages, loaded two
// ahead through registers. A lane reads 16
// bytes of k of a row at a time: eight bf16 feed one v_mfma_f32_16x16x32_bf16, four float32
// four v_mfma_f32_16x16x4_f32, both operands in the same order of k.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gemm_bf16.h"
#include "row_io.h"

namespace flce {
namespace {
namespace small {

constexpr int kThreads = 256;
template <int TS>
constexpr int kStageBytes = TS * 128;              // one operand, one stage
template <int TS>
constexpr int kChunks = TS * 8 / kThreads;         // 16-byte chunks of it a thread loads
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
// (row_t: the place of k-row k, its own inverse.)
template <class T, int TS>
__device__ __forceinline__ int row_t(int k) {
  // rows of 128 bytes of float32 lie two to the banks' window: the upper eight trade places
  // with their neighbours
  return sizeof(T) == 4 && TS == 32 ? k ^ ((k >> 3) & 1) : k;
}
template <class T, int TS>
__device__ __forceinline__ int lds_t(int k, int col) {
  if constexpr (sizeof(T) == 2) {
    // a transposed read takes 32 bytes of four k-rows and of the four 8 rows on: with rows
    // of 256 bytes as the head's transposed tiles (gemm_index.h), with rows of 128 (two to
    // the banks' window) the second pair of rows and the second four move aside
    const int swz = TS == 128 ? gemm::swz_t(k) : (k & 2) ^ ((k >> 1) & 4);
    return (k * (TS / 8) + ((col >> 3) ^ swz)) * 16 + ((col >> 2) & 1) * 8;
  } else {
    // a fragment read takes 16 columns of four k-rows 4 apart: 16 banks each
    return row_t<T, TS>(k) * (TS * 4) + (col ^ (((k >> 2) & (TS == 32 ? 1 : 3)) << 4)) * 4;
  }
}

// The loads of a thread: its chunks of an operand's stage. Chunk `id` of the stage's LDS
// holds the one that the swizzles (which undo themselves) put there, so that a wave's
// direct loads fill consecutive places.
template <class T, int FORM, int TS>
struct Loads {
  static constexpr int E = kPerChunk<T>, C = kChunks<TS>;
  const T* at[C];
  int lds[C];
  int64_t step;                                    // elements between stages
  int row[C], k[C];                                // tile row (column) and stage k of chunk i
  __device__ __forceinline__ Loads(const Operand<T>& o, int64_t r0, int tid) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int id = tid + kThreads * i;
      lds[i] = id * 16;
      if constexpr (FORM == 0) {
        row[i] = id >> 3;
        k[i] = ((lds_n(row[i], id & 7) >> 4) & 7) * E;
        const int64_t r = r0 + row[i] < o.rows ? r0 + row[i] : o.rows - 1;
        at[i] = o.p + r * o.ld + k[i];
      } else {
        constexpr int kPerRow = TS / E;
        k[i] = row_t<T, TS>(id / kPerRow);
        row[i] = ((lds_t<T, TS>(k[i], (id % kPerRow) * E) >> 4) % kPerRow) * E;
        const int64_t c = r0 + row[i] < o.rows ? r0 + row[i] : 0;
        at[i] = o.p + int64_t(k[i]) * o.ld + c;
      }
    }
    step = FORM == 0 ? kStageK<T> : int64_t(kStageK<T>) * o.ld;
  }
  __device__ __forceinline__ void load(row_u32x4 (&v)[C], int64_t stage) const {
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = load_raw(at[i] + stage * step);
  }
  // The stage from k0, whose k past the end are zero: element by element, without a
  // condition on a load (each would be waited for before the next).
  __device__ __forceinline__ void load_end(row_u32x4 (&v)[C], const Operand<T>& o, int64_t r0,
                                           int64_t k0, int64_t K) const {
    T x[C][E];
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int64_t kk = k0 + k[i], r = r0 + row[i];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t ke = FORM == 0 ? kk + e : kk, re = FORM == 0 ? r : r + e;
        const int64_t kc = ke < K ? ke : K - 1, rc = re < o.rows ? re : o.rows - 1;
        x[i][e] = FORM == 0 ? o.p[rc * o.ld + kc] : o.p[kc * o.ld + rc];
      }
    }
#pragma unroll
    for (int i = 0; i < C; ++i) {
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e)
        f[e] = k0 + k[i] + (FORM == 0 ? e : 0) < K ? to_f32(x[i][e]) : 0.f;
      v[i] = pack_chunk<T>(f);
    }
  }
  // Straight into LDS: the wave's chunks i fill 1 KiB of the stage.
  __device__ __forceinline__ void direct(char* stage, int64_t s, int wave) const {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < C; ++i)
      __builtin_amdgcn_global_load_lds(
          at[i] + s * step,
          (__attribute__((address_space(3))) void*)(stage + (kThreads * i + wave * 64) * 16), 16, 0,
          0);
#else
    (void)stage, (void)s, (void)wave;
#endif
  }
  __device__ __forceinline__ void store(char* stage, const row_u32x4 (&v)[C]) const {
#pragma unroll
    for (int i = 0; i < C; ++i) *reinterpret_cast<row_u32x4*>(stage + lds[i]) = v[i];
  }
};

// 16 bytes of k (part p of two: chunk 4 p + lane / 16) of rows row_base + lane % 16.
template <class T, int FORM, int TS>
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
          (lds_s16x4*)(stage + lds_t<T, TS>(32 * p + 8 * g + 4 * r + (i >> 2), row_base + 4 * (i & 3))));
#endif
    const s16x8 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(row_u32x4, v);
  } else {
    row_u32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      v[e] = *reinterpret_cast<const uint32_t*>(stage + lds_t<T, TS>(16 * p + 4 * g + e, row_base + i));
    return v;
  }
}

// A wave's part, TS / 2 a side: acc[i][j][e] is column 16 i + 4 (lane / 16) + e, row
// 16 j + lane % 16.
template <int TS>
struct Acc {
  static constexpr int B = TS / 32;
  f32x4 v[B][B];
};

template <class T, int FA, int FB, int TS>
__device__ __forceinline__ void multiply(Acc<TS>& acc, const char* sa, const char* sb, int wa,
                                         int wb, int lane) {
  constexpr int B = Acc<TS>::B;
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    row_u32x4 fa[B], fb[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      fa[i] = read_frag<T, FA, TS>(sa, wa + 16 * i, p, lane);
      fb[i] = read_frag<T, FB, TS>(sb, wb + 16 * i, p, lane);
    }
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < B; ++i)
#pragma unroll
        for (int j = 0; j < B; ++j)
          acc.v[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, fa[i]), __builtin_bit_cast(bf16x8, fb[j]), acc.v[i][j], 0,
              0, 0);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < B; ++i)
#pragma unroll
          for (int j = 0; j < B; ++j)
            acc.v[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __uint_as_float(fa[i][e]), __uint_as_float(fb[j][e]), acc.v[i][j], 0, 0, 0);
    }
#endif
  }
}

// LDS of a tile: its stages of two operands.
template <int TS, bool DIRECT>
constexpr int kStages = !DIRECT ? 2 : TS == 128 ? 4 : 3;
template <int TS, bool DIRECT>
constexpr int kSmemBytes = 2 * kStages<TS, DIRECT> * kStageBytes<TS>;

// Waits until at most N of the wave's loads are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// One stage of the direct loop. What is read and what is loaded into are different stages
// (__restrict__: the compiler does not order them); the loop's waits and barriers order the
// rest.
template <class T, int FA, int FB, int TS>
__device__ __forceinline__ void direct_step(Acc<TS>& acc, const Loads<T, FA, TS>& la,
                                            const Loads<T, FB, TS>& lb, int64_t load_stage,
                                            const char* __restrict__ read, char* __restrict__ into,
                                            int wa, int wb, int wave, int lane) {
  la.direct(into, load_stage, wave);
  lb.direct(into + kStageBytes<TS>, load_stage, wave);
  multiply<T, FA, FB, TS>(acc, read, read + kStageBytes<TS>, wa, wb, lane);
}

// The tile at column a0, row b0 over k of [0, K). DIRECT: every stored row of both operands
// starts at a multiple of 16 bytes, and form T rows are whole chunks.
template <class T, int FA, int FB, int TS, bool DIRECT>
__device__ __forceinline__ void tile(Acc<TS>& acc, const Operand<T>& A, const Operand<T>& B,
                                     int64_t a0, int64_t b0, int64_t K, char* smem) {
  constexpr int SB = kStageBytes<TS>, C = kChunks<TS>, NS = kStages<TS, DIRECT>;
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wa = (w & 1) * (TS / 2), wb = (w >> 1) * (TS / 2);
#pragma unroll
  for (int i = 0; i < Acc<TS>::B; ++i)
#pragma unroll
    for (int j = 0; j < Acc<TS>::B; ++j) acc.v[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const Loads<T, FA, TS> la(A, a0, tid);
  const Loads<T, FB, TS> lb(B, b0, tid);
  auto st_a = [&](int s) { return smem + s * 2 * SB; };
  auto st_b = [&](int s) { return smem + s * 2 * SB + SB; };
  // Whole stages are loaded without conditions. A form T chunk at the end of a row may
  // run up to 7 elements into the rows behind it (columns that are not stored): the last 8
  // k-rows are then left to the masked loads.
  const bool over = !DIRECT && ((FA == 1 && A.rows % kPerChunk<T> != 0) ||
                                (FB == 1 && B.rows % kPerChunk<T> != 0));
  const int64_t safe = over ? (K > 8 ? K - 8 : 0) : K;
  const int64_t full = safe / kStageK<T>;
  for (int64_t k0 = full * kStageK<T>; k0 < K; k0 += kStageK<T>) {      // once or twice
    row_u32x4 ea[C], eb[C];
    la.load_end(ea, A, a0, k0, K);
    lb.load_end(eb, B, b0, k0, K);
    la.store(st_a(NS - 1), ea);
    lb.store(st_b(NS - 1), eb);
    __syncthreads();
    multiply<T, FA, FB, TS>(acc, st_a(NS - 1), st_b(NS - 1), wa, wb, lane);
    __syncthreads();
  }
  if (full == 0) return;
  // past the last stage that one is loaded again, so that as many loads are always under way
  auto at = [&](int64_t s) { return s < full ? s : full - 1; };
  if constexpr (DIRECT) {
#pragma unroll
    for (int s = 0; s < NS - 1; ++s) {
      la.direct(st_a(s), at(s), w);
      lb.direct(st_b(s), at(s), w);
    }
    int stage = 0;
    for (int64_t s = 0; s < full; ++s) {
      wait_loads<(NS - 2) * 2 * C>();              // this wave's part of stage s has landed
      stage_barrier();                             // every wave's; stage s - 1 is read
      const int into = stage == 0 ? NS - 1 : stage - 1;
      direct_step<T, FA, FB, TS>(acc, la, lb, at(s + NS - 1), st_a(stage), st_a(into), wa, wb, w,
                                 lane);
      stage = stage == NS - 1 ? 0 : stage + 1;
    }
    wait_loads<0>();
    stage_barrier();
  } else {
    row_u32x4 va[2][C], vb[2][C];
    auto load = [&](int u, int64_t s) {
      la.load(va[u], at(s));
      lb.load(vb[u], at(s));
    };
    load(0, 0);
    load(1, 1);
    la.store(st_a(0), va[0]);
    lb.store(st_b(0), vb[0]);
    __syncthreads();
    for (int64_t s0 = 0; s0 < full; s0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        load(u, s0 + u + 2);
        if (s0 + u < full) multiply<T, FA, FB, TS>(acc, st_a(u), st_b(u), wa, wb, lane);
        la.store(st_a(u ^ 1), va[u ^ 1]);
        lb.store(st_b(u ^ 1), vb[u ^ 1]);
        __syncthreads();
      }
    }
  }
}

// A lane's first column and row of the tile; it holds four columns from each 16th column on
// and each 16th row.
template <int TS>
__device__ __forceinline__ int64_t lane_col(int64_t a0) {
  return a0 + ((threadIdx.x >> 6) & 1) * (TS / 2) + 4 * ((threadIdx.x & 63) >> 4);
}
template <int TS>
__device__ __forceinline__ int64_t lane_row(int64_t b0) {
  return b0 + (threadIdx.x >> 7) * (TS / 2) + (threadIdx.x & 15);
}

}  // namespace small
}  // namespace
}  // namespace flce
