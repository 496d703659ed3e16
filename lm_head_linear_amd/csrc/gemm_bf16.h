// The bf16 GEMM core on CDNA4 matrix cores (gfx950), shared by the kernels that
// multiply by the head's weight: direct-to-LDS operand loads, the pipelined K
// loop, the launch of one tile grid, and the token-major stores its epilogues
// share. Included by the .hip files that instantiate it with their epilogues.
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "flce_internal.h"
#include "gemm_index.h"

namespace flce {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr int kBM = gemm::kBM;
constexpr int kThreads = 256;
constexpr int kWaveScratch = 32768;               // LDS bytes per wave in the epilogues
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float bf16_to_f32(uint16_t b) {
  return __uint_as_float(uint32_t(b) << 16);
}
__device__ __forceinline__ uint16_t f32_to_bf16(float f) {
  // Round to nearest even (v_cvt_pk_bf16_f32 on gfx950).
  return __builtin_bit_cast(uint16_t, __bf16(f));
}
// Two values rounded to nearest even and packed (lo = a) in one instruction.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const bf16x2 v = {__bf16(a), __bf16(b)};
  return __builtin_bit_cast(uint32_t, v);
}

using gemm::Geom;
using gemm::kBK;

// An operand of the GEMM: a pointer and its geometry (see gemm_index.h).
struct Operand {
  const uint16_t* ptr;
  Geom g;
};

// Per-thread state of one operand's direct-to-LDS loads: a wave-uniform tile
// base advanced by `kstep` bytes per stage tile, and one 32-bit byte offset
// per load (see gemm::direct_lane for the layout and the edge clamping).
template <int L>
struct DirectLoads {
  const char* base;
  int64_t kstep;
  uint32_t off[L];
};

template <int FORM, int SK>
__device__ __forceinline__ DirectLoads<gemm::loads_per_operand(SK)> setup_direct(
    const Operand& op, int64_t row0, int wave, int lane) {
  constexpr int L = gemm::loads_per_operand(SK);
  DirectLoads<L> d;
  d.base = reinterpret_cast<const char*>(op.ptr + gemm::direct_base(FORM, op.g, row0));
  d.kstep = gemm::direct_kstep(FORM, op.g, SK) * 2;
#pragma unroll
  for (int q = 0; q < L; ++q)
    d.off[q] = uint32_t(gemm::direct_lane(FORM, op.g, row0, wave, lane, q, SK) * 2);
  return d;
}

// Issue one stage tile of direct loads into an LDS tile (256 x SK bf16): load
// q of wave w fills LDS bytes [(L w + q) KiB, +1 KiB), lane l writing 16 B at
// 16 l.
template <int L>
__device__ __forceinline__ void issue_direct(const DirectLoads<L>& d, int64_t kt, char* lds,
                                             int wave) {
#if defined(__HIP_DEVICE_COMPILE__)   // the host pass instantiates templates without gfx950 builtins
  const char* b = d.base + kt * d.kstep;
#pragma unroll
  for (int q = 0; q < L; ++q)
    __builtin_amdgcn_global_load_lds(
        b + d.off[q], (__attribute__((address_space(3))) void*)(lds + (L * wave + q) * 1024), 16,
        0, 0);
#else
  (void)d, (void)kt, (void)lds, (void)wave;
#endif
}

// Load q (0 .. L-1) of issue_direct alone.
template <int L>
__device__ __forceinline__ void issue_one(const DirectLoads<L>& d, int64_t kt, char* lds, int wave,
                                          int q) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_global_load_lds(
      d.base + kt * d.kstep + d.off[q],
      (__attribute__((address_space(3))) void*)(lds + (L * wave + q) * 1024), 16, 0, 0);
#else
  (void)d, (void)kt, (void)lds, (void)wave, (void)q;
#endif
}

// Per-token inputs of an epilogue, staged in LDS past the pipeline stages:
// W 4-byte words per token (W = 1 for float, 2 for int64) of the workgroup's
// 256 token columns n0 .. n0 + 255 (clamped to the last of n tokens), loaded
// with direct-to-LDS loads when the kernel starts, so that their latency
// passes under the K loop instead of stalling the epilogue. Thread tid of
// wave w issues word e = q * 256 + tid of pass q into lds[4 e].
template <int W>
__device__ __forceinline__ void stage_tokens(char* lds, const void* src, int64_t n0, int64_t n,
                                             int wave, int lane) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int q = 0; q < W; ++q) {
    const int e = q * 256 + wave * 64 + lane;
    const int64_t t = n0 + e / W;
    const char* p = static_cast<const char*>(src) + ((t < n ? t : n - 1) * W + e % W) * 4;
    __builtin_amdgcn_global_load_lds(
        p, (__attribute__((address_space(3))) void*)(lds + (q * 256 + wave * 64) * 4), 4, 0, 0);
  }
#else
  (void)lds, (void)src, (void)n0, (void)n, (void)wave, (void)lane;
#endif
}

// Register path for a partial last stage tile: zero-filled past K (and past
// the matrix edge), then stored into the same LDS layout.
template <int FORM, int SK>
__device__ __forceinline__ void load_tail(u32x4 (&r)[gemm::tail_loads(SK)], const Operand& op,
                                          int64_t row0, int64_t k0, int tid) {
#pragma unroll
  for (int i = 0; i < gemm::tail_loads(SK); ++i) {
    int64_t off;
    const bool ok = gemm::tail_src(FORM, op.g, row0, k0, tid + 256 * i, SK, off);
    r[i] = ok ? *reinterpret_cast<const u32x4*>(op.ptr + off) : u32x4{0u, 0u, 0u, 0u};
  }
}

template <int FORM, int SK>
__device__ __forceinline__ void store_tail(char* lds, const u32x4 (&r)[gemm::tail_loads(SK)],
                                           int tid) {
#pragma unroll
  for (int i = 0; i < gemm::tail_loads(SK); ++i)
    *reinterpret_cast<u32x4*>(lds + gemm::tail_lds_pos(FORM, tid + 256 * i, SK) * 16) = r[i];
}

// MFMA fragment of 16 rows (row_base .. row_base + 15 of the tile) for the
// 32-wide K part p (0 .. SK/32 - 1) of a stage tile: lane l holds row
// row_base + l % 16 at k = 32 p + 8 (l / 16) + 0..7. Both operands use the
// same k order, which is all the product needs.
template <int FORM, int SK>
__device__ __forceinline__ bf16x8 read_frag(const char* lds, int row_base, int p, int lane) {
  if (FORM == 0) {
    const int row = row_base + (lane & 15);
    const int c = 4 * p + (lane >> 4);
    const u32x4 v = *reinterpret_cast<const u32x4*>(lds + gemm::lds_chunk_n(row, c, SK) * 16);
    return __builtin_bit_cast(bf16x8, v);
  } else {
    // Lane i of a 16-lane group receives element i % 4 of the 8-byte chunks
    // read by lanes 4e + i / 4 (e = 0..3): lane i reads k-row base + i / 4 at
    // columns 4 (i % 4) .. + 3, so lane i gets column i at k-rows base + 0..3.
    typedef __attribute__((ext_vector_type(4))) short s16x4;
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int g = lane >> 4, i = lane & 15;
    const int col = row_base + 4 * (i & 3);
    s16x4 h[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = 32 * p + 8 * g + 4 * r + (i >> 2);
      h[r] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lds + gemm::lds_byte_t(k, col)));
    }
    typedef __attribute__((ext_vector_type(8))) short s16x8;
    const s16x8 v = {h[0][0], h[0][1], h[0][2], h[0][3], h[1][0], h[1][1], h[1][2], h[1][3]};
    return __builtin_bit_cast(bf16x8, v);
  }
}

// A wave's accumulators: 8 x 8 blocks of 16 x 16, four values per lane.
// Element (i, j, r) sits at tile row wm*128 + i*16 + 4*(lane/16) + r and
// tile column wn*128 + j*16 + lane%16 (the 16x16 MFMA output layout), so a
// lane holds 4 consecutive rows of each block and the four lanes l, l ^ 16,
// l ^ 32, l ^ 48 share its columns.
typedef f32x4 Acc[8][8];

__device__ __forceinline__ int acc_row(int wm, int i, int r, int lane) {
  return wm * 128 + i * 16 + 4 * (lane >> 4) + r;
}
__device__ __forceinline__ int acc_col(int wn, int j, int lane) {
  return wn * 128 + j * 16 + (lane & 15);
}

// Max and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48 that share an
// accumulator column, with the gfx950 lane swaps (VALU, no LDS round trip).
// permlane16_swap(x, x) yields x of lanes l & ~16 and l | 16, and
// permlane32_swap(x, x) those of lanes l & ~32 and l | 32, in that order in
// every lane, so all four lanes get the same bits.
__device__ __forceinline__ float col_max4(float x) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
#endif
  return x;
}
__device__ __forceinline__ float col_sum4(float x) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                  false);
  x = __uint_as_float(b[0]) + __uint_as_float(b[1]);
#endif
  return x;
}

// Waits of the K loop (gfx9 s_waitcnt encoding: vmcnt bits [3:0] and
// [15:14], expcnt [6:4], lgkmcnt [11:8]; a field at its maximum does not
// wait).
__device__ __forceinline__ void wait_vm24() { __builtin_amdgcn_s_waitcnt(0x4F78); }   // vmcnt(24)
__device__ __forceinline__ void wait_vm16() { __builtin_amdgcn_s_waitcnt(0x4F70); }   // vmcnt(16)
__device__ __forceinline__ void wait_vm8() { __builtin_amdgcn_s_waitcnt(0x0F78); }    // vmcnt(8)
__device__ __forceinline__ void wait_vm0() { __builtin_amdgcn_s_waitcnt(0x0F70); }    // vmcnt(0)
__device__ __forceinline__ void wait_vm0_lgkm0() { __builtin_amdgcn_s_waitcnt(0x0070); }

// Workgroup barrier for the K loop. Unlike __syncthreads() it implies no
// memory fence or wait: the waits that order the pipeline are explicit
// before it. The empty asm statements keep the compiler from moving memory
// accesses across it, the scheduling barriers keep MFMAs on their side.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// MFMA fragments of one step (32 k) for the wave's 128 x 128 block: 32-wide
// part `part` of a stage tile, 8 row blocks of each operand.
struct StepFrags {
  bf16x8 a[8], b[8];
};

template <int FA, int FB, int SK>
__device__ __forceinline__ void read_step(StepFrags& f, const char* sa, const char* sb, int part,
                                          int wm, int wn, int lane) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f.a[i] = read_frag<FA, SK>(sa, wm * 128 + i * 16, part, lane);
#pragma unroll
  for (int j = 0; j < 8; ++j) f.b[j] = read_frag<FB, SK>(sb, wn * 128 + j * 16, part, lane);
}

__device__ __forceinline__ void mfma_step(Acc& acc, const StepFrags& f) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(f.a[i], f.b[j], acc[i][j], 0, 0, 0);
}

// Scheduling hints for a step of dH (K-contiguous G, transposed W): its 64
// MFMAs, the fragment reads of the next step after the first MFMAs (all in
// the first half of the step), and the NLOADS direct loads one after every
// second MFMA of the second half, so everything issues under the MFMAs.
template <int FA, int FB, int NLOADS>
__device__ __forceinline__ void interleave_hints() {
  constexpr int kReads = (FA == 0 ? 8 : 16) + (FB == 0 ? 8 : 16);
#pragma unroll
  for (int q = 0; q < 64; ++q) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);                    // MFMA
    const bool load = q >= 32 && q % 2 == 0 && (q - 32) / 2 < NLOADS;
    if (NLOADS > 0 && load) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM read
    if (q < kReads) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);    // DS read
  }
}

// One MFMA step: optionally start the direct loads of a stage tile into its
// (free) stage, read the fragments of the next step (32-wide part
// `next_part` of the stage tile at na/nb) and multiply the current step,
// whose fragments were read during the previous one. The stages are
// __restrict__ so the compiler does not order the direct-to-LDS writes
// against the reads; the real dependencies are the waits and the barriers.
//
// The forward/gradient GEMMs (both operands K-contiguous, 16 loads on every
// other step) and dW (both transposed, 8 loads per step) issue the step as 16
// chunks of 4 MFMAs, fenced by scheduling barriers: the fragment reads of the
// next step in chunks 0..7 (row block c of each operand in chunk c, after the
// first chunk's MFMAs, so that their wait for the current fragments does not
// include the new reads), and the direct loads one per chunk (A and B
// alternating) or one per chunk of the second half. Left to scheduling hints,
// the compiler bunched 14 of the 16 loads of the K-contiguous steps back to
// back. dH measured faster with the hints.
template <int FA, int FB, int SK, bool LOADS, int L>
__device__ __forceinline__ void k_step(Acc& acc, const StepFrags& cur, StepFrags& nxt,
                                       const DirectLoads<L>& da, const DirectLoads<L>& db,
                                       int64_t load_tile, const char* __restrict__ na,
                                       const char* __restrict__ nb, int next_part,
                                       char* __restrict__ la, char* __restrict__ lb, int wave,
                                       int wm, int wn, int lane) {
  if constexpr (FA != FB) {
    if (LOADS) {
      issue_direct<L>(da, load_tile, la, wave);
      issue_direct<L>(db, load_tile, lb, wave);
    }
    read_step<FA, FB, SK>(nxt, na, nb, next_part, wm, wn, lane);
    mfma_step(acc, cur);
    interleave_hints<FA, FB, LOADS ? 2 * L : 0>();
  } else {
    constexpr bool kNN = FA == 0;
    static_assert(2 * L == (kNN ? 16 : 8), "one load per chunk (of the second half)");
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int i = c >> 1;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const int j = 4 * (c & 1) + jj;
        acc[i][j] =
            __builtin_amdgcn_mfma_f32_16x16x32_bf16(cur.a[i], cur.b[j], acc[i][j], 0, 0, 0);
      }
      if (c == 0) __builtin_amdgcn_sched_barrier(0);
      if (c < 8) {
        nxt.a[c] = read_frag<FA, SK>(na, wm * 128 + c * 16, next_part, lane);
        nxt.b[c] = read_frag<FB, SK>(nb, wn * 128 + c * 16, next_part, lane);
      }
      if (LOADS) {
        if (kNN) {
          if (c & 1) issue_one<L>(db, load_tile, lb, wave, c >> 1);
          else       issue_one<L>(da, load_tile, la, wave, c >> 1);
        } else if (c >= 8) {
          const int q = c - 8;
          if (q < L) issue_one<L>(da, load_tile, la, wave, q);
          else       issue_one<L>(db, load_tile, lb, wave, q - L);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The K loop of one tile: acc += A[m0 .. m0 + 255][0, K) . B[n0 .. n0 + 255][0, K)^T
// through the LDS stages at smem: a partial last stage tile first (through
// registers), then the pipelined full stage tiles. Every wave leaves it
// behind a barrier, with no load in flight.
template <int FA, int FB>
__device__ __forceinline__ void k_loop(Acc& acc, const Operand& A, const Operand& B, int64_t K,
                                       int64_t m0, int64_t n0, char* smem, int tid, int lane,
                                       int wave, int wm, int wn) {
  constexpr int SK = gemm::stage_k(FA, FB);
  constexpr int kStages = gemm::num_stages(FA, FB);
  constexpr int L = gemm::loads_per_operand(SK);
  constexpr int kTileBytes = kBM * SK * 2;          // one operand, one stage

  const DirectLoads<L> da = setup_direct<FA, SK>(A, m0, wave, lane);
  const DirectLoads<L> db = setup_direct<FB, SK>(B, n0, wave, lane);
  const int64_t nfull = K / SK;                // stage tiles loaded directly
  const int64_t nk = (K + SK - 1) / SK;        // plus a zero-filled partial tile

  auto st_a = [&](int64_t t) { return smem + (t % kStages) * 2 * kTileBytes; };
  auto st_b = [&](int64_t t) { return smem + (t % kStages) * 2 * kTileBytes + kTileBytes; };
  if (nk > nfull) {
    // The partial last stage tile goes through registers, zero-filled past K,
    // into stage 0, and is multiplied first, before the pipelined loop, whose
    // prologue then reuses the stage (behind the barrier). Placed after the
    // loop instead, it made the register allocator shuffle the 64
    // accumulator tuples through copies and spills inside the loop.
    char* la = st_a(0);
    char* lb = st_b(0);
    u32x4 ta[gemm::tail_loads(SK)], tb[gemm::tail_loads(SK)];
    load_tail<FA, SK>(ta, A, m0, nfull * SK, tid);
    load_tail<FB, SK>(tb, B, n0, nfull * SK, tid);
    store_tail<FA, SK>(la, ta, tid);
    store_tail<FB, SK>(lb, tb, tid);
    __syncthreads();
    StepFrags ft;
#pragma unroll
    for (int part = 0; part < SK / 32; ++part) {
      read_step<FA, FB, SK>(ft, la, lb, part, wm, wn, lane);
      mfma_step(acc, ft);
    }
    __syncthreads();
  }
  if (nfull > 0) {
    const int64_t last = nfull - 1;
    StepFrags f[2];
    if constexpr (SK == 64) {
      // Two stages of 64 k, two MFMA steps (the two 32-wide halves) per stage
      // tile; stage tile t lives in stage t % 2 and the fragments of a step
      // are read during the step before it. Even step (first half of tile
      // t): multiply it, read the second half; no wait, no barrier. Odd step
      // (second half): wait until this wave's loads of tile t+1 have landed
      // and its reads of tile t have returned, then a barrier -- tile t+1 is
      // published and no wave reads tile t's stage any more -- so the loads
      // of tile t+2 go into it; read the first half of tile t+1. A tile's
      // loads thus have two steps to land. Every odd step issues one tile
      // (past the last one it re-loads the last into the free stage), so
      // the body has no branches for the scheduler to stop at.
      issue_direct<L>(da, 0, st_a(0), wave);
      issue_direct<L>(db, 0, st_b(0), wave);
      issue_direct<L>(da, last > 0 ? 1 : 0, st_a(1), wave);
      issue_direct<L>(db, last > 0 ? 1 : 0, st_b(1), wave);
      wait_vm16();                                 // tile 0 landed
      stage_barrier();
      read_step<FA, FB, SK>(f[0], st_a(0), st_b(0), 0, wm, wn, lane);
      for (int64_t t = 0; t < nfull; ++t) {
        __builtin_amdgcn_sched_barrier(0);
        k_step<FA, FB, SK, false>(acc, f[0], f[1], da, db, 0, st_a(t), st_b(t), 1, nullptr,
                                  nullptr, wave, wm, wn, lane);
        __builtin_amdgcn_sched_barrier(0);
        wait_vm0_lgkm0();
        stage_barrier();
        const int64_t lt = t + 2 < last ? t + 2 : last;
        k_step<FA, FB, SK, true>(acc, f[1], f[0], da, db, lt, st_a(t + 1), st_b(t + 1), 0,
                                 st_a(t), st_b(t), wave, wm, wn, lane);
      }
    } else {
      // Five stages of 32 k, one MFMA step per stage tile; tile t lives in
      // stage t % 5, is loaded 4 steps ahead and its fragments are read
      // during step t-1. Every step issues exactly one tile (past the last
      // one it re-loads the last into a free stage), so the number of loads
      // in flight at each wait is the same and the body has no branches for
      // the scheduler to stop at. A barrier only at even steps: the barrier
      // at the top of even step k publishes tiles k+1 and k+2 (only tile k+3
      // may still be in flight) and frees the stages of all tiles up to k,
      // whose fragments were read before it; step k loads tile k+4 into the
      // stage of tile k-1 and the odd step k+1 loads tile k+5 into the stage
      // of tile k. Stage indices advance by one per step in wave-uniform
      // registers (5 is not a power of two). With the LDS bank conflicts of
      // the transposed and 32-k reads removed, five stages measured faster
      // than four with a barrier per step for dH too (its launch 4% faster).
      static_assert(kStages == 5, "five stages of 32 k");
      auto next_stage = [](int x) { return x == kStages - 1 ? 0 : x + 1; };
#pragma unroll
      for (int t = 0; t < kStages - 1; ++t) {
        issue_direct<L>(da, t < last ? t : last, st_a(t), wave);
        issue_direct<L>(db, t < last ? t : last, st_b(t), wave);
      }
      wait_vm24();                                 // tile 0 landed (three more in flight)
      stage_barrier();
      read_step<FA, FB, SK>(f[0], st_a(0), st_b(0), 0, wm, wn, lane);
      int s_read = 1, s_load = kStages - 1;        // stages of tiles k+1 and k+4
      int64_t kt = 0;
      // two steps per iteration: the even one with the barrier, then the odd one
      for (; kt + 1 < nfull; kt += 2) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int64_t k = kt + u;
          __builtin_amdgcn_sched_barrier(0);
          if (u == 0) {
            wait_vm8();                            // all but the newest tile landed
            stage_barrier();
          }
          const int64_t lt = k + kStages - 1;
          char* sa = smem + s_read * 2 * kTileBytes;
          char* la = smem + s_load * 2 * kTileBytes;
          k_step<FA, FB, SK, true>(acc, f[u], f[u ^ 1], da, db, lt < last ? lt : last, sa,
                                   sa + kTileBytes, 0, la, la + kTileBytes, wave, wm, wn, lane);
          s_read = next_stage(s_read);
          s_load = next_stage(s_load);
        }
      }
      if (kt < nfull) {                            // odd number of steps: the last one (even)
        wait_vm8();
        stage_barrier();
        const int64_t lt = kt + kStages - 1;
        char* sa = smem + s_read * 2 * kTileBytes;
        char* la = smem + s_load * 2 * kTileBytes;
        k_step<FA, FB, SK, true>(acc, f[0], f[1], da, db, lt < last ? lt : last, sa,
                                 sa + kTileBytes, 0, la, la + kTileBytes, wave, wm, wn, lane);
      }
    }
    // the re-loads past the last tile may still be in flight
    wait_vm0();
    stage_barrier();
  }
}

// Which dimension of a launch is cut on the device to the count at `dyn`
// (the non-ignored tokens of a compact plan): none, M, N or K. The grid is
// sized for the launch's sizes (an upper bound); a cut M or N makes the tile
// raster run over the live tiles, and the workgroups past them leave at once,
// before any load.
enum Dyn : int { kDynNone = 0, kDynM = 1, kDynN = 2, kDynK = 3 };

// Whether an epilogue asks for the raster that deals M-tiles to the XCDs in
// turn (gemm::tile_coords): one whose first M-tiles do more work.
template <class E, class = void>
struct SpreadM : std::false_type {};
template <class E>
struct SpreadM<E, std::void_t<decltype(E::kSpreadM)>> : std::bool_constant<E::kSpreadM> {};

// LDS bytes of a GEMM's stages (reused by its epilogue: 32 KiB per wave).
template <int FA, int FB>
constexpr int stage_bytes() {
  return gemm::num_stages(FA, FB) * 2 * kBM * gemm::stage_k(FA, FB) * 2;
}

// One workgroup tile of a GEMM launch: workgroup `bid` of the launch's tile
// raster (and K segment `seg` of a split launch), with the LDS at smem: the
// stages, then the epilogue's per-token inputs.
template <int FA, int FB, class Epi, bool BA, int SEGS, bool SPLITK, int DYN>
__device__ __forceinline__ void gemm_tile(char* smem, int64_t bid, int seg, Operand A,
                                          Operand B, int64_t M, int64_t Nn, int64_t K,
                                          int group_m, Epi epi, int64_t a2_off,
                                          const int64_t* dyn) {
  // BA: operand A is the blocked G (gemm::Geom). Fixing blk at compile time
  // for the dense operands lets the address arithmetic drop the blocked case.
  // SEGS = 2: a second K loop over A shifted by a2_off elements (the lo half
  // of a split G) against the same B, into the same accumulators, so the
  // tile is (A + A2) . B^T with one epilogue.
  // SPLITK: the GEMM is split along K into segments of a2_off (a multiple of
  // 64); this workgroup takes segment `seg` and its epilogue writes a partial
  // product.
  static_assert(SEGS == 1 || SEGS == 2, "one or two K segments");
  static_assert(!(SPLITK && SEGS == 2), "a split GEMM has one K segment per workgroup");
  if constexpr (!BA) A.g.blk = 0;
  B.g.blk = 0;
  if constexpr (SPLITK) {
    epi.select_segment(seg);
    const int64_t k0 = int64_t(seg) * a2_off;
    K = (K - k0) < a2_off ? (K - k0) : a2_off;
    A.ptr += gemm::k_origin(FA, A.g, k0);
    B.ptr += gemm::k_origin(FB, B.g, k0);
    A.g.K = K;
    B.g.K = K;
  }
  constexpr int SK = gemm::stage_k(FA, FB);
  constexpr int kStages = gemm::num_stages(FA, FB);
  constexpr int L = gemm::loads_per_operand(SK);
  constexpr int kSmemBytes = stage_bytes<FA, FB>();      // 128 or 160 KiB
  static_assert(kSmemBytes >= 4 * kWaveScratch, "epilogue staging");
  static_assert(kBK == 32 && (SK == 32 || SK == 64), "MFMA steps of 32 k");
  static_assert(2 * L == (SK == 64 ? 16 : 8), "waitcnt immediates");
  static_assert(SK == 64 ? kStages == 2 : kStages == 5, "pipeline depth");
  if constexpr (DYN == kDynM || DYN == kDynN) {
    // The raster runs over the live tiles: the workgroups past them leave at
    // once, and the live ones are spread over all XCDs (a raster over the
    // launch's upper bound would leave the XCDs that own the dead tiles idle).
    const int64_t d = *dyn;
    if constexpr (DYN == kDynM) {
      M = d < M ? d : M;
      epi.N = M;                                   // the epilogue's token rows
    } else {
      Nn = d < Nn ? d : Nn;
      epi.N = Nn;                                  // the epilogue's token columns
    }
    if (bid >= gemm::num_tiles(M, Nn)) return;
  }
  int64_t m0, n0;
  gemm::tile_coords(bid, M, Nn, group_m, m0, n0, SpreadM<Epi>::value);
  if constexpr (DYN == kDynK) {
    const int64_t d = *dyn;
    K = d < K ? d : K;                             // past the count: zero-filled
    A.g.K = K;
    B.g.K = K;
  }
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  // first in the queue, so every later counted wait of the pipeline covers it
  epi.stage(smem + kSmemBytes, n0, wave, lane);

  Acc acc;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.f;

  k_loop<FA, FB>(acc, A, B, K, m0, n0, smem, tid, lane, wave, wm, wn);
  if constexpr (SEGS == 2)
    k_loop<FA, FB>(acc, Operand{A.ptr + a2_off, A.g}, B, K, m0, n0, smem, tid, lane, wave, wm, wn);
  __syncthreads();
  epi(acc, m0, n0, wm, wn, lane, smem, smem + kSmemBytes);
}

// A GEMM launch over dense operands (the forward and gradient GEMMs): one
// workgroup per tile. The stages are one __shared__ array: with a second LDS
// object the compiler can no longer tell the direct-to-LDS writes of one
// stage from the reads of another and serialises the pipeline.
template <int FA, int FB, class Epi, int DYN>
__global__ __launch_bounds__(kThreads, 1) void k_gemm(Operand A, Operand B, int64_t M,
                                                      int64_t Nn, int64_t K, int group_m,
                                                      Epi epi, const int64_t* dyn) {
  __shared__ __attribute__((aligned(1024))) char smem[stage_bytes<FA, FB>() + Epi::kTokBytes];
  gemm_tile<FA, FB, Epi, false, 1, false, DYN>(smem, blockIdx.x, 0, A, B, M, Nn, K, group_m, epi,
                                               0, dyn);
}

// Two independent GEMMs of one backward chunk in one grid: the n1 workgroups
// of the first (padded to a multiple of 8, so the XCD raster of the second
// stays aligned) and then those of the second. The dH GEMM goes first: with
// the kept tokens only, its tiles may fill its last round of workgroups only
// in part, and the shorter dW tiles behind it fill the rest instead of the
// next launch starting on an idle chip. One LDS array serves both.
// SPLIT1: the first GEMM is split along K into segments of off1 rows, its
// n1 = t1 x segments workgroups segment by segment (workgroup b: segment
// b / t1, tile b % t1), each writing a partial product of its own.
// SEGS = 2 (float32 gradients): both GEMMs run their K loop over the hi part
// of G and then over the lo part, off1 (= off2) elements further.
template <int FA1, int FB1, class Epi1, int DYN1, bool SPLIT1, int FA2, int FB2, class Epi2,
          int DYN2, int SEGS>
__global__ __launch_bounds__(kThreads, 1) void k_gemm_pair(
    int64_t n1p, int64_t t1, int64_t n1, int64_t off1, Operand A1, Operand B1, int64_t M1,
    int64_t N1, int64_t K1, Epi1 e1, Operand A2, Operand B2, int64_t M2, int64_t N2, int64_t K2,
    Epi2 e2, int64_t off2, const int64_t* dyn) {
  static_assert(!(SPLIT1 && SEGS == 2), "a split GEMM has one K segment per workgroup");
  constexpr int kB1 = stage_bytes<FA1, FB1>() + Epi1::kTokBytes;
  constexpr int kB2 = stage_bytes<FA2, FB2>() + Epi2::kTokBytes;
  __shared__ __attribute__((aligned(1024))) char smem[kB1 > kB2 ? kB1 : kB2];
  const int64_t b = blockIdx.x;
  if (b < n1p) {
    if (b >= n1) return;
    if constexpr (SPLIT1) {
      const int64_t seg = b / t1;
      gemm_tile<FA1, FB1, Epi1, true, 1, true, DYN1>(smem, b - seg * t1, int(seg), A1, B1, M1,
                                                     N1, K1, gemm::kGroupM, e1, off1, dyn);
    } else {
      gemm_tile<FA1, FB1, Epi1, true, SEGS, false, DYN1>(smem, b, 0, A1, B1, M1, N1, K1,
                                                         gemm::kGroupM, e1, off1, dyn);
    }
  } else {
    gemm_tile<FA2, FB2, Epi2, true, SEGS, false, DYN2>(smem, b - n1p, 0, A2, B2, M2, N2, K2,
                                                       gemm::kGroupM, e2, off2, dyn);
  }
}

// tanh(x) = 1 - 2 / (exp(2x) + 1), from the hardware exp2 and reciprocal.
// Exact limits +-1 for large |x|; absolute error a few 1e-7, which the
// softcap scale s turns into a logit error of a few s * 1e-7.
__device__ __forceinline__ float tanh_fast(float x) {
  const float e = __builtin_amdgcn_exp2f(x * (2.f * kLog2e));
  return 1.f - 2.f * __builtin_amdgcn_rcpf(e + 1.f);
}

// XOR swizzle of the 8-byte slots of a staged token row (32 slots, 256 bytes,
// one bank window): 2 b(t) with b(t) the 4-bit token t % 16 with its two
// halves swapped. Even, so the 16-byte runs read back stay whole. A staging
// write of 32 lanes (two 16-lane groups g, g + 1, 16 tokens each) covers all
// 64 banks once (g goes to bit 0, b(t) to bits 1..4), and so does a 16-lane
// read of 4 chunks of 4 consecutive tokens (the token's two low bits land
// above the chunk's).
__device__ __forceinline__ int token_swizzle(int tl) {
  return 8 * (tl & 3) + 2 * ((tl >> 2) & 3);
}

// ---- token-major bf16 stores of a tile held in the accumulators ----------
// The tile's rows are vocabulary ids, its columns tokens; the destination is
// row-major by token, dst[t][v] with row length ld, or (BLOCKED) blocked,
// dst[blocked_offset(t, v, blk)]. Each wave stages its
// 128 x 128 block in its own 32 KiB of LDS as [token][vocab] (a lane packs
// its 4 consecutive vocab values of a block into 8 bytes; 8-byte slots
// XOR-swizzled by token), then writes whole 16-byte runs of token rows; columns t >= nt and
// rows v >= nv are not written. LO stores the residual v - bf16(v) instead
// of v (the low half of a bf16 pair). Optionally one element per token
// column j of the lane is replaced after staging: patch->pos[j] >= 0 is its
// byte offset in the wave's staging area (target_slot) and patch->val[j] its
// value. The caller separates a second use of the staging area with a
// barrier.
struct TargetPatch {
  int pos[8];
  float val[8];
};

// Byte offset, in a wave's staging area, of row d (0..127, the wave's own
// rows) of token column tl: the 8-byte slot d / 4 of the token row, swizzled.
__device__ __forceinline__ int target_slot(int d, int tl) {
  return tl * 256 + (((d >> 2) ^ token_swizzle(tl)) * 8) + 2 * (d & 3);
}

// The value of accumulator element (i, j, r) is get(i, j, r): the element
// itself, or a function of it formed as it is staged.
template <bool LO, bool PATCH = false, bool BLOCKED = false, class Get>
__device__ __forceinline__ void store_token_major(const Get& get, char* smem, int wm, int wn,
                                                  int lane, uint16_t* dst, int64_t ld,
                                                  int64_t m0, int64_t n0, int64_t nt,
                                                  int64_t nv, const TargetPatch* patch = nullptr,
                                                  int64_t blk = 0) {
  const int g = lane >> 4;
  char* reg = smem + (wm + 2 * wn) * kWaveScratch;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int tl = j * 16 + (lane & 15);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = get(i, j, e);
        if (LO) v[e] -= bf16_to_f32(f32_to_bf16(v[e]));
      }
      const uint32_t lo = pack_bf16x2(v[0], v[1]);
      const uint32_t hi = pack_bf16x2(v[2], v[3]);
      const int slot = (i * 4 + g) ^ token_swizzle(tl);
      *reinterpret_cast<uint2*>(reg + tl * 256 + slot * 8) = make_uint2(lo, hi);
    }
  }
  if (PATCH) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (patch->pos[j] >= 0) {
        float v = patch->val[j];
        if (LO) v -= bf16_to_f32(f32_to_bf16(v));
        *reinterpret_cast<uint16_t*>(reg + patch->pos[j]) = f32_to_bf16(v);
      }
  }
  __syncthreads();
  if constexpr (BLOCKED) {
    // Blocked destination (dst[blocked_offset(t, v, blk)]): store q covers
    // vocabulary block q / 8 of the wave (32 columns) for 16 tokens, one
    // contiguous KiB.
#pragma unroll 4
    for (int q = 0; q < 32; ++q) {
      const int tl = (q & 7) * 16 + (lane >> 2), ch = (q >> 3) * 4 + (lane & 3);
      const u32x4 v =
          *reinterpret_cast<const u32x4*>(reg + tl * 256 + ((2 * ch) ^ token_swizzle(tl)) * 8);
      const int64_t t = n0 + wn * 128 + tl;
      const int64_t vl = m0 + wm * 128 + 8 * ch;
      if (t < nt && vl < nv)
        *reinterpret_cast<u32x4*>(dst + gemm::blocked_offset(t, vl, blk)) = v;
    }
  } else {
#pragma unroll 4
    for (int q = 0; q < 32; ++q) {
      const int idx = q * 64 + lane;
      const int tl = idx >> 4, ch = idx & 15;
      const u32x4 v =
          *reinterpret_cast<const u32x4*>(reg + tl * 256 + ((2 * ch) ^ token_swizzle(tl)) * 8);
      const int64_t t = n0 + wn * 128 + tl;
      const int64_t vl = m0 + wm * 128 + 8 * ch;
      if (t < nt && vl < nv) *reinterpret_cast<u32x4*>(dst + t * ld + vl) = v;
    }
  }
}

const uint16_t* buf_ptr(const Args& a, int buf) {
  return buf == gemm::kBufW  ? static_cast<const uint16_t*>(a.W)
       : buf == gemm::kBufH  ? static_cast<const uint16_t*>(a.h)
       : buf == gemm::kBufHc ? static_cast<const uint16_t*>(a.hc)
                             : static_cast<const uint16_t*>(a.g);
}

// A T-form operand is read in 16-byte column chunks: it needs rows % 8 == 0.
// The per-lane load offsets are 32-bit byte offsets from the tile base: at
// most min(255, rows - 1) rows of ld elements plus 64 k for a K-contiguous
// operand, 63 k-rows of ld elements plus the row length for a T-form one.
// The tile count must fit the grid.
bool operand_offsets_fit(int form, const gemm::Geom& g) {
  const int64_t reach = form == gemm::kFormN ? (g.rows - 1 < 255 ? g.rows - 1 : 255) * g.ld + 64
                        : g.blk ? 7 * g.blk + 64 * 32
                                : 63 * g.ld + g.rows;
  return reach >= 0 && 2 * reach + 16 <= int64_t(0xFFFFFFFF);
}

bool launch_ok(const gemm::Launch& l) {
  if (l.fa == gemm::kFormT && (l.a.rows % 8 != 0 || l.a.rows < 8)) return false;
  if (l.fb == gemm::kFormT && (l.b.rows % 8 != 0 || l.b.rows < 8)) return false;
  if (!operand_offsets_fit(l.fa, l.a) || !operand_offsets_fit(l.fb, l.b)) return false;
  if (gemm::num_tiles(l.M, l.Nn) > kMaxTiles) return false;
  return l.M > 0 && l.Nn > 0 && l.K > 0;
}

template <int FA, int FB, int DYN = kDynNone, class Epi>
hipError_t run_gemm(const gemm::Launch& l, const Args& a, const Epi& e, int kind,
                    const Launcher& L, const int64_t* dyn = nullptr) {
  if (!launch_ok(l)) return hipErrorInvalidValue;
  if (l.a.blk != 0 || l.b.blk != 0) return hipErrorInvalidValue;
  if ((DYN != kDynNone) != (dyn != nullptr)) return hipErrorInvalidValue;
  Operand A{buf_ptr(a, l.buf_a) + l.off_a, l.a};
  Operand B{buf_ptr(a, l.buf_b) + l.off_b, l.b};
  L.pre(kind);
  hipLaunchKernelGGL((k_gemm<FA, FB, Epi, DYN>), dim3(unsigned(gemm::num_tiles(l.M, l.Nn))),
                     dim3(kThreads), 0, L.stream, A, B, l.M, l.Nn, l.K, gemm::kGroupM, e, dyn);
  L.post(kind);
  return hipGetLastError();
}

}  // namespace
}  // namespace flce
