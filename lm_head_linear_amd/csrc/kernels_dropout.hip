// Dropout with the residual's addition: out = round(residual + keep x scale), and its
// backward, dx = round(keep dout scale): the same pass without a residual. A dropped
// value is zero whatever it held.
//
// Bound by memory (2 or 3 rows of N x H). A thread takes a block of eight columns, the
// generator's unit (16 bytes of bf16, 32 of float32), or four of them 256 blocks apart
// where the grid is large, all loaded before the first is used.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "dropout.h"
#include "flce_internal.h"
#include "ops_plan.h"
#include "row_io.h"

namespace flce {
namespace {

constexpr int kDropThreads = 256;

// Blocks first .. first + 256 PER - 1 of the rows' blocks of eight columns, counted along
// the rows (bpr a row).
template <class T, bool RES, int PER>
__global__ __launch_bounds__(kDropThreads) void k_dropout(const T* x, int64_t ldx, const T* res,
                                                          int64_t ldr, int64_t H, uint32_t bpr,
                                                          float inv_bpr, int64_t total,
                                                          DropSpec spec, T* out, int64_t ldo) {
  constexpr int E = kPerChunk<T>, C = 8 / E;
  const DropKey key = drop_key(spec);
  const int64_t first = int64_t(blockIdx.x) * (kDropThreads * PER);
  const int64_t row0 = first / bpr;
  const uint32_t col0 = uint32_t(first - row0 * bpr);
  int64_t row[PER], c[PER];
  float v[PER][C][E], r[PER][C][E];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    // block `at` of row0 onwards; at < 2^24, so its float is exact and the quotient off by
    // one at most
    const uint32_t at = col0 + uint32_t(i) * kDropThreads + threadIdx.x;
    uint32_t q = uint32_t(float(at) * inv_bpr);
    if (q * bpr > at) --q;
    else if (at - q * bpr >= bpr) ++q;
    const bool live = first + i * kDropThreads + threadIdx.x < total;
    row[i] = live ? row0 + q : -1;
    c[i] = int64_t(at - q * bpr) * 8;
    if (!live) continue;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      load_chunk(x + row[i] * ldx, c[i] + k * E, H, v[i][k]);
      if (RES) load_chunk(res + row[i] * ldr, c[i] + k * E, H, r[i][k]);
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (row[i] < 0) continue;
    const Mask8 m = drop_bits(key, uint32_t(row[i]), uint32_t(c[i] >> 3));
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool keep = drop_keeps(m, k * E + e, spec.threshold);
        if (RES) v[i][k][e] = keep ? fmaf(v[i][k][e], spec.scale, r[i][k][e]) : r[i][k][e];
        else v[i][k][e] = keep ? v[i][k][e] * spec.scale : 0.f;
      }
      store_chunk(out + row[i] * ldo, c[i] + k * E, H, v[i][k]);
    }
  }
}

template <class T>
hipError_t dropout(const DropoutArgs& a, const Launcher& L) {
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* out = static_cast<T*>(a.out);
  const int64_t bpr = (a.H + 7) / 8, total = a.N * bpr;
  auto go = [&](auto has_res, auto per) {
    constexpr bool RES = decltype(has_res)::value;
    constexpr int PER = decltype(per)::value, kPerGroup = kDropThreads * PER;
    hipLaunchKernelGGL((k_dropout<T, RES, PER>), dim3(unsigned((total + kPerGroup - 1) / kPerGroup)),
                       dim3(kDropThreads), 0, L.stream, x, a.ld_x, res, a.ld_res, a.H,
                       uint32_t(bpr), 1.f / float(bpr), total, a.drop, out, a.ld_out);
  };
  using Y = std::true_type;
  using No = std::false_type;
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, kDropBlocks>;
  const bool many = total >= kDropMany;
  L.pre(kDropout);
  if (res) many ? go(Y{}, Four{}) : go(Y{}, One{});
  else many ? go(No{}, Four{}) : go(No{}, One{});
  L.post(kDropout);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, const Launcher& L) {
  return a.dtype == FLCE_F32 ? dropout<float>(a, L) : dropout<Bf16Bits>(a, L);
}

}  // namespace flce
