// Dropout with the residual's addition: out = round(residual + keep x scale), and its
// backward, dx = round(keep dout scale): the same pass without a residual. A dropped
// value is zero whatever it held.
//
// Bound by memory (2 or 3 rows of N x H). A thread takes a block of eight columns, the
// generator's unit (16 bytes of bf16, 32 of float32), or four of them 256 blocks apart
// where the grid is large (kDropMany). Rows of whole blocks (WHOLE) are loaded without
// conditions, all before the first is used. 8192 x 4096 bf16: 40 us with the residual (201 MB,
// 5.0 TB/s), 26 without (134 MB); with conditional loads 45 and 32.
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
template <class T, bool RES, int PER, bool WHOLE>
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
  bool live[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    // block `at` of row0 onwards; at < 2^24, so its float is exact and the quotient off by
    // one at most
    const uint32_t at = col0 + uint32_t(i) * kDropThreads + threadIdx.x;
    uint32_t q = uint32_t(float(at) * inv_bpr);
    if (q * bpr > at) --q;
    else if (at - q * bpr >= bpr) ++q;
    live[i] = first + i * kDropThreads + threadIdx.x < total;
    row[i] = live[i] ? row0 + q : 0;               // behind the last: the first, not stored
    c[i] = live[i] ? int64_t(at - q * bpr) * 8 : 0;
  }
  float v[PER][C][E], r[PER][C][E];
  if constexpr (WHOLE) {
    row_u32x4 xr[PER][C], rr[PER][C];
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xr[i][k] = load_raw(x + row[i] * ldx + c[i] + k * E);
        if (RES) rr[i][k] = load_raw(res + row[i] * ldr + c[i] + k * E);
      }
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        unpack_chunk<T>(xr[i][k], v[i][k]);
        if (RES) unpack_chunk<T>(rr[i][k], r[i][k]);
      }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        load_chunk(x + row[i] * ldx, c[i] + k * E, H, v[i][k]);
        if (RES) load_chunk(res + row[i] * ldr, c[i] + k * E, H, r[i][k]);
      }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const Mask8 m = drop_bits(key, uint32_t(row[i]), uint32_t(c[i] >> 3));
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const bool keep = drop_keeps(m, k * E + e, spec.threshold);
        if (RES) v[i][k][e] = keep ? fmaf(v[i][k][e], spec.scale, r[i][k][e]) : r[i][k][e];
        else v[i][k][e] = keep ? v[i][k][e] * spec.scale : 0.f;
      }
      T* o = out + row[i] * ldo;
      if (WHOLE) {
        if (live[i]) *reinterpret_cast<row_u32x4_any*>(o + c[i] + k * E) = pack_chunk<T>(v[i][k]);
      } else {
        store_chunk(o, c[i] + k * E, live[i] ? H : 0, v[i][k]);
      }
    }
  }
}

template <class T>
hipError_t dropout(const DropoutArgs& a, const Launcher& L) {
  const T* x = static_cast<const T*>(a.x);
  const T* res = static_cast<const T*>(a.residual);
  T* out = static_cast<T*>(a.out);
  const int64_t bpr = (a.H + 7) / 8, total = a.N * bpr;
  auto go = [&](auto has_res, auto per, auto whole) {
    constexpr bool RES = decltype(has_res)::value, WHOLE = decltype(whole)::value;
    constexpr int PER = decltype(per)::value, kPerGroup = kDropThreads * PER;
    hipLaunchKernelGGL((k_dropout<T, RES, PER, WHOLE>), dim3(unsigned((total + kPerGroup - 1) / kPerGroup)),
                       dim3(kDropThreads), 0, L.stream, x, a.ld_x, res, a.ld_res, a.H,
                       uint32_t(bpr), 1.f / float(bpr), total, a.drop, out, a.ld_out);
  };
  using Y = std::true_type;
  using No = std::false_type;
  using One = std::integral_constant<int, 1>;
  using Four = std::integral_constant<int, kDropBlocks>;
  const bool many = total >= kDropMany;
  L.pre(kDropout);
  auto pick = [&](auto whole) {
    if (res) many ? go(Y{}, Four{}, whole) : go(Y{}, One{}, whole);
    else many ? go(No{}, Four{}, whole) : go(No{}, One{}, whole);
  };
  a.H % 8 == 0 ? pick(Y{}) : pick(No{});
  L.post(kDropout);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& a, const Launcher& L) {
  return a.dtype == FLCE_F32 ? dropout<float>(a, L) : dropout<Bf16Bits>(a, L);
}

}  // namespace flce
