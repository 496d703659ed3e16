// Root-mean-square norm of the rows in front of the head, with the residual's
// addition:
//   s    = round(x + r)                 (x itself without a residual)
//   rstd = 1 / sqrt(mean(s^2) + eps)
//   y    = round(s rstd (w + offset))
// and its backward, with n = s rstd and g = dy (w + offset):
//   dx = round(ds + rstd (g - n mean(g n)))     (x and r get the same gradient)
//   dw = round(sum over rows of dy n)           (+ the dw in memory)
// Sums, rstd and everything between a load and a store are float32; the norm is
// taken of the stored (rounded) s, so the backward, which reads s, sees the
// values the forward used.
//
// Both are bound by memory: the forward reads 2 and writes 2 rows, the backward
// reads 3 and writes 1. A row is read once: it stays in registers from the load to the
// store. 16 to 1024 threads take a row, by its length, so that each holds one to four
// 16-byte chunks and has its loads under way at once; short rows share a workgroup of
// 256. Rows of more than 4096 chunks are read twice. The backward's workgroups, four
// per CU, walk rows with a fixed stride and keep their share of dw in registers; a
// second kernel adds the shares up in a fixed order.
//
// bf16 with the residual, 8192 rows of 4096: forward 50 us (268 MB, 5.4 TB/s), backward
// 56 us (4.8 TB/s) and 7 us for dw. Both directions together, with this many threads
// and with others: 8192 x 4096, 256 threads 112 us (64: 211, 1024: 151); 16384 x 1024,
// 128 threads 49 (64: 54); 32768 x 512, 64 threads 48 (32: 53); 65536 x 128, 16 threads
// 29 (32: 40, one row a 64-thread workgroup: 126).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "flce_internal.h"
#include "ops_plan.h"
#include "row_io.h"
#include "wave_ops.h"

namespace flce {
namespace {

// Threads of a workgroup whose rows take LANES threads each.
template <int LANES>
constexpr int kBlock = LANES < 256 ? 256 : LANES;

// Sum over the LANES threads of a row, the same bits in each. `red` holds a float a
// wave; a barrier separates two uses.
template <int LANES>
__device__ __forceinline__ float row_sum(float x, float* red) {
  if constexpr (LANES == 16) return group_all<16>(x, AddOp());
  if constexpr (LANES == 32) return pair_rows(group_all<16>(x, AddOp()), AddOp());
  x = wave_all(x, AddOp());
  if constexpr (LANES > 64) {
    static_assert(LANES >= 256 || kBlock<LANES> % LANES == 0, "whole rows");
    const int w = threadIdx.x >> 6, first = w / (LANES / 64) * (LANES / 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[w] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < LANES / 64; ++i) x += red[first + i];
  }
  return x;
}

// LANES threads a row. C > 0: the row stays in registers, C chunks a thread; C = 0:
// rows of any length, read again for the second pass.
template <class T, class WT, int LANES, int C, bool RES>
__global__ __launch_bounds__(kBlock<LANES>) void k_rms_norm(
    const T* x, int64_t ldx, const T* res, int64_t ldr, const WT* __restrict__ w, int64_t N,
    int64_t H, float eps, float offset, T* y, int64_t ldy, T* s, int64_t lds,
    float* __restrict__ rstd) {
  constexpr int E = kPerChunk<T>, R = kBlock<LANES> / LANES;
  __shared__ float red[kBlock<LANES> / 64];
  const int tid = threadIdx.x % LANES;
  const int64_t at = int64_t(blockIdx.x) * R + threadIdx.x / LANES;
  const int64_t row = at < N ? at : N - 1;         // behind the last: it again, not stored
  const int64_t Hs = at < N ? H : 0;               // columns that are stored
  x += row * ldx;
  y += row * ldy;
  if (RES) { res += row * ldr; s += row * lds; }
  float sum = 0.f;
  auto load_sum = [&](int64_t c, float (&v)[E]) {
    load_chunk(x, c, H, v);
    if (RES) {
      float r[E];
      load_chunk(res, c, H, r);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = to_f32(from_f32<T>(v[e] + r[e]));
    }
  };
  auto load_w = [&](int64_t c, float (&f)[E]) {
    if constexpr (sizeof(WT) == sizeof(T)) {
      load_chunk(w, c, H, f);
    } else {
      float a[4], b[4];
      load_chunk(w, c, H, a);
      load_chunk(w, c + 4, H, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) { f[e] = a[e]; f[4 + e] = b[e]; }
    }
  };
  auto finish = [&](float total) {
    const float q = 1.f / sqrtf(total / float(H) + eps);
    if (rstd && tid == 0 && at < N) rstd[row] = q;
    return q;
  };
  if constexpr (C > 0) {
    float v[C][E], f[C][E];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int64_t c = (int64_t(k) * LANES + tid) * E;
      load_sum(c, v[k]);
      load_w(c, f[k]);
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(v[k][e], v[k][e], sum);
      if (RES) store_chunk(s, (int64_t(k) * LANES + tid) * E, Hs, v[k]);
    }
    const float q = finish(row_sum<LANES>(sum, red));
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[k][e] = (v[k][e] * q) * (f[k][e] + offset);
      store_chunk(y, (int64_t(k) * LANES + tid) * E, Hs, v[k]);
    }
  } else {
    for (int64_t c = int64_t(tid) * E; c < H; c += LANES * E) {
      float v[E];
      load_sum(c, v);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(v[e], v[e], sum);
      if (RES) store_chunk(s, c, H, v);
    }
    const float q = finish(row_sum<LANES>(sum, red));
    // a thread reads back only what it wrote itself (s), or x, whose element it
    // replaces last when y is x
    for (int64_t c = int64_t(tid) * E; c < H; c += LANES * E) {
      float v[E], f[E];
      load_chunk(RES ? const_cast<const T*>(s) : x, c, H, v);
      load_w(c, f);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = (v[e] * q) * (f[e] + offset);
      store_chunk(y, c, H, v);
    }
  }
}

// dx of every gridDim.x R-th row (R rows a workgroup, LANES threads each), and the
// workgroup's share of dw (DW) in dw_part[blockIdx.x][H], its R rows' shares joined in
// LDS. C = 0: rows of any length; dw's share is then added up in memory (each thread its
// own columns).
template <class T, class WT, int LANES, int C, bool DS, bool DW>
__global__ __launch_bounds__(kBlock<LANES>) void k_rms_norm_bwd(
    const T* dy, int64_t lddy, const T* ds, int64_t ldds, const T* __restrict__ s, int64_t lds,
    const WT* __restrict__ w, const float* __restrict__ rstd, int64_t N, int64_t H, float offset,
    T* dx, int64_t lddx, float* __restrict__ dw_part) {
  constexpr int E = kPerChunk<T>, R = kBlock<LANES> / LANES;
  __shared__ float red[kBlock<LANES> / 64];
  const int tid = threadIdx.x % LANES, group = threadIdx.x / LANES;
  auto load_w = [&](int64_t c, float (&f)[E]) {
    if constexpr (sizeof(WT) == sizeof(T)) {
      load_chunk(w, c, H, f);
    } else {
      float a[4], b[4];
      load_chunk(w, c, H, a);
      load_chunk(w, c + 4, H, b);
#pragma unroll
      for (int e = 0; e < 4; ++e) { f[e] = a[e]; f[4 + e] = b[e]; }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] += offset;
  };
  const float inv_h = 1.f / float(H);
  if constexpr (C > 0) {
    float f[C][E], acc[C][E];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      load_w((int64_t(k) * LANES + tid) * E, f[k]);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[k][e] = 0.f;
    }
    for (int64_t r0 = int64_t(blockIdx.x) * R; r0 < N; r0 += int64_t(gridDim.x) * R) {
      // behind the last row: it again, with a rstd of 0 and nothing stored
      const bool live = R == 1 || r0 + group < N;
      const int64_t row = live ? r0 + group : N - 1;
      const float q = live ? rstd[row] : 0.f;
      float g[C][E], n[C][E], d[C][E];
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int64_t c = (int64_t(k) * LANES + tid) * E;
        load_chunk(dy + row * lddy, c, H, g[k]);
        load_chunk(s + row * lds, c, H, n[k]);
        if (DS) load_chunk(ds + row * ldds, c, H, d[k]);
      }
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          n[k][e] *= q;
          if (DW && live) acc[k][e] = fmaf(g[k][e], n[k][e], acc[k][e]);
          g[k][e] *= f[k][e];
          sum = fmaf(g[k][e], n[k][e], sum);
        }
      const float mean = row_sum<LANES>(sum, red) * inv_h;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float v = q * (g[k][e] - n[k][e] * mean);
          g[k][e] = DS ? d[k][e] + v : v;
        }
        store_chunk(dx + row * lddx, (int64_t(k) * LANES + tid) * E, live ? H : 0, g[k]);
      }
    }
    if (DW) {
      float* out = dw_part + int64_t(blockIdx.x) * H;
      if constexpr (R == 1) {
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const int64_t c = (int64_t(k) * LANES + tid) * E;
#pragma unroll
          for (int e = 0; e < E; ++e)
            if (c + e < H) out[c + e] = acc[k][e];
        }
      } else {
        __shared__ float share[R][LANES * C * E];
#pragma unroll
        for (int k = 0; k < C; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) share[group][(k * LANES + tid) * E + e] = acc[k][e];
        __syncthreads();
        for (int64_t c = threadIdx.x; c < H; c += kBlock<LANES>) {
          float v = share[0][c];
#pragma unroll
          for (int i = 1; i < R; ++i) v += share[i][c];
          out[c] = v;
        }
      }
    }
  } else {
    float* out = dw_part + int64_t(blockIdx.x) * H;
    bool first = true;
    for (int64_t row = blockIdx.x; row < N; row += gridDim.x) {
      const float q = rstd[row];
      float sum = 0.f;
      for (int64_t c = int64_t(tid) * E; c < H; c += LANES * E) {
        float g[E], n[E], f[E];
        load_chunk(dy + row * lddy, c, H, g);
        load_chunk(s + row * lds, c, H, n);
        load_w(c, f);
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(g[e] * f[e], n[e] * q, sum);
      }
      const float mean = row_sum<LANES>(sum, red) * inv_h;
      for (int64_t c = int64_t(tid) * E; c < H; c += LANES * E) {
        float g[E], n[E], f[E], d[E];
        load_chunk(dy + row * lddy, c, H, g);
        load_chunk(s + row * lds, c, H, n);
        if (DS) load_chunk(ds + row * ldds, c, H, d);
        load_w(c, f);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          n[e] *= q;
          if (DW && c + e < H) out[c + e] = first ? g[e] * n[e] : fmaf(g[e], n[e], out[c + e]);
          const float v = q * (g[e] * f[e] - n[e] * mean);
          g[e] = DS ? d[e] + v : v;
        }
        store_chunk(dx + row * lddx, c, H, g);
      }
      first = false;
    }
  }
}

// dw[c] = the shares of the nb workgroups added up: 16 columns per workgroup,
// 64 groups of 16 threads that each add every 64th share in order, then the
// groups' sums in order.
template <class WT>
__global__ __launch_bounds__(1024) void k_rms_norm_dw(const float* __restrict__ part, int64_t nb,
                                                      int64_t H, WT* __restrict__ dw,
                                                      int accumulate) {
  __shared__ float red[64][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 16 + col;
  float a = 0.f;
  if (c < H) {
#pragma unroll 8
    for (int64_t b = grp; b < nb; b += 64) a += part[b * H + c];
  }
  red[grp][col] = a;
  __syncthreads();
  for (int k = 32; k > 0; k >>= 1) {
    if (grp < k) red[grp][col] += red[grp + k][col];
    __syncthreads();
  }
  if (grp == 0 && c < H) {
    const float v = red[0][col];
    dw[c] = from_f32<WT>(accumulate ? to_f32(dw[c]) + v : v);
  }
}

// Calls run(lanes, chunks) with the integral constants of the variant for rows
// of n chunks.
template <int I>
using Int = std::integral_constant<int, I>;
template <class F>
auto with_variant(int64_t n, F&& run) {
  if (n <= 16) return run(Int<16>{}, Int<1>{});
  if (n <= 32) return run(Int<32>{}, Int<1>{});
  if (n <= 64) return run(Int<64>{}, Int<1>{});
  if (n <= 128) return run(Int<128>{}, Int<1>{});
  if (n <= 256) return run(Int<256>{}, Int<1>{});
  if (n <= 512) return run(Int<256>{}, Int<2>{});
  if (n <= 1024) return run(Int<256>{}, Int<4>{});
  if (n <= 4096) return run(Int<1024>{}, Int<4>{});
  return run(Int<1024>{}, Int<0>{});
}

template <class T, class WT>
hipError_t norm_forward(const NormArgs& a, const Launcher& L) {
  const int64_t chunks = (a.H + kPerChunk<T> - 1) / kPerChunk<T>;
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.residual);
  const WT* w = static_cast<const WT*>(a.weight);
  T* y = static_cast<T*>(a.y);
  T* s = static_cast<T*>(a.s);
  // a row a workgroup, and a grid holds less than 2^32 threads
  constexpr int64_t kRows = int64_t(1) << 21;
  L.pre(kNorm);
  for (int64_t t0 = 0; t0 < a.N; t0 += kRows) {
    const int64_t n = a.N - t0 < kRows ? a.N - t0 : kRows;
    const T* xt = x + t0 * a.ld_x;
    T* yt = y + t0 * a.ld_y;
    float* q = a.rstd ? a.rstd + t0 : nullptr;
    with_variant(chunks, [&](auto lanes, auto c) {
      constexpr int LN = decltype(lanes)::value, C = decltype(c)::value, R = kBlock<LN> / LN;
      const dim3 grid(unsigned((n + R - 1) / R)), block(kBlock<LN>);
      if (r)
        hipLaunchKernelGGL((k_rms_norm<T, WT, LN, C, true>), grid, block, 0, L.stream, xt, a.ld_x,
                           r + t0 * a.ld_res, a.ld_res, w, n, a.H, a.eps, a.offset, yt, a.ld_y,
                           s + t0 * a.ld_s, a.ld_s, q);
      else
        hipLaunchKernelGGL((k_rms_norm<T, WT, LN, C, false>), grid, block, 0, L.stream, xt, a.ld_x,
                           r, a.ld_res, w, n, a.H, a.eps, a.offset, yt, a.ld_y, s, a.ld_s, q);
    });
  }
  L.post(kNorm);
  return hipGetLastError();
}

template <class T, class WT>
hipError_t norm_backward(const NormBwdArgs& a, const Launcher& L) {
  const int64_t chunks = (a.H + kPerChunk<T> - 1) / kPerChunk<T>;
  const T* dy = static_cast<const T*>(a.dy);
  const T* ds = static_cast<const T*>(a.ds);
  const T* s = static_cast<const T*>(a.s);
  const WT* w = static_cast<const WT*>(a.weight);
  T* dx = static_cast<T*>(a.dx);
  int64_t nb = 0;                                  // workgroups, each with a share of dw
  L.pre(kNormBwd);
  with_variant(chunks, [&](auto lanes, auto c) {
    constexpr int LN = decltype(lanes)::value, C = decltype(c)::value, R = kBlock<LN> / LN;
    nb = norm_shares((a.N + R - 1) / R);
    auto go = [&](auto has_ds, auto has_dw) {
      constexpr bool DS = decltype(has_ds)::value, DW = decltype(has_dw)::value;
      hipLaunchKernelGGL((k_rms_norm_bwd<T, WT, LN, C, DS, DW>), dim3(unsigned(nb)),
                         dim3(kBlock<LN>), 0, L.stream, dy, a.ld_dy, ds, a.ld_ds, s, a.ld_s, w, a.rstd, a.N, a.H,
                         a.offset, dx, a.ld_dx, a.dw_part);
    };
    using Y = std::true_type;
    using No = std::false_type;
    if (ds) a.dweight ? go(Y{}, Y{}) : go(Y{}, No{});
    else a.dweight ? go(No{}, Y{}) : go(No{}, No{});
  });
  L.post(kNormBwd);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.dweight) return e;
  L.pre(kNormBwd);
  hipLaunchKernelGGL(k_rms_norm_dw<WT>, dim3(unsigned((a.H + 15) / 16)), dim3(1024), 0, L.stream,
                     a.dw_part, nb, a.H, static_cast<WT*>(a.dweight), a.accumulate);
  L.post(kNormBwd);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, const Launcher& L) {
  if (a.dtype == FLCE_F32) return norm_forward<float, float>(a, L);
  if (a.weight_dtype == FLCE_F32) return norm_forward<Bf16Bits, float>(a, L);
  return norm_forward<Bf16Bits, Bf16Bits>(a, L);
}

hipError_t launch_rms_norm_backward(const NormBwdArgs& a, const Launcher& L) {
  if (a.dtype == FLCE_F32) return norm_backward<float, float>(a, L);
  if (a.weight_dtype == FLCE_F32) return norm_backward<Bf16Bits, float>(a, L);
  return norm_backward<Bf16Bits, Bf16Bits>(a, L);
}

}  // namespace flce
