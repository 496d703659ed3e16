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
// With dropout (DROP) the same passes take x's mask (dropout.h) in stride: s is then
// round(r + keep x scale), and the backward writes two rows, the sum's gradient for the
// residual and the masked one for x.
//
// Rows of whole chunks are loaded without conditions, all before the first value is used, in
// the forward, with dropout, and elsewhere where it pays (kLoadsAhead): a branch around a
// load has it waited for before the next.
//
// bf16 with the residual, 8192 rows of 4096: forward 40 us, backward 57 with dw's 7 (268 MB
// each); with dropout 42 and 79 (335 MB; loads with conditions 44 and 107). Both directions
// together, by threads a row: 8192 x 4096, 256 threads 97 us; 16384 x 1024, 128 threads 48;
// 32768 x 512, 64 threads 47; 65536 x 128, 16 threads 28. With conditional loads those took
// 103, 50, 48 and 30, and other counts: 64 threads 211 and 1024 151; 64 threads 54; 32 threads
// 53; 32 threads 40, and one row a 64-thread workgroup 126.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "dropout.h"
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
// DROP: x is dropped out before the residual (null: none) is added, s is always written;
// row 0 is row `row0` of the mask.
template <class T, class WT, int LANES, int C, bool RES, bool DROP>
__global__ __launch_bounds__(kBlock<LANES>) void k_rms_norm(
    const T* x, int64_t ldx, const T* res, int64_t ldr, const WT* __restrict__ w, int64_t N,
    int64_t H, float eps, float offset, T* y, int64_t ldy, T* s, int64_t lds,
    float* __restrict__ rstd, DropSpec drop, int64_t row0) {
  constexpr bool SUM = RES || DROP;                // s is another value than x
  constexpr int E = kPerChunk<T>, R = kBlock<LANES> / LANES;
  __shared__ float red[kBlock<LANES> / 64];
  const int tid = threadIdx.x % LANES;
  const int64_t at = int64_t(blockIdx.x) * R + threadIdx.x / LANES;
  const int64_t row = at < N ? at : N - 1;         // behind the last: it again, not stored
  const int64_t Hs = at < N ? H : 0;               // columns that are stored
  x += row * ldx;
  y += row * ldy;
  if (RES) res += row * ldr;
  if (SUM) s += row * lds;
  DropKey key{};
  if constexpr (DROP) key = drop_key(drop);
  float sum = 0.f;
  // s of a chunk: v is x's and becomes s
  auto add = [&](int64_t c, float (&v)[E], const float (&r)[E]) {
    if constexpr (DROP) {
      const Mask8 m = drop_chunk<E>(key, row0 + row, c);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float with = RES ? r[e] : 0.f;
        v[e] = drop_keeps(m, e, drop.threshold) ? fmaf(v[e], drop.scale, with) : with;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = to_f32(from_f32<T>(v[e]));
    } else if (RES) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = to_f32(from_f32<T>(v[e] + r[e]));
    }
  };
  auto load_sum = [&](int64_t c, float (&v)[E]) {
    float r[E];
    load_chunk(x, c, H, v);
    if (RES) load_chunk(res, c, H, r);
    add(c, v, r);
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
    if (H % E == 0) {                              // every load before the first is used
      row_u32x4 rx[C], rr[C];
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int64_t c = (int64_t(k) * LANES + tid) * E;
        rx[k] = load_whole(x, c, H);
        if (RES) rr[k] = load_whole(res, c, H);
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int64_t c = (int64_t(k) * LANES + tid) * E;
        float r[E];
        unpack_whole<T>(rx[k], c, H, v[k]);
        if (RES) unpack_whole<T>(rr[k], c, H, r);
        add(c, v[k], r);
        load_w(c, f[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const int64_t c = (int64_t(k) * LANES + tid) * E;
        load_sum(c, v[k]);
        load_w(c, f[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(v[k][e], v[k][e], sum);
      if (SUM) store_chunk(s, (int64_t(k) * LANES + tid) * E, Hs, v[k]);
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
      if (SUM) store_chunk(s, c, H, v);
    }
    const float q = finish(row_sum<LANES>(sum, red));
    // a thread reads back only what it wrote itself (s), or x, whose element it
    // replaces last when y is x
    for (int64_t c = int64_t(tid) * E; c < H; c += LANES * E) {
      float v[E], f[E];
      load_chunk(SUM ? const_cast<const T*>(s) : x, c, H, v);
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
// own columns). DROP: d, the gradient of the sum, goes to dres (null: not wanted), and dx
// gets keep d scale. WHOLE: rows of whole chunks, loaded without conditions (with DROP that
// is found at run time).
template <class T, class WT, int LANES, int C, bool DS, bool DW, bool DROP, bool WHOLE>
__global__ __launch_bounds__(kBlock<LANES>) void k_rms_norm_bwd(
    const T* dy, int64_t lddy, const T* ds, int64_t ldds, const T* __restrict__ s, int64_t lds,
    const WT* __restrict__ w, const float* __restrict__ rstd, int64_t N, int64_t H, float offset,
    T* dx, int64_t lddx, float* __restrict__ dw_part, T* dres, int64_t lddres, DropSpec drop) {
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
  const bool whole = DROP ? H % E == 0 : WHOLE;
  DropKey key{};
  if constexpr (DROP) key = drop_key(drop);
  // a bit for each value of a chunk that stays
  auto keep_bits = [&](int64_t row, int64_t c) {
    uint32_t bits = 0;
    if constexpr (DROP) {
      const Mask8 m = drop_chunk<E>(key, row, c);
#pragma unroll
      for (int e = 0; e < E; ++e) bits |= drop_keeps(m, e, drop.threshold) ? 1u << e : 0u;
    }
    return bits;
  };
  // the gradients of columns c .. of a row, d that of the sum
  auto store_grads = [&](int64_t row, int64_t c, int64_t Hs, float (&d)[E], uint32_t bits) {
    if constexpr (DROP) {
      if (dres) store_chunk(dres + row * lddres, c, Hs, d);
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = (bits >> e) & 1 ? d[e] * drop.scale : 0.f;
    }
    store_chunk(dx + row * lddx, c, Hs, d);
  };
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
      uint32_t bits[C];
      auto masks = [&] {
#pragma unroll
        for (int k = 0; k < C; ++k) bits[k] = keep_bits(row, (int64_t(k) * LANES + tid) * E);
      };
      if (whole) {
        row_u32x4 rg[C], rn[C], rd[C];
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const int64_t c = (int64_t(k) * LANES + tid) * E;
          rg[k] = load_whole(dy + row * lddy, c, H);
          rn[k] = load_whole(s + row * lds, c, H);
          if (DS) rd[k] = load_whole(ds + row * ldds, c, H);
        }
        masks();                                   // while the loads are under way
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const int64_t c = (int64_t(k) * LANES + tid) * E;
          unpack_whole<T>(rg[k], c, H, g[k]);
          unpack_whole<T>(rn[k], c, H, n[k]);
          if (DS) unpack_whole<T>(rd[k], c, H, d[k]);
        }
      } else {
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const int64_t c = (int64_t(k) * LANES + tid) * E;
          load_chunk(dy + row * lddy, c, H, g[k]);
          load_chunk(s + row * lds, c, H, n[k]);
          if (DS) load_chunk(ds + row * ldds, c, H, d[k]);
        }
        masks();
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
        const int64_t c = (int64_t(k) * LANES + tid) * E;
        if constexpr (DROP) store_grads(row, c, live ? H : 0, g[k], bits[k]);
        else store_chunk(dx + row * lddx, c, live ? H : 0, g[k]);
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
        store_grads(row, c, H, g, keep_bits(row, c));
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

// Whether the backward without dropout of rows of whole chunks loads all of them before the
// first is used. Where registers are short, or a row's loads are few, that costs more than
// the wait it saves. us with conditional loads and without, bf16: 2048 x 8192 (four chunks
// for each of 256 threads) 60 and 55 with ds and dw, 28 and 24 with ds, 22 and 18 with
// neither; 8192 x 4096 (two) 61 and 57 with both, 39 and 41, 30 and 31; 4096 x 16384 (four
// for each of 1024 threads) 691 and 522 with both, 382 and 480 with dw, 222 and 230 with ds,
// 99 and 106. float32: 8192 x 4096 107 and 114 with both, 32768 x 512 29 and 31 with neither,
// the same elsewhere.
template <class T, int LANES, int C, bool DS, bool DW, bool DROP>
constexpr bool kLoadsAhead =
    !DROP && C > 0 && sizeof(T) == 2 && (LANES == 1024 ? DS && DW : C != 2 || DW);

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
      auto go = [&](auto has_res, auto has_drop) {
        constexpr bool RES = decltype(has_res)::value, DROP = decltype(has_drop)::value;
        hipLaunchKernelGGL((k_rms_norm<T, WT, LN, C, RES, DROP>), grid, block, 0, L.stream, xt,
                           a.ld_x, RES ? r + t0 * a.ld_res : r, a.ld_res, w, n, a.H, a.eps, a.offset,
                           yt, a.ld_y, RES || DROP ? s + t0 * a.ld_s : s, a.ld_s, q,
                           DROP ? *a.drop : DropSpec{}, t0);
      };
      using Y = std::true_type;
      using No = std::false_type;
      if (a.drop) r ? go(Y{}, Y{}) : go(No{}, Y{});
      else r ? go(Y{}, No{}) : go(No{}, No{});
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
    auto go = [&](auto has_ds, auto has_dw, auto has_drop) {
      constexpr bool DS = decltype(has_ds)::value, DW = decltype(has_dw)::value;
      constexpr bool DROP = decltype(has_drop)::value;
      auto launch = [&](auto whole) {
        hipLaunchKernelGGL((k_rms_norm_bwd<T, WT, LN, C, DS, DW, DROP, decltype(whole)::value>),
                           dim3(unsigned(nb)), dim3(kBlock<LN>), 0, L.stream, dy, a.ld_dy, ds, a.ld_ds, s,
                           a.ld_s, w, a.rstd, a.N, a.H, a.offset, dx, a.ld_dx, a.dw_part,
                           static_cast<T*>(a.dres), a.ld_dres, DROP ? *a.drop : DropSpec{});
      };
      if constexpr (kLoadsAhead<T, LN, C, DS, DW, DROP>) {
        if (a.H % kPerChunk<T> == 0) return launch(std::true_type{});
      }
      launch(std::false_type{});
    };
    using Y = std::true_type;
    using No = std::false_type;
    auto pick = [&](auto has_drop) {
      if (ds) a.dweight ? go(Y{}, Y{}, has_drop) : go(Y{}, No{}, has_drop);
      else a.dweight ? go(No{}, Y{}, has_drop) : go(No{}, No{}, has_drop);
    };
    a.drop ? pick(Y{}) : pick(No{});
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
