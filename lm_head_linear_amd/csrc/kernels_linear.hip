// The linear transform y = act(x W^T + b) + r, with W [O][I], and its backward:
//   dz = dy act'(z);  dx = dz W;  dW = dz^T x;  db = sum over rows of dz   (dr is dy)
// The forward stores the slope act'(z) where a backward will want it: dz then needs no z
// and no exponential. With bf16 rows it is an IEEE half: slopes are at most 1.13, so its
// range does, and half a step of it, at most 2^-11 of the value, leaves dz's own rounding
// (2^-8) the only one that counts; a bf16 slope made the gradients' error 0.0029 of their
// size instead of 0.0024, where rounding the exact ones once leaves 0.0017.
//
// Everything is float32 between a load and a store; what is rounded besides the outputs
// is the slope and dz (bf16 rows: the products' operand, at half the time of a pair of bf16
// for dz). db sums dz before its rounding.
//
// Products of bf16 rows whose lengths and addresses are multiples of 16 bytes, with enough
// tiles of 256 x 256 to fill the chip, run on the head's product (gemm_bf16.h); others
// on the one of smaller tiles (gemm_small.h; 2048 x 1024 x 1024: forward 20 us on 128 x 128
// tiles, 11 to 13 on 64 x 64). 8192 x 4096 x 4096 with silu, bias and residual, in one run:
// a step 720 us, loops of the forward alone 241 to 267, of the backward 463 to 471 (dz and db
// 41 of it); all on 128 x 128 tiles, before those had direct loads, 1058. Few rows forward,
// where reading W is all there is to it, take k_linear_few (up to 64), or, for a wide W (a
// head), k_linear_wide (up to 128).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "../../include/flce.h"
#include "activation.h"
#include "few_rows.h"
#include "flce_internal.h"
#include "gemm_bf16.h"
#include "gemm_small.h"
#include "ops_plan.h"
#include "row_io.h"
#include "wave_ops.h"

namespace flce {
namespace {

// Columns [c, c + 4) of a row of n: zero past the end.
__device__ __forceinline__ void load4(const float* row, int64_t c, int64_t n, float (&f)[4]) {
  load_chunk(row, c, n, f);
}
__device__ __forceinline__ void load4(const Bf16Bits* row, int64_t c, int64_t n, float (&f)[4]) {
  typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
  typedef u32x2 __attribute__((aligned(2))) u32x2_any;
  if (c + 4 <= n) {
    const u32x2 v = *reinterpret_cast<const u32x2_any*>(row + c);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      f[2 * e] = __uint_as_float(v[e] << 16);
      f[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = c + e < n ? to_f32(row[c + e]) : 0.f;
  }
}
__device__ __forceinline__ void store4(float* row, int64_t c, int64_t n, const float (&f)[4]) {
  store_chunk(row, c, n, f);
}
__device__ __forceinline__ void store4(Bf16Bits* row, int64_t c, int64_t n, const float (&f)[4]) {
  typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
  typedef u32x2 __attribute__((aligned(2))) u32x2_any;
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  if (c + 4 <= n) {
    u32x2 v;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bf16x2 p = {__bf16(f[2 * e]), __bf16(f[2 * e + 1])};
      v[e] = __builtin_bit_cast(uint32_t, p);
    }
    *reinterpret_cast<u32x2_any*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) row[c + e] = from_f32<Bf16Bits>(f[e]);
  }
}

__device__ __forceinline__ void store4(_Float16* row, int64_t c, int64_t n, const float (&f)[4]) {
  typedef __attribute__((ext_vector_type(4))) _Float16 f16x4;
  typedef f16x4 __attribute__((aligned(2))) f16x4_any;
  if (c + 4 <= n) {
    *reinterpret_cast<f16x4_any*>(row + c) =
        f16x4{_Float16(f[0]), _Float16(f[1]), _Float16(f[2]), _Float16(f[3])};
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < n) row[c + e] = _Float16(f[e]);
  }
}
// A chunk of slopes.
__device__ __forceinline__ void load_slope(const float* row, int64_t c, int64_t n, float (&f)[4]) {
  load_chunk(row, c, n, f);
}
__device__ __forceinline__ void load_slope(const _Float16* row, int64_t c, int64_t n,
                                           float (&f)[8]) {
  typedef __attribute__((ext_vector_type(8))) _Float16 f16x8;
  if (c + 8 <= n) {
    const f16x8 v = __builtin_bit_cast(f16x8, load_raw(row + c));
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = float(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = c + e < n ? float(row[c + e]) : 0.f;
  }
}
template <class T>
using Slope = std::conditional_t<sizeof(T) == 2, _Float16, float>;

// Columns [c, c + 4) of row r of a matrix of rows x n: as they are where the tile lies inside
// it (WHOLE), otherwise element by element from clamped places. No load has a condition:
// one would be waited for before the next is issued.
template <bool WHOLE, class T>
__device__ __forceinline__ void load4_at(const T* p, int64_t ld, int64_t r, int64_t c, int64_t rows,
                                         int64_t n, float (&f)[4]) {
  if constexpr (WHOLE) {
    load4(p + r * ld, c, c + 4, f);
  } else {
    const T* row = p + (r < rows ? r : rows - 1) * ld;
    T x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = row[c + e < n ? c + e : n - 1];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = to_f32(x[e]);
  }
}
template <bool WHOLE, class T>
__device__ __forceinline__ void store4_at(T* p, int64_t ld, int64_t r, int64_t c, int64_t rows,
                                          int64_t n, const float (&f)[4]) {
  if (WHOLE) store4(p + r * ld, c, c + 4, f);
  else if (r < rows && c < n) store4(p + r * ld, c, n, f);
}

// What follows z in the forward.
template <class T, class OT>
struct Finish {
  const T* bias;              // may be null
  const T* res;               // may be null
  int64_t ld_res;
  OT* y;
  int64_t ld_y;
  Slope<T>* slope;            // may be null; [N][O]
  int64_t N, O;
  // Columns c .. c + 3 of row r; bias and residual as load() left them, in memory's type (a
  // conversion would wait for them there).
  struct Ends {
    T b[4], t[4];
  };
  __device__ __forceinline__ Ends load(int64_t c, int64_t r) const {
    Ends s{};
    const int64_t rr = r < N ? r : N - 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t at = c + e < O ? c + e : O - 1;
      if (bias) s.b[e] = bias[at];
      if (res) s.t[e] = res[rr * ld_res + at];
    }
    return s;
  }
  __device__ __forceinline__ void store(int act, int64_t c, int64_t r, const float (&z)[4],
                                        const Ends& s) const {
    float v[4], d[4];
    with_activation(act, [&](auto k) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const Activated a = activate<decltype(k)::value, sizeof(OT) == 2>(z[e] + to_f32(s.b[e]));
        v[e] = a.y + to_f32(s.t[e]);
        d[e] = a.slope;
      }
    });
    if (slope) store4_at<false>(slope, O, r, c, N, O, d);
    store4_at<false>(y, ld_y, r, c, N, O, v);
  }
  // A lane's part of a tile of the small product.
  template <int ACT, bool WHOLE, int TS>
  __device__ __forceinline__ void store(const small::Acc<TS>& acc, int64_t c0, int64_t r0) const {
    constexpr int B = small::Acc<TS>::B;
    float b[B][4] = {}, t[B][B][4] = {};
    if (bias) {
#pragma unroll
      for (int i = 0; i < B; ++i) load4_at<WHOLE>(bias, 0, 0, c0 + 16 * i, 1, O, b[i]);
    }
    if (res) {
#pragma unroll
      for (int j = 0; j < B; ++j)
#pragma unroll
        for (int i = 0; i < B; ++i)
          load4_at<WHOLE>(res, ld_res, r0 + 16 * j, c0 + 16 * i, N, O, t[j][i]);
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int64_t r = r0 + 16 * j, c = c0 + 16 * i;
        float v[4], d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const Activated a = activate<ACT, sizeof(OT) == 2>(acc.v[i][j][e] + b[i][e]);
          v[e] = a.y + t[j][i][e];
          d[e] = a.slope;
        }
        if (slope) store4_at<WHOLE>(slope, O, r, c, N, O, d);
        store4_at<WHOLE>(y, ld_y, r, c, N, O, v);
      }
  }
};

// Tile `b` of na x nb: the XCDs (workgroups go to them in turn) take contiguous runs of
// tiles, in groups of four rows of tiles, so that one's tiles share operands in its L2.
template <int TS>
__device__ __forceinline__ void tile_at(int64_t b, int64_t na, int64_t nb, int64_t& a0,
                                        int64_t& b0) {
  constexpr int kGroup = 4;
  const int64_t total = na * nb, q = total / 8, rem = total % 8, x = b % 8;
  const int64_t t = x * q + (x < rem ? x : rem) + b / 8;
  const int64_t g = t / (kGroup * na), first = g * kGroup;
  const int64_t rows = nb - first < kGroup ? nb - first : kGroup;
  const int64_t in = t - g * kGroup * na;
  b0 = (first + in % rows) * TS;
  a0 = (in / rows) * TS;
}
template <int TS>
__host__ __device__ __forceinline__ int64_t tiles_of(int64_t n) {
  return (n + TS - 1) / TS;
}

template <class T, class OT, int TS, bool DIRECT>
__global__ __launch_bounds__(small::kThreads) void k_linear(small::Operand<T> W,
                                                            small::Operand<T> x, int64_t I,
                                                            Finish<T, OT> fin, int act) {
  __shared__ __attribute__((aligned(1024))) char smem[small::kSmemBytes<TS, DIRECT>];
  int64_t a0, b0;
  tile_at<TS>(blockIdx.x, tiles_of<TS>(W.rows), tiles_of<TS>(x.rows), a0, b0);
  small::Acc<TS> acc;
  small::tile<T, 0, 0, TS, DIRECT>(acc, W, x, a0, b0, I, smem);
  const int64_t c0 = small::lane_col<TS>(a0), r0 = small::lane_row<TS>(b0);
  const bool whole = a0 + TS <= W.rows && b0 + TS <= x.rows;
  with_activation(act, [&](auto k) {
    constexpr int ACT = decltype(k)::value;
    if (whole) fin.template store<ACT, true>(acc, c0, r0);
    else fin.template store<ACT, false>(acc, c0, r0);
  });
}

// ---- few rows -----------------------------------------------------------------------------
// A workgroup: 16 of W's rows and 16 NT rows of x; its eight waves take 256 bytes of k in
// turn, so that each loads both operands of its matrix instructions straight into registers
// and all of a short row is under way at once; their sums are joined in LDS in wave order.
// Bound by reading W, if it is large. What 64 rows of W a workgroup, each wave over all of k
// (as a head's), leave of a W of 4096 rows is 64 workgroups for 256 CUs.
// 16 rows of 4096, W 4096 x 4096: 10.7 us; tiles of 64 x 64 17, of 128 x 128 39.
constexpr int kFewWaves = 8;

template <class T, class OT, int NT>
__global__ __launch_bounds__(64 * kFewWaves) void k_linear_few(small::Operand<T> W,
                                                               small::Operand<T> x, int64_t I,
                                                               Finish<T, OT> fin, int act) {
  constexpr int E = kPerChunk<T>, KC = 16 * E;     // k of a chunk: four steps of 4 lanes' 16 bytes
  constexpr int D = NT == 1 ? 4 : 2;               // chunks loaded at once
  __shared__ __attribute__((aligned(16))) f32x4 red[kFewWaves][NT][64];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int r = lane & 15, kg = (lane >> 4) * E;
  const int64_t v0 = int64_t(blockIdx.x) * 16;
  const int64_t c = v0 + 4 * (lane >> 4);          // the finishing waves' column, row 16 w + r
  typename Finish<T, OT>::Ends ends{};
  if (w < NT) ends = fin.load(c, 16 * w + r);
  const T* wrow = W.p + (v0 + r < W.rows ? v0 + r : W.rows - 1) * I;
  const T* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xrow[j] = x.p + (16 * j + r < x.rows ? 16 * j + r : x.rows - 1) * x.ld;
  f32x4 acc[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) acc[j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const row_u32x4 (&a)[4], const row_u32x4 (&b)[NT][4]) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (sizeof(T) == 2) {
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a[s]),
                                                           __builtin_bit_cast(bf16x8, b[j][s]),
                                                           acc[j], 0, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                __uint_as_float(a[s][e]), __uint_as_float(b[j][s][e]), acc[j], 0, 0, 0);
        }
      }
#endif
  };
  const int64_t full = I / KC, end = full * KC;
  if (end < I && full % kFewWaves == w) {          // the rest of the rows, element by element
    T ea[4][E], eb[NT][4][E];
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int64_t k = end + s * 4 * E + kg + e, at = k < I ? k : I - 1;
        ea[s][e] = wrow[at];
#pragma unroll
        for (int j = 0; j < NT; ++j) eb[j][s][e] = xrow[j][at];
      }
    row_u32x4 a[4], b[NT][4];
    auto pack = [&](const T (&v)[E], int s) {
      float f[E];
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = end + s * 4 * E + kg + e < I ? to_f32(v[e]) : 0.f;
      return pack_chunk<T>(f);
    };
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      a[s] = pack(ea[s], s);
#pragma unroll
      for (int j = 0; j < NT; ++j) b[j][s] = pack(eb[j][s], s);
    }
    multiply(a, b);
  }
  // G chunks of the wave from its i-th on
  auto group = [&](auto count, int64_t i) {
    constexpr int G = decltype(count)::value;
    row_u32x4 a[G][4], b[G][NT][4];
#pragma unroll
    for (int u = 0; u < G; ++u) {
      const int64_t k = (w + (i + u) * kFewWaves) * KC + kg;
#pragma unroll
      for (int s = 0; s < 4; ++s) a[u][s] = load_raw(wrow + k + s * 4 * E);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s) b[u][j][s] = load_raw(xrow[j] + k + s * 4 * E);
    }
#pragma unroll
    for (int u = 0; u < G; ++u) multiply(a[u], b[u]);
  };
  int64_t i = 0, n = full > w ? (full - w + kFewWaves - 1) / kFewWaves : 0;
  for (; n - i >= D; i += D) group(std::integral_constant<int, D>{}, i);
  if (D > 3 && n - i == 3) group(std::integral_constant<int, 3>{}, i);
  else if (D > 2 && n - i == 2) group(std::integral_constant<int, 2>{}, i);
  else if (n - i == 1) group(std::integral_constant<int, 1>{}, i);
#pragma unroll
  for (int j = 0; j < NT; ++j) red[w][j][lane] = acc[j];
  __syncthreads();
  if (w >= NT) return;
  f32x4 v = red[0][w][lane];
#pragma unroll
  for (int i = 1; i < kFewWaves; ++i) v += red[i][w][lane];
  const float z[4] = {v[0], v[1], v[2], v[3]};
  fin.store(act, c, 16 * w + r, z, ends);
}

// A wide W, as a head: 64 RB of its rows a workgroup (few_rows.h). maxima, where given
// (float32 y): [N][gridDim.x], the largest of each workgroup's part of a row, so that what
// samples from it need not read it all again.
template <int NT, int ALIGN, int RB, class OT>
__global__ __launch_bounds__(256) void k_linear_wide(const uint16_t* __restrict__ W,
                                                     const uint16_t* __restrict__ x, int64_t ld_x,
                                                     int64_t I, Finish<Bf16Bits, OT> fin, int act,
                                                     float* __restrict__ maxima) {
  __shared__ __attribute__((aligned(16))) FewSmem<NT, RB> sm;
  const int64_t v0 = int64_t(blockIdx.x) * (64 * RB);
  few_logits<NT, ALIGN, RB>(x, ld_x, W, fin.N, I, fin.O, v0, sm);
  for (int i = threadIdx.x; i < 16 * NT * 16 * RB; i += 256) {
    const int64_t r = i / (16 * RB), c = v0 + 4 * (i % (16 * RB));
    if (r >= fin.N) break;
    const float* s = &sm.z[r][4 * (i % (16 * RB))];
    const float z[4] = {s[0], s[1], s[2], s[3]};
    fin.store(act, c, r, z, fin.load(c, r));
    if (maxima) {
      float m = -INFINITY;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < fin.O) m = MaxNanOp()(m, z[e]);
      m = group_all<16>(m, MaxNanOp());
      if (RB == 2) m = pair_rows(m, MaxNanOp());
      if (i % (16 * RB) == 0) maxima[r * gridDim.x + blockIdx.x] = m;
    }
  }
}

// The same behind the head's tiles: rows are tokens, columns W's rows. A lane has the same
// four columns in every row of its wave's 128 x 128 block; the residual's are loaded a
// pass of 32 rows ahead.
template <class OT, int ACT>
struct EpiLinear {
  Finish<Bf16Bits, OT> fin;
  bool res;

  struct Pass {
    const EpiLinear& e;
    int64_t r0, c0;
    int lane;
    float bias[4];
    uint2 res[2][16];
    __device__ __forceinline__ void prefetch(int i, int) {
      if (!e.res) return;
      const int64_t c = c0 + 4 * (lane & 31);
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t r = r0 + i * 32 + 2 * q + (lane >> 5);
        if (r < e.fin.N && c < e.fin.O)
          res[i & 1][q] = *reinterpret_cast<const uint2*>(e.fin.res + r * e.fin.ld_res + c);
      }
    }
    __device__ __forceinline__ void store(int i, int q, int row, int col, float4 v) {
      const int64_t r = r0 + i * 32 + row, c = c0 + col;
      if (r >= e.fin.N || c >= e.fin.O) return;
      const float z[4] = {v.x, v.y, v.z, v.w};
      float y[4], d[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const Activated a = activate<ACT, sizeof(OT) == 2>(z[k] + bias[k]);
        y[k] = a.y;
        d[k] = a.slope;
      }
      if (e.fin.slope) store4(e.fin.slope + r * e.fin.O, c, e.fin.O, d);
      if (e.res) {
        const uint2 o = res[i & 1][q];
        y[0] += bf16_to_f32(uint16_t(o.x));
        y[1] += bf16_to_f32(uint16_t(o.x >> 16));
        y[2] += bf16_to_f32(uint16_t(o.y));
        y[3] += bf16_to_f32(uint16_t(o.y >> 16));
      }
      store4(e.fin.y + r * e.fin.ld_y, c, e.fin.O, y);
    }
  };

  static constexpr int kTokBytes = 0;
  __device__ __forceinline__ void stage(char*, int64_t, int, int) const {}
  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char*) const {
    Pass pass{*this, m0 + wm * 128, n0 + wn * 128, lane, {0.f, 0.f, 0.f, 0.f}, {}};
    const int64_t c = n0 + wn * 128 + 4 * (lane & 31);
    if (fin.bias && c < fin.O) load4(fin.bias, c, fin.O, pass.bias);
    staged_rows(acc, wm, wn, lane, smem, pass);
  }
};

// A gradient's rows behind the head's tiles.
template <bool ACCUM>
struct EpiGrad {
  Bf16Bits* p;
  int64_t ld, rows, cols;

  struct Pass {
    const EpiGrad& e;
    int64_t r0, c0;
    __device__ __forceinline__ void prefetch(int, int) {}
    __device__ __forceinline__ void store(int i, int, int row, int col, float4 v) {
      const int64_t r = r0 + i * 32 + row, c = c0 + col;
      if (r >= e.rows || c >= e.cols) return;
      float f[4] = {v.x, v.y, v.z, v.w};
      if (ACCUM) {
        float o[4];
        load4(e.p + r * e.ld, c, e.cols, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] += o[k];
      }
      store4(e.p + r * e.ld, c, e.cols, f);
    }
  };

  static constexpr int kTokBytes = 0;
  __device__ __forceinline__ void stage(char*, int64_t, int, int) const {}
  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char*) const {
    Pass pass{*this, m0 + wm * 128, n0 + wn * 128};
    staged_rows(acc, wm, wn, lane, smem, pass);
  }
};

// A gradient's tiles: C[rows][cols], row stride ld.
template <class T>
struct GradOut {
  T* p;
  int64_t ld, rows, cols;
  int accumulate;
  template <bool WHOLE, int TS>
  __device__ __forceinline__ void store(const small::Acc<TS>& acc, int64_t c0, int64_t r0) const {
    constexpr int B = small::Acc<TS>::B;
    float t[B][B][4] = {};
    if (accumulate) {
#pragma unroll
      for (int j = 0; j < B; ++j)
#pragma unroll
        for (int i = 0; i < B; ++i)
          load4_at<WHOLE>(p, ld, r0 + 16 * j, c0 + 16 * i, rows, cols, t[j][i]);
    }
#pragma unroll
    for (int j = 0; j < B; ++j)
#pragma unroll
      for (int i = 0; i < B; ++i) {
        float f[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = acc.v[i][j][e] + t[j][i][e];
        store4_at<WHOLE>(p, ld, r0 + 16 * j, c0 + 16 * i, rows, cols, f);
      }
  }
  template <int TS>
  __device__ __forceinline__ void store_tile(const small::Acc<TS>& acc, int64_t a0,
                                             int64_t b0) const {
    const int64_t c0 = small::lane_col<TS>(a0), r0 = small::lane_row<TS>(b0);
    if (a0 + TS <= cols && b0 + TS <= rows) store<true>(acc, c0, r0);
    else store<false>(acc, c0, r0);
  }
};

// db from the workgroups' sums, in a fixed order: 16 columns a workgroup, 16 chains of
// every 16th sum, joined pairwise.
template <class T>
struct BiasGrad {
  const float* part;          // [np][O]; null: none
  int64_t np, O;
  T* db;
  int accumulate;
  __host__ __device__ int64_t groups() const { return part ? (O + 15) / 16 : 0; }
  __device__ __forceinline__ void run(int64_t group, float (*red)[17]) const {
    const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
    const int64_t c = group * 16 + col;
    float a = 0.f;
    if (c < O) {
#pragma unroll 8
      for (int64_t i = grp; i < np; i += 16) a += part[i * O + c];
    }
    red[grp][col] = a;
    __syncthreads();
    for (int k = 8; k > 0; k >>= 1) {
      if (grp < k) red[grp][col] += red[grp + k][col];
      __syncthreads();
    }
    if (grp == 0 && c < O) {
      const float v = red[0][col];
      db[c] = from_f32<T>(accumulate ? to_f32(db[c]) + v : v);
    }
  }
};

template <class T>
__global__ __launch_bounds__(256) void k_linear_db(BiasGrad<T> b) {
  __shared__ float red[16][17];
  b.run(blockIdx.x, red);
}

// One of the backward's products: C[rows][cols] = sum_k B(row, k) A(col, k) in tiles of TS,
// `segs` segments of k of each (1: whole).
template <class T>
struct Product {
  small::Operand<T> A, B;
  int64_t K, seg;
  int64_t tiles, segs;
  GradOut<T> out;             // segs = 1
  float* part;                // [segs][rows][cols] otherwise
  __host__ __device__ int64_t groups() const { return tiles * segs; }
  template <int FB, int TS, bool DIRECT>
  __device__ __forceinline__ void run(int64_t i, char* smem) const {
    const int64_t s = segs > 1 ? i / tiles : 0;
    small::Operand<T> a = A, b = B;
    int64_t k = K, a0, b0;
    if (segs > 1) {
      const int64_t k0 = s * seg;
      k = K - k0 < seg ? K - k0 : seg;
      a.p += k0 * a.ld;                            // form T
      b.p += FB == 0 ? k0 : k0 * b.ld;
    }
    tile_at<TS>(i - s * tiles, tiles_of<TS>(out.cols), tiles_of<TS>(out.rows), a0, b0);
    small::Acc<TS> acc;
    small::tile<T, 1, FB, TS, DIRECT>(acc, a, b, a0, b0, k, smem);
    if (segs > 1)
      GradOut<float>{part + s * out.rows * out.cols, out.cols, out.rows, out.cols, 0}.store_tile(
          acc, a0, b0);
    else
      out.store_tile(acc, a0, b0);
  }
};

// dx's tiles (n1 of them) and dW's (n2), those of the longer k first, the first kind's count
// padded to a multiple of 8, then db, in one grid. The mapping of tiles to XCDs goes by a
// tile's index, so segments of tiles that are no multiple of 8 are dealt a little unevenly.
template <class T, int TS, bool DIRECT>
__global__ __launch_bounds__(small::kThreads) void k_linear_grads(Product<T> dx, Product<T> dw,
                                                                  bool dw_first, BiasGrad<T> db) {
  __shared__ __attribute__((aligned(1024))) char smem[small::kSmemBytes<TS, DIRECT>];
  const int64_t b = blockIdx.x, n1 = dx.groups(), n2 = dw.groups();
  const int64_t first = ((dw_first ? n2 : n1) + 7) / 8 * 8, second = dw_first ? n1 : n2;
  if (b >= first + second) {
    db.run(b - first - second, reinterpret_cast<float (*)[17]>(smem));
    return;
  }
  const bool is_dw = (b < first) == dw_first;
  const int64_t t = b < first ? b : b - first;
  if (t >= (is_dw ? n2 : n1)) return;
  if (is_dw) dw.template run<1, TS, DIRECT>(t, smem);
  else dx.template run<0, TS, DIRECT>(t, smem);
}

// The partial products of split products added up, in order: dx's n1 groups of 256 chunks of
// four values, then dW's.
template <class T>
__global__ __launch_bounds__(256) void k_linear_join(Product<T> dx, Product<T> dw, int64_t n1) {
  const bool is_dw = int64_t(blockIdx.x) >= n1;
  const Product<T>& p = is_dw ? dw : dx;
  const int64_t cols = p.out.cols, n = p.out.rows * cols;
  const int64_t i = ((int64_t(blockIdx.x) - (is_dw ? n1 : 0)) * 256 + threadIdx.x) * 4;
  if (i >= n) return;
  float v[4];
  load_chunk(p.part, i, n, v);
#pragma unroll 4
  for (int64_t s = 1; s < p.segs; ++s) {
    float o[4];
    load_chunk(p.part + s * n, i, n, o);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += o[e];
  }
  const int64_t r = i / cols, c = i - r * cols;
  if (c + 4 <= cols) {
    T* row = p.out.p + r * p.out.ld;
    if (p.out.accumulate) {
      float o[4];
      load4(row, c, cols, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += o[e];
    }
    store4(row, c, cols, v);
  } else {
    for (int e = 0; e < 4 && i + e < n; ++e) {
      T* at = p.out.p + (i + e) / cols * p.out.ld + (i + e) % cols;
      *at = from_f32<T>(p.out.accumulate ? to_f32(*at) + v[e] : v[e]);
    }
  }
}

// dz = dy slope (rounded; SLOPE false: dz is dy, not written), and the workgroup's rows'
// sums of dz in its row of part[][O] (null: not wanted). A workgroup takes `rows` rows
// of 32 chunks of columns, 8 rows at a time; cols workgroups stand side by side.
template <class T, bool SLOPE>
__global__ __launch_bounds__(256) void k_linear_dz(const T* __restrict__ dy, int64_t ld_dy,
                                                   const Slope<T>* __restrict__ slope,
                                                   int64_t N, int64_t O, T* __restrict__ dz,
                                                   float* __restrict__ part, uint32_t cols,
                                                   int rows) {
  constexpr int E = kPerChunk<T>;
  __shared__ float red[8][32 * E + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const uint32_t by = blockIdx.x / cols, bx = blockIdx.x - by * cols;
  const int64_t c = (int64_t(bx) * 32 + tx) * E;
  const int64_t r0 = int64_t(by) * rows;
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
  if (c < O) {
#pragma unroll 4
    for (int i = ty; i < rows; i += 8) {
      const int64_t r = r0 + i;
      if (r >= N) break;
      float g[E];
      load_chunk(dy + r * ld_dy, c, O, g);
      if (SLOPE) {
        float d[E];
        load_slope(slope + r * O, c, O, d);
#pragma unroll
        for (int e = 0; e < E; ++e) g[e] *= d[e];
        store_chunk(dz + r * O, c, O, g);
      }
#pragma unroll
      for (int e = 0; e < E; ++e) sum[e] += g[e];
    }
  }
  if (!part) return;
#pragma unroll
  for (int e = 0; e < E; ++e) red[ty][tx * E + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * E; i += 256) {
    const int64_t col = int64_t(bx) * 32 * E + i;
    if (col >= O) break;
    float v = red[0][i];
#pragma unroll
    for (int k = 1; k < 8; ++k) v += red[k][i];
    part[int64_t(by) * O + col] = v;
  }
}

// Whether every row starts at a multiple of 16 bytes.
template <class T>
bool aligned16(std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  for (int64_t l : lds)
    if (l % kPerChunk<T>) return false;
  return true;
}

// run(the tile's edge, whether its loads are direct).
template <class T, class F>
void with_tile(int64_t edge, bool direct, F&& run) {
  auto go = [&](auto e) { direct ? run(e, std::true_type{}) : run(e, std::false_type{}); };
  if (edge == 128) go(std::integral_constant<int, 128>{});
  else if (edge == 64) go(std::integral_constant<int, 64>{});
  else if constexpr (sizeof(T) == 4) go(std::integral_constant<int, 32>{});
}

// Whether a product of a x b outputs runs on the head's tiles: enough of them for most of
// the 256 CUs (a workgroup each).
bool on_large_tiles(int64_t a, int64_t b) { return gemm::num_tiles(a, b) >= kLinearLargeTiles; }

// An operand of the head's product.
struct Large {
  int form;
  const void* p;
  gemm::Geom g;
  bool fits() const {
    return operand_offsets_fit(form, g) && (form == gemm::kFormN || g.rows >= 8);
  }
  Operand op() const { return Operand{static_cast<const uint16_t*>(p), g}; }
};

template <class OT>
bool forward_large(const LinearArgs& a, const Finish<Bf16Bits, OT>& fin, const Launcher& L) {
  const Large x{gemm::kFormN, a.x, {a.ld_x, a.N, a.I}}, W{gemm::kFormN, a.weight, {a.I, a.O, a.I}};
  if (!on_large_tiles(a.N, a.O) || !x.fits() || !W.fits()) return false;
  if (!aligned16<Bf16Bits>({a.x, a.weight, a.bias, a.residual, a.y, a.slope},
                 {a.I, a.O, a.ld_x, a.ld_y, a.residual ? a.ld_res : 0}))
    return false;
  with_activation(a.activation, [&](auto act) {
    using Epi = EpiLinear<OT, decltype(act)::value>;
    hipLaunchKernelGGL((k_gemm<0, 0, Epi, kDynNone>), dim3(unsigned(gemm::num_tiles(a.N, a.O))),
                       dim3(kThreads), 0, L.stream, x.op(), W.op(), a.N, a.O, a.I, gemm::kGroupM,
                       Epi{fin, a.residual != nullptr}, nullptr);
  });
  return true;
}

// Whether a forward takes k_linear_wide. few_rows.h reads odd rows as the words they lie in:
// dense rows, from aligned addresses.
bool takes_wide(const LinearArgs& a) {
  if (a.dtype != FLCE_BF16 || a.N > kFewTokens || a.O < kLinearWide) return false;
  return aligned16<Bf16Bits>({a.weight, a.x}, {}) &&
         (a.ld_x == a.I || aligned16<Bf16Bits>({}, {a.I, a.ld_x}));
}

template <class T, class OT>
bool forward_few(const LinearArgs& a, const Finish<T, OT>& fin, const Launcher& L) {
  const T* W = static_cast<const T*>(a.weight);
  const T* x = static_cast<const T*>(a.x);
  if constexpr (sizeof(T) == 2) {
    if (takes_wide(a)) {
      const bool whole = aligned16<T>({}, {a.I, a.ld_x});
      with_few(a.N, [&](auto nt, auto rb) {
        constexpr int NT = decltype(nt)::value, RB = decltype(rb)::value;
        auto go = [&](auto align) {
          hipLaunchKernelGGL((k_linear_wide<NT, decltype(align)::value, RB, OT>),
                             dim3(unsigned((a.O + 64 * RB - 1) / (64 * RB))), dim3(256), 0, L.stream,
                             W, x, a.ld_x, a.I, fin, a.activation, a.maxima);
        };
        if (whole) go(std::integral_constant<int, 16>{});
        else if (a.I % 2 == 0) go(std::integral_constant<int, 4>{});
        else go(std::integral_constant<int, 2>{});
      });
      return true;
    }
  }
  if (a.N > kLinearFew) return false;
  auto go = [&](auto nt) {
    hipLaunchKernelGGL((k_linear_few<T, OT, decltype(nt)::value>), dim3(unsigned((a.O + 15) / 16)),
                       dim3(64 * kFewWaves), 0, L.stream, small::Operand<T>{W, a.I, a.O},
                       small::Operand<T>{x, a.ld_x, a.N}, a.I, fin, a.activation);
  };
  if (a.N <= 16) go(std::integral_constant<int, 1>{});
  else if (a.N <= 32) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 4>{});
  return true;
}

template <class T, class OT>
hipError_t forward(const LinearArgs& a, const Launcher& L) {
  const T* W = static_cast<const T*>(a.weight);
  const T* x = static_cast<const T*>(a.x);
  const Finish<T, OT> fin{static_cast<const T*>(a.bias), static_cast<const T*>(a.residual),
                          a.ld_res, static_cast<OT*>(a.y), a.ld_y, static_cast<Slope<T>*>(a.slope),
                          a.N, a.O};
  L.pre(kLinear);
  if (forward_few<T, OT>(a, fin, L)) {
    L.post(kLinear);
    return hipGetLastError();
  }
  if constexpr (sizeof(T) == 2) {
    if (forward_large<OT>(a, fin, L)) {
      L.post(kLinear);
      return hipGetLastError();
    }
  }
  const bool direct = aligned16<T>({a.x, a.weight}, {a.I, a.ld_x});
  with_tile<T>(linear_tile(tiles_of<128>(a.O) * tiles_of<128>(a.N), a.dtype), direct, [&](auto ts, auto di) {
    constexpr int TS = decltype(ts)::value;
    const dim3 grid(unsigned(tiles_of<TS>(a.O) * tiles_of<TS>(a.N)));
    hipLaunchKernelGGL((k_linear<T, OT, TS, decltype(di)::value>), grid, dim3(small::kThreads), 0,
                       L.stream, small::Operand<T>{W, a.I, a.O},
                       small::Operand<T>{x, a.ld_x, a.N}, a.I, fin, a.activation);
  });
  L.post(kLinear);
  return hipGetLastError();
}

// dx and dW in one grid, dx's tiles first.
bool backward_large(const LinearBwdArgs& a, const Bf16Bits* g, int64_t ld_g, const Launcher& L) {
  if (!a.dx || !a.dweight || !on_large_tiles(a.N + a.O, a.I)) return false;
  const Large g1{gemm::kFormN, g, {ld_g, a.N, a.O}}, W{gemm::kFormT, a.weight, {a.I, a.I, a.O}};
  const Large g2{gemm::kFormT, g, {ld_g, a.O, a.N}}, x{gemm::kFormT, a.x, {a.ld_x, a.I, a.N}};
  if (!g1.fits() || !W.fits() || !g2.fits() || !x.fits()) return false;
  if (!aligned16<Bf16Bits>({g, a.weight, a.x, a.dx, a.dweight}, {a.I, a.O, ld_g, a.ld_x, a.ld_dx}))
    return false;
  const int64_t n1 = gemm::num_tiles(a.N, a.I), n1p = (n1 + 7) / 8 * 8;
  const int64_t n2 = gemm::num_tiles(a.O, a.I);
  const EpiGrad<false> e1{static_cast<Bf16Bits*>(a.dx), a.ld_dx, a.N, a.I};
  auto go = [&](auto accum) {
    using Epi2 = EpiGrad<decltype(accum)::value>;
    hipLaunchKernelGGL((k_gemm_pair<0, 1, EpiGrad<false>, kDynNone, false, 1, 1, Epi2, kDynNone, 1>),
                       dim3(unsigned(n1p + n2)), dim3(kThreads), 0, L.stream, n1p, n1, n1, int64_t(0),
                       g1.op(), W.op(), a.N, a.I, a.O, e1, g2.op(), x.op(), a.O, a.I, a.N,
                       Epi2{static_cast<Bf16Bits*>(a.dweight), a.I, a.O, a.I}, int64_t(0), nullptr);
  };
  L.pre(kLinearGrad);
  a.accumulate ? go(std::true_type{}) : go(std::false_type{});
  L.post(kLinearGrad);
  return true;
}

template <class T>
hipError_t backward(const LinearPlan& p, const LinearBwdArgs& a, char* ws, const Launcher& L) {
  const T* dy = static_cast<const T*>(a.dy);
  const auto* slope = static_cast<const Slope<T>*>(a.slope);
  const T* x = static_cast<const T*>(a.x);
  T* dz = reinterpret_cast<T*>(ws + p.off_dz);
  float* part = a.dbias ? reinterpret_cast<float*>(ws + p.off_part) : nullptr;
  hipError_t e = hipSuccess;
  if (slope || part) {
    constexpr int kCols = 32 * kPerChunk<T>;
    const uint32_t cols = uint32_t((a.O + kCols - 1) / kCols);
    const dim3 grid(unsigned(cols * p.dz_parts));
    L.pre(kLinearGrad);
    if (slope)
      hipLaunchKernelGGL((k_linear_dz<T, true>), grid, dim3(256), 0, L.stream, dy, a.ld_dy, slope,
                         a.N, a.O, dz, part, cols, int(p.dz_rows));
    else
      hipLaunchKernelGGL((k_linear_dz<T, false>), grid, dim3(256), 0, L.stream, dy, a.ld_dy, slope,
                         a.N, a.O, dz, part, cols, int(p.dz_rows));
    L.post(kLinearGrad);
    e = hipGetLastError();
  }
  if (e != hipSuccess) return e;
  BiasGrad<T> db{part, p.dz_parts, a.O, static_cast<T*>(a.dbias), a.accumulate};
  auto bias_alone = [&] {
    if (!part) return hipSuccess;
    L.pre(kLinearGrad);
    hipLaunchKernelGGL(k_linear_db<T>, dim3(unsigned(db.groups())), dim3(256), 0, L.stream, db);
    L.post(kLinearGrad);
    return hipGetLastError();
  };
  if (!a.dx && !a.dweight) return bias_alone();
  const T* g = slope ? dz : dy;
  const int64_t ld_g = slope ? a.O : a.ld_dy;
  if constexpr (sizeof(T) == 2) {
    if (backward_large(a, g, ld_g, L)) {
      e = hipGetLastError();
      return e == hipSuccess ? bias_alone() : e;
    }
  }
  L.pre(kLinearGrad);
  bool direct = aligned16<T>({g}, {ld_g, a.I});
  if (a.dx) direct = direct && aligned16<T>({a.weight}, {});
  if (a.dweight) direct = direct && aligned16<T>({x}, {a.ld_x, a.O});
  Product<T> dx{{static_cast<const T*>(a.weight), a.I, a.I}, {g, ld_g, a.N}, a.O, p.dx.seg, 0,
                p.dx.segs, {static_cast<T*>(a.dx), a.ld_dx, a.N, a.I, 0},
                reinterpret_cast<float*>(ws + p.off_dx)};
  Product<T> dw{{x, a.ld_x, a.I}, {g, ld_g, a.O}, a.N, p.dw.seg, 0, p.dw.segs,
                {static_cast<T*>(a.dweight), a.I, a.O, a.I, a.accumulate},
                reinterpret_cast<float*>(ws + p.off_dw)};
  const bool dw_first = a.N > a.O;
  with_tile<T>(p.tile, direct, [&](auto ts, auto di) {
    constexpr int TS = decltype(ts)::value;
    if (a.dx) dx.tiles = tiles_of<TS>(a.I) * tiles_of<TS>(a.N);
    if (a.dweight) dw.tiles = tiles_of<TS>(a.I) * tiles_of<TS>(a.O);
    const int64_t n1 = dx.groups(), n2 = dw.groups();
    const int64_t tiles = ((dw_first ? n2 : n1) + 7) / 8 * 8 + (dw_first ? n1 : n2);
    hipLaunchKernelGGL((k_linear_grads<T, TS, decltype(di)::value>),
                       dim3(unsigned(tiles + db.groups())), dim3(small::kThreads), 0, L.stream, dx,
                       dw, dw_first, db);
  });
  L.post(kLinearGrad);
  e = hipGetLastError();
  auto join_groups = [](const Product<T>& q) {
    return q.tiles && q.segs > 1 ? (q.out.rows * q.out.cols + 1023) / 1024 : 0;
  };
  const int64_t j1 = join_groups(dx), j2 = join_groups(dw);
  if (e != hipSuccess || j1 + j2 == 0) return e;
  L.pre(kLinearGrad);
  hipLaunchKernelGGL(k_linear_join<T>, dim3(unsigned(j1 + j2)), dim3(256), 0, L.stream, dx, dw, j1);
  L.post(kLinearGrad);
  return hipGetLastError();
}

}  // namespace

int64_t linear_max_blocks(const LinearArgs& a) {
  if (!takes_wide(a)) return 0;
  int64_t n = 0;
  with_few(a.N, [&](auto, auto rb) {
    constexpr int kCols = 64 * decltype(rb)::value;
    n = (a.O + kCols - 1) / kCols;
  });
  return n;
}

hipError_t launch_linear(const LinearArgs& a, const Launcher& L) {
  if (a.dtype == FLCE_F32) return forward<float, float>(a, L);
  if (a.y_dtype == FLCE_F32) return forward<Bf16Bits, float>(a, L);
  return forward<Bf16Bits, Bf16Bits>(a, L);
}

hipError_t launch_linear_backward(const LinearPlan& p, const LinearBwdArgs& a, char* ws,
                                  const Launcher& L) {
  return a.dtype == FLCE_F32 ? backward<float>(p, a, ws, L) : backward<Bf16Bits>(p, a, ws, L);
}

}  // namespace flce
