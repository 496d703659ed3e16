// The linear transform y = act(x W^T + b) + r, with W [O][I], and its backward:
//   dz = dy act'(z);  dx = dz W;  dW = dz^T x;  db = sum over rows of dz   (dr is dy)
// The forward stores the slope act'(z) where a backward will want it: dz then needs no z
// and no exponential. With bf16 rows it is an IEEE half: slopes are at most 1.13, so its
// range does, and its half step of 2^-12 leaves dz's own rounding (2^-9) the only one
// that counts; a bf16 slope made the gradients' error 0.0029 of their size instead of
// 0.0024, where rounding the exact ones once leaves 0.0017.
//
// Everything is float32 between a load and a store; what is rounded besides the outputs
// is the slope and dz (bf16 rows: the products' operand). db sums dz before its rounding.
//
// Products of bf16 rows whose lengths and addresses are multiples of 16 bytes, with enough
// tiles of 256 x 256 to fill the chip, run on the head's product (gemm_bf16.h); all others
// on the one of 128 x 128 tiles (gemm_small.h).
#include <hip/hip_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <type_traits>

#include "../../include/flce.h"
#include "activation.h"
#include "flce_internal.h"
#include "gemm_bf16.h"
#include "gemm_small.h"
#include "ops_plan.h"
#include "row_io.h"

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

// What follows z in the forward, four columns of a row at a time.
template <class T, class OT>
struct Finish {
  const T* bias;              // may be null
  const T* res;               // may be null
  int64_t ld_res;
  OT* y;
  int64_t ld_y;
  Slope<T>* slope;            // may be null; [N][O]
  int64_t N, O;
  template <int ACT>
  __device__ __forceinline__ void store(int64_t c, int64_t r, float (&z)[4]) const {
    if (r >= N || c >= O) return;
    float t[4], d[4];
    if (bias) {
      load4(bias, c, O, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += t[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const Activated a = activate<ACT, sizeof(OT) == 2>(z[e]);
      z[e] = a.y;
      d[e] = a.slope;
    }
    if (slope) store4(slope + r * O, c, O, d);
    if (res) {
      load4(res + r * ld_res, c, O, t);
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] += t[e];
    }
    store4(y + r * ld_y, c, O, z);
  }
};

// Tile `b` of na x nb: the XCDs (workgroups go to them in turn) take contiguous runs of
// tiles, in groups of four rows of tiles, so that one's tiles share operands in its L2.
__device__ __forceinline__ void tile_at(int64_t b, int64_t na, int64_t nb, int64_t& a0,
                                        int64_t& b0) {
  constexpr int kGroup = 4;
  const int64_t total = na * nb, q = total / 8, rem = total % 8, x = b % 8;
  const int64_t t = x * q + (x < rem ? x : rem) + b / 8;
  const int64_t g = t / (kGroup * na), first = g * kGroup;
  const int64_t rows = nb - first < kGroup ? nb - first : kGroup;
  const int64_t in = t - g * kGroup * na;
  b0 = (first + in % rows) * small::kTile;
  a0 = (in / rows) * small::kTile;
}
__host__ __device__ __forceinline__ int64_t tiles_of(int64_t n) {
  return (n + small::kTile - 1) / small::kTile;
}

template <class T, class OT, int ACT>
__global__ __launch_bounds__(small::kThreads) void k_linear(small::Operand<T> W,
                                                            small::Operand<T> x, int64_t I,
                                                            Finish<T, OT> fin) {
  __shared__ __attribute__((aligned(16))) char smem[4 * small::kStageBytes];
  int64_t a0, b0;
  tile_at(blockIdx.x, tiles_of(W.rows), tiles_of(x.rows), a0, b0);
  small::Acc acc;
  small::tile<T, 0, 0>(acc, W, x, a0, b0, I, smem);
  small::for_acc(acc, a0, b0, [&](int64_t c, int64_t r, const small::f32x4& v) {
    float z[4] = {v[0], v[1], v[2], v[3]};
    fin.template store<ACT>(c, r, z);
  });
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
      if (ACT != FLCE_ACT_NONE && e.fin.slope) store4(e.fin.slope + r * e.fin.O, c, e.fin.O, d);
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
  __device__ __forceinline__ void store(int64_t c, int64_t r, const small::f32x4& v) const {
    if (r >= rows || c >= cols) return;
    float f[4] = {v[0], v[1], v[2], v[3]};
    if (accumulate) {
      float o[4];
      load4(p + r * ld, c, cols, o);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] += o[e];
    }
    store4(p + r * ld, c, cols, f);
  }
};

// dx's tiles (n1 of them, padded to a multiple of 8) and then dW's, in one grid.
template <class T>
__global__ __launch_bounds__(small::kThreads) void k_linear_grads(
    int64_t n1, int64_t n1p, small::Operand<T> Wt, small::Operand<T> dz, int64_t O,
    GradOut<T> dx, small::Operand<T> xt, small::Operand<T> dzt, int64_t N, GradOut<T> dw) {
  __shared__ __attribute__((aligned(16))) char smem[4 * small::kStageBytes];
  const int64_t b = blockIdx.x;
  int64_t a0, b0;
  small::Acc acc;
  if (b < n1p) {
    if (b >= n1) return;
    tile_at(b, tiles_of(dx.cols), tiles_of(dx.rows), a0, b0);
    small::tile<T, 1, 0>(acc, Wt, dz, a0, b0, O, smem);
    small::for_acc(acc, a0, b0,
                   [&](int64_t c, int64_t r, const small::f32x4& v) { dx.store(c, r, v); });
  } else {
    tile_at(b - n1p, tiles_of(dw.cols), tiles_of(dw.rows), a0, b0);
    small::tile<T, 1, 1>(acc, xt, dzt, a0, b0, N, smem);
    small::for_acc(acc, a0, b0,
                   [&](int64_t c, int64_t r, const small::f32x4& v) { dw.store(c, r, v); });
  }
}

// dz = dy slope (rounded; SLOPE false: dz is dy, not written), and the workgroup's rows'
// sums of dz in its row of part[][O] (null: not wanted). A workgroup takes kLinearDzRows
// rows of 32 chunks of columns, 8 rows at a time; cols workgroups stand side by side.
template <class T, bool SLOPE>
__global__ __launch_bounds__(256) void k_linear_dz(const T* __restrict__ dy, int64_t ld_dy,
                                                   const Slope<T>* __restrict__ slope,
                                                   int64_t N, int64_t O, T* __restrict__ dz,
                                                   float* __restrict__ part, uint32_t cols) {
  constexpr int E = kPerChunk<T>;
  __shared__ float red[8][32 * E + 1];
  const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const uint32_t by = blockIdx.x / cols, bx = blockIdx.x - by * cols;
  const int64_t c = (int64_t(bx) * 32 + tx) * E;
  const int64_t r0 = int64_t(by) * kLinearDzRows;
  float sum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) sum[e] = 0.f;
  if (c < O) {
#pragma unroll 4
    for (int i = ty; i < kLinearDzRows; i += 8) {
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

// db from the workgroups' sums, in a fixed order: 16 columns a workgroup, 16 chains of
// every 16th sum, joined pairwise.
template <class T>
__global__ __launch_bounds__(256) void k_linear_db(const float* __restrict__ part, int64_t np,
                                                   int64_t O, T* __restrict__ db, int accumulate) {
  __shared__ float red[16][17];
  const int col = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 16 + col;
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

bool aligned16(std::initializer_list<const void*> ptrs, std::initializer_list<int64_t> lds) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) % 16) return false;
  for (int64_t l : lds)
    if (l % 8) return false;
  return true;
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
  if (!aligned16({a.x, a.weight, a.bias, a.residual, a.y, a.slope},
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

template <class T, class OT>
hipError_t forward(const LinearArgs& a, const Launcher& L) {
  const T* W = static_cast<const T*>(a.weight);
  const T* x = static_cast<const T*>(a.x);
  const Finish<T, OT> fin{static_cast<const T*>(a.bias), static_cast<const T*>(a.residual),
                          a.ld_res, static_cast<OT*>(a.y), a.ld_y, static_cast<Slope<T>*>(a.slope),
                          a.N, a.O};
  L.pre(kLinear);
  if constexpr (sizeof(T) == 2) {
    if (forward_large<OT>(a, fin, L)) {
      L.post(kLinear);
      return hipGetLastError();
    }
  }
  with_activation(a.activation, [&](auto act) {
    const dim3 grid(unsigned(tiles_of(a.O) * tiles_of(a.N)));
    hipLaunchKernelGGL((k_linear<T, OT, decltype(act)::value>), grid, dim3(small::kThreads), 0,
                       L.stream, small::Operand<T>{W, a.I, a.O}, small::Operand<T>{x, a.ld_x, a.N},
                       a.I, fin);
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
  if (!aligned16({g, a.weight, a.x, a.dx, a.dweight}, {a.I, a.O, ld_g, a.ld_x, a.ld_dx}))
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
  a.accumulate ? go(std::true_type{}) : go(std::false_type{});
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
                         a.N, a.O, dz, part, cols);
    else
      hipLaunchKernelGGL((k_linear_dz<T, false>), grid, dim3(256), 0, L.stream, dy, a.ld_dy, slope,
                         a.N, a.O, dz, part, cols);
    L.post(kLinearGrad);
    e = hipGetLastError();
  }
  if (e == hipSuccess && part) {
    L.pre(kLinearGrad);
    hipLaunchKernelGGL(k_linear_db<T>, dim3(unsigned((a.O + 15) / 16)), dim3(256), 0, L.stream, part,
                       p.dz_parts, a.O, static_cast<T*>(a.dbias), a.accumulate);
    L.post(kLinearGrad);
    e = hipGetLastError();
  }
  if (e != hipSuccess || (!a.dx && !a.dweight)) return e;
  const T* g = slope ? dz : dy;
  const int64_t ld_g = slope ? a.O : a.ld_dy;
  if constexpr (sizeof(T) == 2) {
    L.pre(kLinearGrad);
    const bool done = backward_large(a, g, ld_g, L);
    L.post(kLinearGrad);
    if (done) return hipGetLastError();
  }
  const int64_t n1 = a.dx ? tiles_of(a.I) * tiles_of(a.N) : 0, n1p = (n1 + 7) / 8 * 8;
  const int64_t n2 = a.dweight ? tiles_of(a.I) * tiles_of(a.O) : 0;
  L.pre(kLinearGrad);
  hipLaunchKernelGGL(k_linear_grads<T>, dim3(unsigned(n1p + n2)), dim3(small::kThreads), 0, L.stream,
                     n1, n1p, small::Operand<T>{static_cast<const T*>(a.weight), a.I, a.I},
                     small::Operand<T>{g, ld_g, a.N}, a.O,
                     GradOut<T>{static_cast<T*>(a.dx), a.ld_dx, a.N, a.I, 0},
                     small::Operand<T>{x, a.ld_x, a.I}, small::Operand<T>{g, ld_g, a.O}, a.N,
                     GradOut<T>{static_cast<T*>(a.dweight), a.I, a.O, a.I, a.accumulate});
  L.post(kLinearGrad);
  return hipGetLastError();
}

}  // namespace

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
