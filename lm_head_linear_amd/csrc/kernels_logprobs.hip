// Log probabilities of given tokens, entropy and top alternatives over the head's
// logits, and the logit gradient of the first two.
//
// With z = h W^T, x = softcap(z) / temperature, one pass over the vocabulary
// keeps per tile and token
//   m = max x,  s = sum exp(x - m),  d = sum exp(x - m) (x - m)
// which join over tiles by rescaling to the larger max:
//   s' = s exp(m - M),  d' = exp(m - M) (d + (m - M) s)
// so that  lse = M + log S,  log p_y = (x_y - M) - log S,  entropy = log S - D / S.
// log S is taken apart from M: a token that holds nearly all of the probability
// keeps its small log probability. Alternatives are ranked by the raw logit z (the
// order of x, without the ties that rounding x makes), equal ones by lowest id:
// each tile leaves its kc largest, sorted, and the join merges the lists.
//
// Three kernels compute logits:
//  - the 256 x 256 bf16 tiles of the head's own forward (gemm_bf16.h), live tokens
//    gathered first: bound by the matrix cores;
//  - few bf16 tokens: 64 vocabulary rows a workgroup, W streamed from memory
//    straight into the matrix cores' operand registers: bound by reading W once;
//  - float32: 64 x 64 tiles on the float32 matrix instruction.
// Logits are never stored in device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/flce.h"
#include "flce_internal.h"
#include "gemm_bf16.h"
#include "ops_plan.h"
#include "row_io.h"

namespace flce {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kLpTop = FLCE_MAX_TOP;

// x of a raw logit: capped, then divided by the temperature. cap_t = cap / T.
struct Warp {
  float inv_cap, cap_t, inv_t;
};
template <bool SOFTCAP>
__device__ __forceinline__ float warp_logit(const Warp& w, float z) {
  return SOFTCAP ? w.cap_t * tanh_fast(z * w.inv_cap) : z * w.inv_t;
}
// dx / dz
template <bool SOFTCAP>
__device__ __forceinline__ float warp_slope(const Warp& w, float z) {
  if (!SOFTCAP) return w.inv_t;
  const float th = tanh_fast(z * w.inv_cap);
  return w.inv_t * (1.f - th * th);
}
Warp make_warp(float softcap, float temperature) {
  const float it = 1.f / temperature;
  return Warp{softcap > 0.f ? 1.f / softcap : 0.f, softcap * it, it};
}

// Where a tile's results go (see LpPlan's strides).
struct LpOut {
  float2* part;               // m, s
  float* pd;                  // d
  float* zt;                  // x of the given token, one writer per token
  float* cv;                  // candidates: raw logit, -inf behind the last
  uint8_t* ci;                //   and its row within the list
  int64_t sp, st, cl, ck, ct;
  int kc;
};

__device__ __forceinline__ uint32_t min4(uint32_t x) {
  // min over the four lanes of an accumulator column (see col_max4)
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = a[0] < a[1] ? a[0] : a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = b[0] < b[1] ? b[0] : b[1];
#endif
  return x;
}

// ---- epilogue of the 256 x 256 tiles ----------------------------------------------
// The accumulators are raw logits, tile rows vocabulary ids, columns tokens (see
// EpiLse for the layout). The two waves of a column join their (m, s, d) through
// LDS; each wave leaves candidates of its own 128 rows. A candidate has to exceed
// tau, the token's kc-th largest logit among lower ids (-inf before any are known):
// an equal one with a higher id could not be listed either. Each round takes the
// column's largest logit left, lowest row first, in the four lanes that hold the
// column; a wave stops when none of its 16 columns has one left.
template <bool SOFTCAP, bool TOPK>
struct EpiLp {
  const int64_t* labels;      // null: no given tokens
  int64_t N, V, v0;           // v0: vocabulary id of launch row 0
  Warp warp;
  LpOut out;
  const float* tau;           // TOPK; null: -inf

  static constexpr int kTokBytes = 3072;
  __device__ __forceinline__ void stage(char* tok, int64_t n0, int wave, int lane) const {
    if (labels) stage_tokens<2>(tok, labels, n0, N, wave, lane);
    if (TOPK && tau) stage_tokens<1>(tok + 2048, tau, n0, N, wave, lane);
  }

  template <bool FULL>
  __device__ __forceinline__ void columns(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                          int lane, const char* tok, float (&mx)[8],
                                          float (&sm)[8], float (&dm)[8]) const {
    const int64_t* lab = reinterpret_cast<const int64_t*>(tok);
    const float* tau_t = reinterpret_cast<const float*>(tok + 2048);
    const int g = lane >> 4;
    const int64_t vbase = v0 + m0 + wm * 128;        // vocabulary id of the wave's row 0
    const int live = FULL ? 128 : int(V - vbase < 128 ? (V - vbase > 0 ? V - vbase : 0) : 128);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t t = n0 + acc_col(wn, j, lane);
      auto in = [&](int i, int r) { return FULL || i * 16 + 4 * g + r < live; };
      float x[8][4];
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[i][r] = warp_logit<SOFTCAP>(warp, acc[i][j][r]);
          mq[r] = fmaxf(mq[r], in(i, r) ? x[i][r] : -INFINITY);
        }
      if (labels) {
        const int64_t y = t < N ? lab[acc_col(wn, j, lane)] : -1;
        if (y >= vbase && y < vbase + live) {
          const int d = int(y - vbase);
          if (((d >> 2) & 3) == g) {
            const int ti = d >> 4, tr = d & 3;
            float val = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
              for (int r = 0; r < 4; ++r) val = (i == ti && r == tr) ? x[i][r] : val;
            out.zt[t] = val;
          }
        }
      }
      const float m = col_max4(fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3])));
      float s = 0.f, d = 0.f;
      if (m != -INFINITY) {
        // in powers of two: u = (x - m) log2 e, d in units of ln 2
        const float mb = m * kLog2e;
        float sq[2] = {0.f, 0.f}, dq[2] = {0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            // a row past the vocabulary: 2^-200 = 0; a logit of -inf keeps -inf out of d
            float u = fmaf(x[i][r], kLog2e, -mb);
            u = (in(i, r) && u != -INFINITY) ? u : -200.f;
            const float e = __builtin_amdgcn_exp2f(u);
            sq[r & 1] += e;
            dq[r & 1] = fmaf(e, u, dq[r & 1]);
          }
        s = sq[0] + sq[1];
        d = (dq[0] + dq[1]) * kLn2;
      }
      mx[j] = m;
      sm[j] = col_sum4(s);
      dm[j] = col_sum4(d);
      if (TOPK && live > 0) {                      // rows past V have no list
        const float th = tau ? tau_t[acc_col(wn, j, lane)] : -INFINITY;
        float z[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) z[i][r] = in(i, r) ? acc[i][j][r] : -INFINITY;
        const int64_t list = (vbase >> 7) * out.cl + t * out.ct;
        int n = 0;
        for (; n < out.kc; ++n) {
          float b = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) b = fmaxf(b, z[i][r]);
          b = col_max4(b);
          const bool go = b > th && t < N;
          if (__ballot(go) == 0) break;
          uint32_t row = 255;
#pragma unroll
          for (int i = 7; i >= 0; --i)
#pragma unroll
            for (int r = 3; r >= 0; --r) row = z[i][r] == b ? uint32_t(i * 16 + 4 * g + r) : row;
          row = min4(row);
          const int mine = int(row) - 4 * g;         // the lane's register of that row
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) z[i][r] = mine == i * 16 + r ? -INFINITY : z[i][r];
          if (g == 0 && t < N) {
            out.cv[list + n * out.ck] = go ? b : -INFINITY;
            out.ci[list + n * out.ck] = uint8_t(row);
          }
        }
        if (n < out.kc && g == 0 && t < N) out.cv[list + n * out.ck] = -INFINITY;
      }
    }
  }

  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char* tok) const {
    float mx[8], sm[8], dm[8];
    if (v0 + m0 + kBM <= V) columns<true>(acc, m0, n0, wm, wn, lane, tok, mx, sm, dm);
    else columns<false>(acc, m0, n0, wm, wn, lane, tok, mx, sm, dm);
    float4* buf = reinterpret_cast<float4*>(smem);
    const int g = lane >> 4;
    if (wm == 1 && g == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        buf[wn * 128 + j * 16 + lane] = make_float4(mx[j], sm[j], dm[j], 0.f);
    }
    __syncthreads();
    if (wm == 0 && g == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 o = buf[wn * 128 + j * 16 + lane];
        const float M = fmaxf(mx[j], o.x);
        float S = 0.f, D = 0.f;
        auto add = [&](float m, float s, float d) {
          if (m == -INFINITY) return;
          const float dl = m - M, f = __builtin_amdgcn_exp2f(dl * kLog2e);
          S += s * f;
          D += f * fmaf(dl, s, d);
        };
        add(mx[j], sm[j], dm[j]);
        add(o.x, o.y, o.z);
        const int64_t t = n0 + acc_col(wn, j, lane);
        if (t < N) {
          const int64_t at = ((v0 + m0) / kBM) * out.sp + t * out.st;
          out.part[at] = make_float2(M, S);
          out.pd[at] = D;
        }
      }
    }
  }
};

// ---- epilogue of the 64-row tiles ---------------------------------------------------
// z[e] is the raw logit of row e TPT + q (q = this lane's place among the TPT
// adjacent lanes of token t) of the 64 vocabulary rows from v0; `live` of them exist.
template <int TPT, bool SOFTCAP>
__device__ __forceinline__ void tile_epilogue(float (&z)[64 / TPT], int q, int64_t t, int64_t N,
                                              const int64_t* labels, int64_t v0, int live,
                                              const Warp& warp, const LpOut& out) {
  constexpr int E = 64 / TPT;
  const int64_t list = v0 / 64;
  const bool tok = t < N;
  float x[E];
  float m = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = warp_logit<SOFTCAP>(warp, z[e]);
    if (e * TPT + q < live) m = fmaxf(m, x[e]);
    else z[e] = -INFINITY;
  }
#pragma unroll
  for (int o = TPT / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  float s = 0.f, d = 0.f;
  const float mb = m * kLog2e;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float u = fmaf(x[e], kLog2e, -mb);
    u = (e * TPT + q < live && m != -INFINITY && u != -INFINITY) ? u : -200.f;
    const float p = __builtin_amdgcn_exp2f(u);
    s += p;
    d = fmaf(p, u, d);
  }
  d *= kLn2;
#pragma unroll
  for (int o = TPT / 2; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    d += __shfl_xor(d, o);
  }
  if (tok && q == 0) {
    out.part[list * out.sp + t * out.st] = make_float2(m, s);
    out.pd[list * out.sp + t * out.st] = d;
  }
  if (labels && tok) {
    const int64_t y = labels[t] - v0;
    if (y >= 0 && y < live && int(y) % TPT == q) {
      float val = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) val = int(y) / TPT == e ? x[e] : val;
      out.zt[t] = val;
    }
  }
  if (out.kc == 0) return;
  const int64_t at = list * out.cl + t * out.ct;
  int n = 0;
  for (; n < out.kc; ++n) {
    float b = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) b = fmaxf(b, z[e]);
#pragma unroll
    for (int o = TPT / 2; o > 0; o >>= 1) b = fmaxf(b, __shfl_xor(b, o));
    const bool go = b > -INFINITY && tok;
    if (__ballot(go) == 0) break;
    int row = 255;
#pragma unroll
    for (int e = E - 1; e >= 0; --e) row = z[e] == b ? e * TPT + q : row;
#pragma unroll
    for (int o = TPT / 2; o > 0; o >>= 1) {
      const int other = __shfl_xor(row, o);
      row = other < row ? other : row;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = row == e * TPT + q ? -INFINITY : z[e];
    if (q == 0 && tok) {
      out.cv[at + n * out.ck] = go ? b : -INFINITY;
      out.ci[at + n * out.ck] = uint8_t(row);
    }
  }
  if (n < out.kc && q == 0 && tok) out.cv[at + n * out.ck] = -INFINITY;
}

// ---- few tokens -----------------------------------------------------------------------
// A workgroup: 64 vocabulary rows, 16 NT tokens, the four waves taking every
// fourth 32-k chunk each, so that they read 256 adjacent bytes of a row between
// them. A wave's lane loads 16 bytes of row l % 16 at k = 8 (l / 16): the matrix
// instruction's operand as it is, no LDS. h comes from the caches. The waves'
// partial logits meet in LDS. Rows may start at any element (ANY: 2-byte aligned
// 16-byte loads); the last chunk is read element by element where it would leave
// the row.
template <bool ANY>
__device__ __forceinline__ bf16x8 load_k8(const uint16_t* row, int64_t k, int64_t H) {
  if (k + 8 <= H) {
    if constexpr (ANY) return __builtin_bit_cast(bf16x8, load_raw(row + k));
    else return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(row + k));
  }
  typedef __attribute__((ext_vector_type(8))) uint16_t u16x8;
  u16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = k + e < H ? row[k + e] : uint16_t(0);
  return __builtin_bit_cast(bf16x8, v);
}

template <int NT, bool SOFTCAP, bool ANY>
__global__ __launch_bounds__(256) void k_lp_few(const uint16_t* __restrict__ h,
                                                const uint16_t* __restrict__ W,
                                                const int64_t* __restrict__ labels, int64_t N,
                                                int64_t H, int64_t V, Warp warp, LpOut out) {
  constexpr int U = NT == 1 ? 4 : 2;               // chunks in flight per wave
  constexpr int LD = 68;                           // floats per token of the partial logits
  __shared__ __attribute__((aligned(16))) float zb[4][16 * NT][LD];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t v0 = int64_t(blockIdx.x) * 64;
  const int r = lane & 15, kg = (lane >> 4) * 8;
  const uint16_t* wrow[4];
  const uint16_t* hrow[NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t v = v0 + i * 16 + r;
    wrow[i] = W + (v < V ? v : V - 1) * H;
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int64_t t = i * 16 + r;
    hrow[i] = h + (t < N ? t : N - 1) * H;
  }
  f32x4 acc[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int64_t k0, auto count) {
    constexpr int C = decltype(count)::value;
    bf16x8 a[C][4], b[C][NT];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t k = k0 + c * 128 + kg;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[c][i] = load_k8<ANY>(wrow[i], k, H);
#pragma unroll
      for (int j = 0; j < NT; ++j) b[c][j] = load_k8<ANY>(hrow[j], k, H);
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[c][i], b[c][j], acc[i][j], 0, 0, 0);
  };
  int64_t k = w * 32;
  for (; k + (U - 1) * 128 + 32 <= H; k += U * 128) step(k, std::integral_constant<int, U>{});
  for (; k < H; k += 128) step(k, std::integral_constant<int, 1>{});
  // acc[i][j][e]: row 16 i + 4 (lane / 16) + e, token 16 j + lane % 16
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f32x4*>(&zb[w][j * 16 + r][i * 16 + (lane >> 4) * 4]) = acc[i][j];
  __syncthreads();
  constexpr int TPT = 256 / (16 * NT), E = 64 / TPT;
  const int t = tid / TPT, q = tid % TPT;
  float z[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int row = e * TPT + q;
    z[e] = (zb[0][t][row] + zb[1][t][row]) + (zb[2][t][row] + zb[3][t][row]);
  }
  tile_epilogue<TPT, SOFTCAP>(z, q, t, N, labels, v0, int(V - v0 < 64 ? V - v0 : 64), warp, out);
}

// ---- float32 --------------------------------------------------------------------------
// 64 vocabulary rows x 64 tokens a workgroup, a wave 32 x 32 of it in 2 x 2 blocks
// of v_mfma_f32_16x16x4_f32. Both operands go through LDS in 32-k chunks, the next
// chunk loaded while one is multiplied; a lane reads four k of a row at once and
// feeds them to four instructions (both operands in the same order).
constexpr int kF32Ld = 36;                         // floats per row of a chunk in LDS
constexpr int kZLd = 68;

struct F32Stage {
  float a[64][kF32Ld], b[64][kF32Ld];
};

__device__ __forceinline__ void f32_logits(const float* __restrict__ W,
                                           const float* __restrict__ h, int64_t v0, int64_t V,
                                           int64_t t0, int64_t N, int64_t H, F32Stage& st,
                                           float (*z)[kZLd]) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lr = tid >> 3, lc = (tid & 7) * 4;     // rows lr, lr + 32, column lc of a chunk
  const float* ar[2];
  const float* br[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t v = v0 + lr + 32 * i, t = t0 + lr + 32 * i;
    ar[i] = W + (v < V ? v : V - 1) * H;
    br[i] = h + (t < N ? t : N - 1) * H;
  }
  float ra[2][4], rb[2][4];
  auto load = [&](int64_t k0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      load_chunk(ar[i], k0 + lc, H, ra[i]);
      load_chunk(br[i], k0 + lc, H, rb[i]);
    }
  };
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = (w & 1) * 32, wn = (w >> 1) * 32, r = lane & 15, kg = (lane >> 4) * 4;
  load(0);
  for (int64_t k0 = 0; k0 < H; k0 += 32) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      *reinterpret_cast<f32x4*>(&st.a[lr + 32 * i][lc]) = f32x4{ra[i][0], ra[i][1], ra[i][2], ra[i][3]};
      *reinterpret_cast<f32x4*>(&st.b[lr + 32 * i][lc]) = f32x4{rb[i][0], rb[i][1], rb[i][2], rb[i][3]};
    }
    __syncthreads();
    if (k0 + 32 < H) load(k0 + 32);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      f32x4 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        fa[i] = *reinterpret_cast<const f32x4*>(&st.a[wm + 16 * i + r][p * 16 + kg]);
        fb[i] = *reinterpret_cast<const f32x4*>(&st.b[wn + 16 * i + r][p * 16 + kg]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i][e], fb[j][e], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<f32x4*>(&z[wn + 16 * j + r][wm + 16 * i + kg]) = acc[i][j];
  __syncthreads();
}

template <bool SOFTCAP>
__global__ __launch_bounds__(256) void k_lp_f32(const float* __restrict__ h,
                                                const float* __restrict__ W,
                                                const int64_t* __restrict__ labels, int64_t N,
                                                int64_t H, int64_t V, Warp warp, LpOut out) {
  __shared__ __attribute__((aligned(16))) F32Stage st;
  __shared__ __attribute__((aligned(16))) float z[64][kZLd];
  const int64_t v0 = int64_t(blockIdx.x) * 64, t0 = int64_t(blockIdx.y) * 64;
  f32_logits(W, h, v0, V, t0, N, H, st, z);
  const int tl = threadIdx.x >> 2, q = threadIdx.x & 3;
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) v[e] = z[tl][e * 4 + q];
  tile_epilogue<4, SOFTCAP>(v, q, t0 + tl, N, labels, v0, int(V - v0 < 64 ? V - v0 : 64), warp,
                            out);
}

// ---- the joins --------------------------------------------------------------------------
struct JoinArgs {
  LpOut in;
  int64_t parts, lists, list_rows, V;
  int64_t N;                  // tokens of this chunk
  const int64_t* count;       // live ones among them (gathered order); null: N
  const int32_t* idx;         // their positions; null: t
  const int64_t* labels;      // in this order; null: no given tokens
  int64_t ignore_index;
  int top_k;
  Warp warp;
  float* logp;
  float* entropy;
  float* lse;
  float* top_logp;
  int64_t* top_ids;
};

// Token t's scalars at its position o, from M, S, D.
__device__ __forceinline__ void write_token(const JoinArgs& a, int64_t t, int64_t o, bool live,
                                            float M, float S, float D) {
  const float ls = logf(S);
  if (a.lse) a.lse[o] = live ? M + ls : 0.f;
  if (a.entropy) a.entropy[o] = live ? ls - D / S : 0.f;
  if (a.labels) {
    const int64_t y = a.labels[t];
    a.logp[o] = !live ? 0.f : (y < 0 || y >= a.V) ? NAN : (a.in.zt[t] - M) - ls;
  }
}
__device__ __forceinline__ void write_alternative(const JoinArgs& a, int64_t o, int k, float x,
                                                  int64_t id, float M, float ls) {
  a.top_logp[o * a.top_k + k] = id >= 0 ? (x - M) - ls : -INFINITY;
  a.top_ids[o * a.top_k + k] = id;
}

// (m, s, d) joined into (M, S, D).
__device__ __forceinline__ void join_part(float& M, float& S, float& D, float m, float s, float d) {
  if (m == -INFINITY && s == 0.f) return;
  const float Mn = fmaxf(M, m);
  const float a = M == -INFINITY ? 0.f : exp2f((M - Mn) * kLog2e);
  const float b = exp2f((m - Mn) * kLog2e);
  D = (M == -INFINITY ? 0.f : a * fmaf(M - Mn, S, D)) + b * fmaf(m - Mn, s, d);
  S = (M == -INFINITY ? 0.f : S * a) + s * b;
  M = Mn;
}

// Many tokens: 32 tokens a workgroup, 8 threads each taking every 8th part and list
// of its token, then the eight in order. A thread's sorted candidates live in LDS.
constexpr int kJoinTokens = 32;

template <bool SOFTCAP, bool TAU_ONLY, int KM>     // top_k <= KM
__global__ __launch_bounds__(256) void k_lp_join(JoinArgs a, float* __restrict__ tau) {
  __shared__ float lv[KM * 256];                   // [top_k][256]
  __shared__ int32_t li[KM * 256];
  __shared__ float4 grp[8][kJoinTokens];
  __shared__ int cnt[256];
  const int tid = threadIdx.x, tk = tid % kJoinTokens, g = tid / kJoinTokens;
  const int64_t t = int64_t(blockIdx.x) * kJoinTokens + tk;
  int64_t n_live = a.N;
  if (a.count) { const int64_t c = *a.count; n_live = c < n_live ? c : n_live; }
  const bool live = t < n_live;
  const int K = a.top_k;
  float M = -INFINITY, S = 0.f, D = 0.f;
  if (!TAU_ONLY && live) {
    for (int64_t p = g; p < a.parts; p += 8) {
      const int64_t at = p * a.in.sp + t * a.in.st;
      const float2 ms = a.in.part[at];
      join_part(M, S, D, ms.x, ms.y, a.in.pd[at]);
    }
  }
  int n = 0;
  // v behind n sorted candidates of this thread, at its place; the last drops out
  auto insert = [&](float v, int32_t id) {
    auto after = [&](int k) {                      // candidate k ranks behind (v, id)
      const float o = lv[k * 256 + tid];
      return o < v || (o == v && li[k * 256 + tid] > id);
    };
    if (n == K) {
      if (!after(K - 1)) return false;
      --n;
    }
    int k = n;
    while (k > 0 && after(k - 1)) {
      lv[k * 256 + tid] = lv[(k - 1) * 256 + tid];
      li[k * 256 + tid] = li[(k - 1) * 256 + tid];
      --k;
    }
    lv[k * 256 + tid] = v;
    li[k * 256 + tid] = id;
    ++n;
    return true;
  };
  if (K > 0) {
    if (live) {
      for (int64_t l = g; l < a.lists; l += 8) {
        const int64_t at = l * a.in.cl + t * a.in.ct;
        for (int k = 0; k < a.in.kc; ++k) {
          const float v = a.in.cv[at + k * a.in.ck];
          if (!(v > -INFINITY)) break;
          if (!insert(v, int32_t(l * a.list_rows + a.in.ci[at + k * a.in.ck]))) break;
        }
      }
    }
    for (int half = 4; half > 0; half >>= 1) {
      cnt[tid] = n;
      __syncthreads();
      if (g < half) {
        const int o = tid + half * kJoinTokens;
        for (int k = 0; k < cnt[o]; ++k)
          if (!insert(lv[k * 256 + o], li[k * 256 + o])) break;
      }
      __syncthreads();
    }
    if (TAU_ONLY) {
      if (g == 0 && t < a.N) tau[t] = (live && n == K) ? lv[(K - 1) * 256 + tid] : -INFINITY;
      return;
    }
  }
  grp[g][tk] = make_float4(M, S, D, 0.f);
  __syncthreads();
  if (g == 0 && t < a.N) {
    M = -INFINITY; S = 0.f; D = 0.f;
    for (int i = 0; i < 8; ++i) join_part(M, S, D, grp[i][tk].x, grp[i][tk].y, grp[i][tk].z);
    const int64_t o = a.idx ? int64_t(a.idx[t]) : t;
    const bool shown = live && (!a.labels || a.labels[t] != a.ignore_index);
    write_token(a, t, o, shown, M, S, D);
    const float ls = logf(S);
    for (int k = 0; k < K; ++k) {
      const bool has = shown && k < n;
      write_alternative(a, o, k, has ? warp_logit<SOFTCAP>(a.warp, lv[k * 256 + tid]) : 0.f,
                        has ? int64_t(li[k * 256 + tid]) : -1, M, ls);
    }
  }
}

// Few tokens: a workgroup joins one token. Every thread holds the heads of up to
// LPT sorted lists as 64-bit keys (the logit's order, then the lower id first);
// each round takes the workgroup's largest and moves that list on.
constexpr int kFewThreads = 1024;

__device__ __forceinline__ uint64_t rank_key(float v, int64_t id) {
  if (!(v > -INFINITY)) return 0;                  // none
  const uint32_t b = __float_as_uint(v + 0.f);     // -0 ranks as 0
  const uint32_t o = (b >> 31) ? ~b : b | 0x80000000u;
  return (uint64_t(o) << 32) | uint32_t(~uint32_t(id));
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = uint32_t(k >> 32);
  return __uint_as_float((o >> 31) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <bool SOFTCAP, int LPT>
__global__ __launch_bounds__(kFewThreads) void k_lp_join_few(JoinArgs a) {
  constexpr int kWaves = kFewThreads / 64;
  __shared__ float red[3][kWaves];
  __shared__ uint64_t best[2][kWaves];
  __shared__ uint64_t won[kLpTop];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x;
  const bool live = !a.labels || a.labels[t] != a.ignore_index;
  const float2* part = a.in.part + t * a.in.st;
  const float* pd = a.in.pd + t * a.in.st;
  float M = -INFINITY, S = 0.f, D = 0.f;
  for (int64_t p = tid; p < a.parts; p += kFewThreads)
    join_part(M, S, D, part[p].x, part[p].y, pd[p]);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1)
    join_part(M, S, D, __shfl_xor(M, o), __shfl_xor(S, o), __shfl_xor(D, o));
  if (lane == 0) { red[0][w] = M; red[1][w] = S; red[2][w] = D; }
  // heads of the lists
  uint64_t head[LPT];
  int pos[LPT];
  const float* cv = a.in.cv + t * a.in.ct;
  const uint8_t* ci = a.in.ci + t * a.in.ct;
  auto key_of = [&](int j, int k) -> uint64_t {
    const int64_t l = tid + int64_t(j) * kFewThreads;
    if (k >= a.in.kc || l >= a.lists) return 0;
    const int64_t at = l * a.in.cl + k * a.in.ck;
    return rank_key(cv[at], l * a.list_rows + ci[at]);
  };
  if (a.top_k > 0) {
#pragma unroll
    for (int j = 0; j < LPT; ++j) { head[j] = key_of(j, 0); pos[j] = 0; }
    for (int k = 0; k < a.top_k; ++k) {
      uint64_t b = 0;
#pragma unroll
      for (int j = 0; j < LPT; ++j) b = max_u64(b, head[j]);
      uint64_t m = b;
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) m = max_u64(m, __shfl_xor(m, o));
      if (lane == 0) best[k & 1][w] = m;
      __syncthreads();
      m = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) m = max_u64(m, best[k & 1][i]);
      if (tid == 0) won[k] = m;
      if (b == m && m != 0) {                      // keys are distinct: one thread
#pragma unroll
        for (int j = 0; j < LPT; ++j)
          if (head[j] == m) head[j] = key_of(j, ++pos[j]);
      }
    }
  }
  __syncthreads();
  M = -INFINITY; S = 0.f; D = 0.f;
  for (int i = 0; i < kWaves; ++i) join_part(M, S, D, red[0][i], red[1][i], red[2][i]);
  if (tid == 0) write_token(a, t, t, live, M, S, D);
  if (tid < a.top_k) {
    const uint64_t m = won[tid];
    const bool has = live && m != 0;
    write_alternative(a, t, tid, has ? warp_logit<SOFTCAP>(a.warp, key_value(m)) : 0.f,
                      has ? int64_t(uint32_t(~uint32_t(m))) : -1, M, logf(S));
  }
}

// ---- the logit gradient -------------------------------------------------------------------
// With a = dL/dlogp, b = dL/dentropy, l = x - lse and p = exp(l):
//   dL/dx_v = a [v = y] - p (a + b (l + entropy))
// so G = (ca [v = y] + p (c0 + c1 l)) dx/dz with ca = a, c0 = -(a + b entropy),
// c1 = -b, formed once per live token in the gathered order. A token outside the
// vocabulary gets NaN: its gradients fail closed, as the head's loss does.
__global__ __launch_bounds__(256) void k_lp_coef(
    const int32_t* __restrict__ idx, const int64_t* __restrict__ labels,
    const int64_t* __restrict__ count, int64_t N, int64_t V, int64_t ignore_index,
    const float* __restrict__ lse, const float* __restrict__ ent, const float* __restrict__ ga,
    const float* __restrict__ gb, float* __restrict__ lse_g, float* __restrict__ c0,
    float* __restrict__ c1, float* __restrict__ ca) {
  const int64_t r = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (r >= N || (count && r >= *count)) return;
  const int64_t t = idx ? int64_t(idx[r]) : r, y = labels[r];
  float a = ga ? ga[t] : 0.f;
  const float b = gb ? gb[t] : 0.f, s = gb ? ent[t] : 0.f;
  if (y != ignore_index && (y < 0 || y >= V)) a = NAN;
  lse_g[r] = lse[t];
  c0[r] = -(a + b * s);
  c1[r] = -b;
  ca[r] = a;
}

template <bool SOFTCAP, bool SPLIT>
struct EpiLpGrad {
  const int64_t* labels;
  const float* lse;
  const float* c0;
  const float* c1;
  const float* ca;
  int64_t N, V, v0, vcur, gblk;
  Warp warp;
  uint16_t* g;
  int64_t lo_off;             // elements from the hi to the lo chunk (SPLIT)

  static constexpr int kTokBytes = 6144;
  __device__ __forceinline__ void stage(char* tok, int64_t n0, int wave, int lane) const {
    stage_tokens<2>(tok, labels, n0, N, wave, lane);
    stage_tokens<1>(tok + 2048, lse, n0, N, wave, lane);
    stage_tokens<1>(tok + 3072, c0, n0, N, wave, lane);
    stage_tokens<1>(tok + 4096, c1, n0, N, wave, lane);
    stage_tokens<1>(tok + 5120, ca, n0, N, wave, lane);
  }

  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char* tok) const {
    const int64_t* lab = reinterpret_cast<const int64_t*>(tok);
    const float* lse_t = reinterpret_cast<const float*>(tok + 2048);
    const float* c0_t = reinterpret_cast<const float*>(tok + 3072);
    const float* c1_t = reinterpret_cast<const float*>(tok + 4096);
    const float* ca_t = reinterpret_cast<const float*>(tok + 5120);
    const int lg = lane >> 4;
    const int64_t vbase = v0 + m0 + wm * 128;
    float l0[8], k0[8], k1[8];
    TargetPatch tp;
    auto grad = [&](int i, int j, int r) {
      const float z = acc[i][j][r];
      const float l = warp_logit<SOFTCAP>(warp, z) - l0[j];
      return __builtin_amdgcn_exp2f(l * kLog2e) * fmaf(k1[j], l, k0[j]) *
             warp_slope<SOFTCAP>(warp, z);
    };
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int tl = wn * 128 + j * 16 + (lane & 15);
      const bool in = n0 + tl < N;                 // columns past N: exact zeros
      l0[j] = lse_t[tl];
      k0[j] = in ? c0_t[tl] : 0.f;
      k1[j] = in ? c1_t[tl] : 0.f;
      tp.pos[j] = -1;
      tp.val[j] = 0.f;
      const int64_t y = lab[tl];
      if (in && y >= vbase && y < vbase + 128 && y < V) {
        const int d = int(y - vbase);
        if (((d >> 2) & 3) == lg) {
          const int ti = d >> 4, tr = d & 3;
          float z = 0.f, v = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (i == ti && r == tr) { z = acc[i][j][r]; v = grad(i, j, r); }
          tp.pos[j] = target_slot(d, j * 16 + (lane & 15));
          tp.val[j] = fmaf(ca_t[tl], warp_slope<SOFTCAP>(warp, z), v);
        }
      }
    }
    if (!SPLIT) {
      store_token_major<false, true, true>(grad, smem, wm, wn, lane, g, 0, m0, n0, N, vcur, &tp,
                                           gblk);
      return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = grad(i, j, r);
    auto held = [&](int i, int j, int r) { return acc[i][j][r]; };
    store_token_major<false, true, true>(held, smem, wm, wn, lane, g, 0, m0, n0, N, vcur, &tp,
                                         gblk);
    __syncthreads();                               // the staging area is reused
    store_token_major<true, true, true>(held, smem, wm, wn, lane, g + lo_off, 0, m0, n0, N, vcur,
                                        &tp, gblk);
  }
};

// float32: G^T[v - v0][t] of one vocabulary chunk, zero for ignored tokens and for
// the columns N <= t < ldg.
template <bool SOFTCAP>
__global__ __launch_bounds__(256) void k_lp_f32_grad(
    const float* __restrict__ h, const float* __restrict__ W, const int64_t* __restrict__ labels,
    int64_t N, int64_t H, int64_t V, int64_t ignore_index, Warp warp,
    const float* __restrict__ lse, const float* __restrict__ c0, const float* __restrict__ c1,
    const float* __restrict__ ca, int64_t v0, int64_t vcur, int64_t ldg, float* __restrict__ gt) {
  __shared__ __attribute__((aligned(16))) F32Stage st;
  __shared__ __attribute__((aligned(16))) float z[64][kZLd];
  const int64_t m0 = int64_t(blockIdx.x) * 64, t0 = int64_t(blockIdx.y) * 64;
  f32_logits(W + v0 * H, h, m0, vcur, t0, N, H, st, z);
  const int tl = threadIdx.x & 63;
  const int64_t t = t0 + tl;
  if (t >= ldg) return;
  const int64_t y = t < N ? labels[t] : ignore_index;
  const bool live = t < N && y != ignore_index;
  const float l0 = live ? lse[t] : 0.f, k0 = live ? c0[t] : 0.f, k1 = live ? c1[t] : 0.f;
  for (int r = threadIdx.x >> 6; r < 64; r += 4) {
    if (m0 + r >= vcur) break;
    float v = 0.f;
    if (live) {
      const float zz = z[tl][r], l = warp_logit<SOFTCAP>(warp, zz) - l0;
      v = exp2f(l * kLog2e) * fmaf(k1, l, k0);
      if (v0 + m0 + r == y) v += ca[t];
      v *= warp_slope<SOFTCAP>(warp, zz);
    }
    gt[(m0 + r) * ldg + t] = v;
  }
}

unsigned cdiv(int64_t a, int64_t b) { return unsigned((a + b - 1) / b); }

template <bool SOFTCAP>
hipError_t run_join(const LpPlan& q, const JoinArgs& j, const Launcher& L) {
  L.pre(kLpJoin);
  if (q.sp == 1) {
    const dim3 grid(unsigned(j.N)), block(kFewThreads);
    const int64_t lpt = (q.lists + kFewThreads - 1) / kFewThreads;
    if (lpt <= 1) hipLaunchKernelGGL((k_lp_join_few<SOFTCAP, 1>), grid, block, 0, L.stream, j);
    else if (lpt <= 2) hipLaunchKernelGGL((k_lp_join_few<SOFTCAP, 2>), grid, block, 0, L.stream, j);
    else if (lpt <= 4) hipLaunchKernelGGL((k_lp_join_few<SOFTCAP, 4>), grid, block, 0, L.stream, j);
    else hipLaunchKernelGGL((k_lp_join_few<SOFTCAP, 8>), grid, block, 0, L.stream, j);
  } else {
    const dim3 grid(cdiv(j.N, kJoinTokens)), block(256);
    if (j.top_k <= 1)
      hipLaunchKernelGGL((k_lp_join<SOFTCAP, false, 1>), grid, block, 0, L.stream, j, nullptr);
    else if (j.top_k <= 8)
      hipLaunchKernelGGL((k_lp_join<SOFTCAP, false, 8>), grid, block, 0, L.stream, j, nullptr);
    else
      hipLaunchKernelGGL((k_lp_join<SOFTCAP, false, kLpTop>), grid, block, 0, L.stream, j, nullptr);
  }
  L.post(kLpJoin);
  return hipGetLastError();
}

template <bool SOFTCAP>
hipError_t run_few(const LpArgs& a, const Warp& warp, const LpOut& out, const Launcher& L) {
  const auto* h = static_cast<const uint16_t*>(a.h);
  const auto* W = static_cast<const uint16_t*>(a.W);
  const dim3 grid(cdiv(a.V, kLpRows));
  auto go = [&](auto nt) {
    constexpr int NT = decltype(nt)::value;
    if (a.H % 8 == 0)
      hipLaunchKernelGGL((k_lp_few<NT, SOFTCAP, false>), grid, dim3(256), 0, L.stream, h, W,
                         a.tokens, a.N, a.H, a.V, warp, out);
    else
      hipLaunchKernelGGL((k_lp_few<NT, SOFTCAP, true>), grid, dim3(256), 0, L.stream, h, W,
                         a.tokens, a.N, a.H, a.V, warp, out);
  };
  L.pre(kLpTiles);
  if (a.N <= 16) go(std::integral_constant<int, 1>{});
  else if (a.N <= 32) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 4>{});
  L.post(kLpTiles);
  return hipGetLastError();
}

template <bool SOFTCAP>
hipError_t logprobs(const LpPlan& q, const LpArgs& a, char* ws, const Launcher& L) {
  const Warp warp = make_warp(a.softcap, a.temperature);
  LpOut out{reinterpret_cast<float2*>(ws + q.off_part), reinterpret_cast<float*>(ws + q.off_pd),
            reinterpret_cast<float*>(ws + q.off_zt), reinterpret_cast<float*>(ws + q.off_cv),
            reinterpret_cast<uint8_t*>(ws + q.off_ci), q.sp, q.st, q.cl, q.ck, q.ct, int(q.kc)};
  JoinArgs j{out, q.parts, q.lists, q.list_rows, a.V, a.N, nullptr, nullptr, a.tokens,
             a.ignore_index, q.top_k, warp, a.logp, a.entropy, a.lse, a.top_logp, a.top_ids};
  hipError_t e = hipSuccess;
  if (a.dtype == FLCE_F32 || q.few) {
    if (a.status)
      e = a.tokens ? launch_token_status(a.tokens, a.N, a.V, a.ignore_index, a.status, L)
                   : launch_token_status(nullptr, 0, a.V, a.ignore_index, a.status, L);
    if (e != hipSuccess) return e;
  }
  if (q.few) {
    e = run_few<SOFTCAP>(a, warp, out, L);
    return e == hipSuccess ? run_join<SOFTCAP>(q, j, L) : e;
  }
  // the outputs of a chunk of tokens in their own order start at its first token
  auto at_token = [&](JoinArgs& c, int64_t t0) {
    if (a.tokens) c.labels = a.tokens + t0, c.logp = a.logp + t0;
    if (a.entropy) c.entropy = a.entropy + t0;
    if (a.lse) c.lse = a.lse + t0;
    if (q.top_k) c.top_logp = a.top_logp + t0 * q.top_k, c.top_ids = a.top_ids + t0 * q.top_k;
  };
  if (a.dtype == FLCE_F32) {
    for (int64_t t0 = 0; e == hipSuccess && t0 < a.N; t0 += q.nc) {
      JoinArgs c = j;
      at_token(c, t0);
      c.N = a.N - t0 < q.nc ? a.N - t0 : q.nc;
      L.pre(kLpTiles);
      hipLaunchKernelGGL(k_lp_f32<SOFTCAP>, dim3(cdiv(a.V, 64), cdiv(c.N, 64)), dim3(256), 0,
                         L.stream, static_cast<const float*>(a.h) + t0 * a.H,
                         static_cast<const float*>(a.W), c.labels, c.N, a.H, a.V, warp, out);
      L.post(kLpTiles);
      e = hipGetLastError();
      if (e == hipSuccess) e = run_join<SOFTCAP>(q, c, L);
    }
    return e;
  }
  // bf16 tiles
  Plan p = q.p;
  p.nc = q.nc;
  p.n_tok_chunks = q.n_chunks;
  Args ag{};
  ag.h = a.h; ag.W = a.W; ag.labels = a.tokens;
  ag.N = a.N; ag.H = p.H; ag.V = a.V;
  ag.ignore_index = a.ignore_index;
  ag.status = a.status;
  ag.mb_scale = 1.f;
  ag.sc = reinterpret_cast<Scalars*>(ws + q.off_sc);
  ag.num_tokens = reinterpret_cast<int64_t*>(ws + q.off_nt);
  ag.tok_loss = reinterpret_cast<double*>(ws + q.off_tokloss);
  ag.idx = reinterpret_cast<int32_t*>(ws + q.off_idx);
  ag.yc = reinterpret_cast<int64_t*>(ws + q.off_yc);
  ag.bcnt = reinterpret_cast<int32_t*>(ws + q.off_bcnt);
  ag.ccnt = reinterpret_cast<int64_t*>(ws + q.off_ccnt);
  ag.hc = ws + q.off_h;
  if (p.pad_h) {
    void* wp = ws + q.off_wp;
    e = launch_copy_rows(a.W, p.h_in, wp, p.H, p.V, p.h_in, p.H, 2, L);
    ag.W = wp;
    if (e == hipSuccess && !q.gather) {
      e = launch_copy_rows(a.h, p.h_in, ag.hc, p.H, p.N, p.h_in, p.H, 2, L);
      ag.h = ag.hc;
    }
  }
  if (e == hipSuccess && q.gather) e = launch_scan_gather(p, ag, false, L);
  if (e == hipSuccess && q.gather) e = launch_chunk_counts(p, ag, false, L);
  if (e == hipSuccess && !q.gather && a.status)
    e = launch_token_status(nullptr, 0, a.V, a.ignore_index, a.status, L);
  constexpr int NF = gemm::kFormN;
  for (int64_t c = 0; e == hipSuccess && c < q.n_chunks; ++c) {
    const int64_t t0 = c * q.nc;
    JoinArgs jc = j;
    jc.N = a.N - t0 < q.nc ? a.N - t0 : q.nc;
    if (q.gather) {
      jc.labels = ag.yc + t0;
      jc.idx = ag.idx + t0;
      jc.count = ag.ccnt + c;
    } else {
      at_token(jc, t0);
    }
    // vocabulary rows [v0, v1) of the chunk's live tokens
    auto tiles = [&](int64_t v0, int64_t v1, const float* tau) {
      gemm::Launch l = gemm::forward_launch(p);
      l.M = l.a.rows = v1 - v0;
      l.off_a = v0 * p.H;
      l.Nn = l.b.rows = jc.N;
      l.off_b = t0 * p.H;
      auto run = [&](auto epi) {
        return q.gather ? run_gemm<NF, NF, kDynN>(l, ag, epi, kLpTiles, L, jc.count)
                        : run_gemm<NF, NF>(l, ag, epi, kLpTiles, L);
      };
      if (q.top_k > 0)
        return run(EpiLp<SOFTCAP, true>{jc.labels, jc.N, a.V, v0, warp, out, tau});
      return run(EpiLp<SOFTCAP, false>{jc.labels, jc.N, a.V, v0, warp, out, nullptr});
    };
    e = tiles(0, a.V, nullptr);
    if (e == hipSuccess) e = run_join<SOFTCAP>(q, jc, L);
  }
  return e;
}

}  // namespace

hipError_t launch_logprobs(const LpPlan& q, const LpArgs& a, char* ws, const Launcher& L) {
  return a.softcap > 0.f ? logprobs<true>(q, a, ws, L) : logprobs<false>(q, a, ws, L);
}

hipError_t launch_lp_coefficients(const Plan& p, const Args& a, const LpGradArgs& g,
                                  const Launcher& L) {
  L.pre(kLpJoin);
  hipLaunchKernelGGL(k_lp_coef, dim3(cdiv(p.N, 256)), dim3(256), 0, L.stream,
                     p.compact ? a.idx : nullptr, p.compact ? a.yc : a.labels,
                     p.compact ? &a.sc->n_valid : nullptr, p.N, p.V, a.ignore_index, g.lse,
                     g.entropy, g.grad_logp, g.grad_entropy, g.lse_g, g.c0, g.c1, g.ca);
  L.post(kLpJoin);
  return hipGetLastError();
}

hipError_t launch_lp_gradient(const Plan& p, const Args& a, const LpGradArgs& g, int64_t chunk,
                              const Launcher& L) {
  const int64_t v0 = chunk * p.vchunk, vcur = gemm::chunk_rows(p, chunk);
  const Warp warp = make_warp(a.softcap, g.temperature);
  if (p.dtype == FLCE_F32) {
    auto run = [&](auto cap) {
      hipLaunchKernelGGL(k_lp_f32_grad<decltype(cap)::value>, dim3(cdiv(vcur, 64), cdiv(p.ldg, 64)),
                         dim3(256), 0, L.stream, static_cast<const float*>(a.h),
                         static_cast<const float*>(a.W), a.labels, p.N, p.H, p.V, a.ignore_index,
                         warp, g.lse_g, g.c0, g.c1, g.ca, v0, vcur, p.ldg,
                         static_cast<float*>(a.g));
    };
    L.pre(kGradLogits);
    a.softcap > 0.f ? run(std::true_type{}) : run(std::false_type{});
    L.post(kGradLogits);
    return hipGetLastError();
  }
  if (!p.compact) return hipErrorInvalidValue;
  constexpr int NF = gemm::kFormN;
  const gemm::Launch l = gemm::backward_launch(p, chunk, 0);
  auto run = [&](auto cap, auto split) {
    const EpiLpGrad<decltype(cap)::value, decltype(split)::value> epi{
        a.yc, g.lse_g, g.c0, g.c1, g.ca, p.N, p.V, v0, vcur, gemm::g_block(p), warp,
        static_cast<uint16_t*>(a.g), p.vchunk * p.ldg};
    return run_gemm<NF, NF, kDynN>(l, a, epi, kGradLogits, L, &a.sc->n_valid);
  };
  using Y = std::true_type;
  using No = std::false_type;
  if (p.g_parts == 2) return a.softcap > 0.f ? run(Y{}, Y{}) : run(No{}, Y{});
  return a.softcap > 0.f ? run(Y{}, No{}) : run(No{}, No{});
}

}  // namespace flce
