// Log probabilities of given tokens, entropy and top alternatives over the head's
// logits, and the logit gradient of the first two.
//
// With z = h W^T, x = softcap(z) / temperature, one pass over the vocabulary
// keeps per tile and token
//   m = max x,  s = sum exp(x - m),  d = sum exp(x - m) (x - m)
// which join over tiles by rescaling to the larger max:
//   s' = s exp(m - M),  d' = exp(m - M) (d + (m - M) s)
// so that  lse = M + log S,  log p_y = (x_y - M) - log S,  entropy = log S - D / S.
// The exponents are formed from the difference x - m, so the largest term is exactly 1,
// S >= 1 and no log probability is above 0; log S is taken apart from M, so a token that
// holds nearly all of the probability keeps its small one to some 2^-24, wherever its
// logit lies. Alternatives are ranked by the raw logit z (the
// order of x, without the ties that rounding x makes), equal ones by lowest id.
//
// Three kernels compute logits:
//  - the 256 x 256 bf16 tiles of the head's own forward (gemm_bf16.h), live tokens
//    gathered first: bound by the matrix cores;
//  - few bf16 tokens: 64 or 128 vocabulary rows a workgroup, W streamed from memory
//    straight into the matrix cores' operand registers: bound by reading W once;
//  - float32: 64 x 64 tiles on the float32 matrix instruction.
// The 256 x 256 tiles never store a logit; each leaves its top_k largest logits
// that could still be listed, and the join selects from those lists. The other two
// store the logits of their tokens (N V 4 bytes, for few tokens next to the V H 2 of W)
// and the largest of each 64 vocabulary rows; the join then looks only into the top_k
// of those parts with the largest, which hold all top_k alternatives.
//
// Measured: 6144 live rows of 4096 over 131072 with 8 alternatives 4.97 ms in the tiles
// (1326 TFLOP/s; 3687 rows without alternatives 2.85 ms, 1390 TFLOP/s); one row over
// the same table 196 us (5.5 TB/s); float32 512 rows of 1024 over 32000 303 us (111
// TFLOP/s, where the library's product of that type reaches 138).
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/flce.h"
#include "flce_internal.h"
#include "gemm_bf16.h"
#include "join_sparse.h"
#include "ops_plan.h"
#include "row_io.h"
#include "wave_ops.h"

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
// a - b of the two rounded values. Contracted with the product that made a, it would be
// what rounding a left and not 0 where they are equal.
__device__ __forceinline__ float minus(float a, float b) {
#pragma clang fp contract(off)
  return a - b;
}
// How far the max of a part lies below another one, m - M. Held above -1e30, where the
// part's factor exp(m - M) is 0 and the factor of its weighted sum still finite: the
// difference of two logits may leave float32's range.
__device__ __forceinline__ float below(float m, float M) { return fmaxf(minus(m, M), -1e30f); }
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
  float* cv;                  // 256 x 256 tiles: candidates, -inf behind the last,
  uint8_t* ci;                //   and their rows within the list
  float* zmax;                // parts of 64 rows: the largest raw logit
  float* z;                   //   and all of them, [token][vocabulary]; null: not wanted
  int64_t sp, st, cl, ck, ct;
  int kc, top_k;
};

// x summed over the lanes of this column with a smaller g (lane / 16).
__device__ __forceinline__ int before_rows(int x, int g) {
  int at = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_permlane16_swap(uint32_t(x), uint32_t(x), false, false);
  const uint32_t pair = a[0] + a[1];
  const auto b = __builtin_amdgcn_permlane32_swap(pair, pair, false, false);
  at = int(((g & 1) ? a[0] : 0u) + ((g & 2) ? b[0] : 0u));
#endif
  return at;
}

// ---- epilogue of the 256 x 256 tiles ----------------------------------------------
// The accumulators are raw logits, tile rows vocabulary ids, columns tokens (see
// EpiLse for the layout). The two waves of a column join their (m, s, d) through
// LDS; each wave leaves candidates of its own 128 rows. A candidate has to exceed
// tau, the token's top_k-th largest logit among lower ids: an equal one with a higher
// id could not be listed either. Few do, so the wave counts them and stores them in
// any order. Without a tau yet, or with more of them than the list holds, it looks for
// a bound that top_k to kc exceed (top_k > 8). Where that fails (equal logits at the
// bound) or does not pay, the column's top_k largest are taken in rounds: the largest
// logit left, lowest row first, in the four lanes that hold the column; a wave stops
// when none of its 16 columns has one.
template <bool SOFTCAP, bool TOPK>
struct EpiLp {
  const int64_t* labels;      // null: no given tokens
  int64_t N, V, v0;           // v0: vocabulary id of launch row 0
  Warp warp;
  LpOut out;
  const float* tau;           // TOPK; null: -inf

  static constexpr int kTokBytes = 3 * 1024;
  __device__ __forceinline__ void stage(char* tok, int64_t n0, int wave, int lane) const {
    if (labels) stage_tokens<2>(tok, labels, n0, N, wave, lane);
    if (TOPK && tau) stage_tokens<1>(tok + 2048, tau, n0, N, wave, lane);
  }

  // The accumulators of column block j, as they are.
  __device__ __forceinline__ static void column(const Acc& acc, int j, float (&z)[8][4]) {
    auto take = [&](auto c) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = acc[i][decltype(c)::value][r];
    };
    switch (j) {
      case 0: take(std::integral_constant<int, 0>{}); break;
      case 1: take(std::integral_constant<int, 1>{}); break;
      case 2: take(std::integral_constant<int, 2>{}); break;
      case 3: take(std::integral_constant<int, 3>{}); break;
      case 4: take(std::integral_constant<int, 4>{}); break;
      case 5: take(std::integral_constant<int, 5>{}); break;
      case 6: take(std::integral_constant<int, 6>{}); break;
      default: take(std::integral_constant<int, 7>{}); break;
    }
  }

  // FULL: all 128 rows of the wave exist. `to`: this wave's [256] (m, s, d) in LDS.
  template <bool FULL>
  __device__ __forceinline__ void columns(const Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                          int lane, const char* tok, float4* to) const {
    const int64_t* lab = reinterpret_cast<const int64_t*>(tok);
    const float* tau_t = reinterpret_cast<const float*>(tok + 2048);
    const int g = lane >> 4;
    const int64_t vbase = v0 + m0 + wm * 128;        // vocabulary id of the wave's row 0
    const int live = FULL ? 128 : int(V - vbase < 128 ? (V - vbase > 0 ? V - vbase : 0) : 128);
    auto in = [&](int i, int r) { return FULL || i * 16 + 4 * g + r < live; };
    // one column block at a time through the same code: unrolled over the blocks, the
    // epilogue is several times the instruction cache and waits for its own fetches
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      float z[8][4];
      column(acc, j, z);
      const int col = acc_col(wn, j, lane);
      const int64_t t = n0 + col;
      float x[8][4];
      float mq[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[i][r] = warp_logit<SOFTCAP>(warp, z[i][r]);
          mq[r] = fmaxf(mq[r], in(i, r) ? x[i][r] : -INFINITY);
        }
      if (labels) {
        const int64_t y = t < N ? lab[col] : -1;
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
      // in powers of two: u = (x - m) log2 e, d in units of ln 2. The form
      // x log2 e - (m log2 e) saves an instruction, but its largest term is not 1
      const float mb = m == -INFINITY ? 0.f : m;
      float sq[4] = {0.f, 0.f, 0.f, 0.f}, dq[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // a row past the vocabulary: 2^-200 = 0; a logit of -inf keeps -inf out of d
          float u = minus(x[i][r], mb) * kLog2e;
          u = (in(i, r) && u != -INFINITY) ? u : -200.f;
          const float e = __builtin_amdgcn_exp2f(u);
          sq[r] += e;
          dq[r] = fmaf(e, u, dq[r]);
        }
      const float s = col_sum4((sq[0] + sq[1]) + (sq[2] + sq[3]));
      const float d = col_sum4((dq[0] + dq[1]) + (dq[2] + dq[3]));
      if (g == 0) to[col] = make_float4(m, s, d * kLn2, 0.f);
      if (!TOPK || live == 0) continue;              // rows past V have no list
      float th = tau ? tau_t[col] : -INFINITY;
      const int64_t list = (vbase >> 7) * out.cl + t * out.ct;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) z[i][r] = in(i, r) ? z[i][r] : -INFINITY;
      auto above = [&](float x) {                    // this lane's logits above x
        int c = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) c += z[i][r] > x ? 1 : 0;
        return c;
      };
      int n = 0, own = 0;
      bool rounds = false;
      // x rises with z: no x as large as that of tau, no logit above tau
      if (!tau || SOFTCAP || __ballot(t < N && m >= th * warp.inv_t) != 0) {
        own = above(th);
        n = rows_all(own, AddOp());
        bool fits = n <= out.kc || t >= N;
        rounds = __ballot(!fits) != 0;
        if (rounds && out.top_k > 8) {
          // a bound that top_k to kc logits exceed, by bisection between the column's
          // smallest and largest: a few counts, cheaper than more than 8 rounds (2000
          // rows of 1024 over 32000, 20 alternatives: 54 us less than with a bound
          // that exactly 20 exceed; 300 rows, 4 alternatives: 86 us by rounds, 92 so)
          float lo = INFINITY, hi = -INFINITY;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              hi = fmaxf(hi, z[i][r]);
              lo = fminf(lo, z[i][r] > th ? z[i][r] : INFINITY);
            }
          hi = col_max4(hi);
          lo = -col_max4(-lo);
          // where the bound lies in the range of 128 normal values
          float part = 0.86f - 0.00375f * float(out.top_k + out.kc);
#pragma unroll 1
          for (int it = 0; it < 16 && __ballot(!fits) != 0; ++it) {
            const float mid = fmaf(part, hi - lo, lo);
            part = 0.5f;
            const int c = above(mid), total = rows_all(c, AddOp());
            if (!fits) {
              if (total >= out.top_k && total <= out.kc) { fits = true; th = mid; own = c; n = total; }
              else if (total > out.kc) lo = mid;
              else hi = mid;
            }
          }
          rounds = __ballot(!fits) != 0;
        }
        int at = before_rows(own, g);
        if (!rounds && t < N && own > 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (z[i][r] > th) {
                out.cv[list + at * out.ck] = z[i][r];
                out.ci[list + at * out.ck] = uint8_t(i * 16 + 4 * g + r);
                ++at;
              }
        }
      }
      if (rounds) {
        th = tau ? tau_t[col] : -INFINITY;
#pragma unroll 1
        for (n = 0; n < out.top_k; ++n) {
          float bq[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            bq[r] = z[0][r];
#pragma unroll
            for (int i = 1; i < 8; ++i) bq[r] = fmaxf(bq[r], z[i][r]);
          }
          const float b = col_max4(fmaxf(fmaxf(bq[0], bq[1]), fmaxf(bq[2], bq[3])));
          const bool go = b > th && t < N;
          if (__ballot(go) == 0) break;
          uint32_t rq[4] = {255, 255, 255, 255};
#pragma unroll
          for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int i = 7; i >= 0; --i)
              rq[r] = z[i][r] == b ? uint32_t(i * 16 + 4 * g + r) : rq[r];
          MinOp least;
          const uint32_t row = rows_all(least(least(rq[0], rq[1]), least(rq[2], rq[3])), least);
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
      }
      if (n < out.kc && g == 0 && t < N) out.cv[list + n * out.ck] = -INFINITY;
    }
  }

  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char* tok) const {
    float4* buf = reinterpret_cast<float4*>(smem);   // [2][256]
    if (v0 + m0 + kBM <= V) columns<true>(acc, m0, n0, wm, wn, lane, tok, buf + wm * 256);
    else columns<false>(acc, m0, n0, wm, wn, lane, tok, buf + wm * 256);
    __syncthreads();
    // a token a thread: the two waves' rows joined
    const int col = (wm + 2 * wn) * 64 + lane;
    const int64_t t = n0 + col;
    if (t >= N) return;
    const float4 a = buf[col], b = buf[256 + col];
    const float M = fmaxf(a.x, b.x);
    float S = 0.f, D = 0.f;
    auto add = [&](const float4& q) {
      // nothing from so far below, also where the difference leaves float32's range; NaN stays
      const float dl = q.x == M ? 0.f : q.x - M;
      if (dl < -1e30f && q.y == q.y) return;
      const float f = __builtin_amdgcn_exp2f(dl * kLog2e);
      S += q.y * f;
      D += f * fmaf(dl, q.y, q.z);
    };
    add(a);
    add(b);
    const int64_t at = ((v0 + m0) / kBM) * out.sp + t * out.st;
    out.part[at] = make_float2(M, S);
    out.pd[at] = D;
  }
};

// ---- epilogue of parts of 64 rows ---------------------------------------------------
// z[e] is the raw logit of row q E + e (q = this lane's place among the TPT adjacent
// lanes of token t, E = 64 / TPT) of the 64 vocabulary rows from v0; `live` exist.
template <int TPT, bool SOFTCAP>
__device__ __forceinline__ void tile_epilogue(const float (&z)[64 / TPT], int q, int64_t t,
                                              int64_t N, const int64_t* labels, int64_t v0,
                                              int live, int64_t V, const Warp& warp,
                                              const LpOut& out) {
  constexpr int E = 64 / TPT;
  const bool tok = t < N;
  const int n = live - q * E;                      // rows of this lane that exist
  float x[E];
  float m = -INFINITY, zm = -INFINITY;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    x[e] = warp_logit<SOFTCAP>(warp, z[e]);
    m = fmaxf(m, e < n ? x[e] : -INFINITY);
    zm = fmaxf(zm, e < n ? z[e] : -INFINITY);
  }
  m = group_all<TPT>(m, MaxOp());
  // 16 groups of four rows, each in order, then a tree over the groups: whichever lanes
  // hold them, the same order of additions, so that a token's sums do not depend on how
  // many others the call has
  constexpr int Q = E / 4;
  float sq[Q] = {}, dq[Q] = {};
  // no largest logit: all are -inf (their u too) or NaN, which the sums keep
  const float mb = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float u = minus(x[e], mb) * kLog2e;
    u = (e < n && u != -INFINITY) ? u : -200.f;
    const float p = __builtin_amdgcn_exp2f(u);
    sq[e / 4] += p;
    dq[e / 4] = fmaf(p, u, dq[e / 4]);
  }
#pragma unroll
  for (int w = 1; w < Q; w *= 2)
#pragma unroll
    for (int i = 0; i < Q; i += 2 * w) {
      sq[i] += sq[i + w];
      dq[i] += dq[i + w];
    }
  const float s = group_all<TPT>(sq[0], AddOp());
  const float d = group_all<TPT>(dq[0], AddOp()) * kLn2;
  const int64_t at = (v0 / 64) * out.sp + t * out.st;
  if (tok && q == 0) {
    out.part[at] = make_float2(m, s);
    out.pd[at] = d;
  }
  if (labels && tok) {
    const int64_t y = labels[t] - v0;
    if (y >= 0 && y < live && int(y) / E == q) {
      float val = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) val = int(y) % E == e ? x[e] : val;
      out.zt[t] = val;
    }
  }
  if (!out.z) return;
  zm = group_all<TPT>(zm, MaxOp());
  if (!tok) return;
  if (q == 0) out.zmax[at] = zm;
  float* row = out.z + t * V + v0 + q * E;
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    if (e + 4 <= n) {
      const float f[4] = {z[e], z[e + 1], z[e + 2], z[e + 3]};
      store_chunk(row, e, int64_t(e + 4), f);
    } else {
#pragma unroll
      for (int i = e; i < e + 4; ++i)
        if (i < n) row[i] = z[i];
    }
  }
}

// ---- few tokens -----------------------------------------------------------------------
// A workgroup: 64 RB vocabulary rows, 16 RB of them a wave, and 16 NT tokens. A lane
// loads 16 bytes of W's row l % 16 at k = 8 (l / 16): the matrix instruction's operand
// as it is, no LDS. The h of a 128-k chunk is shared by the waves through LDS, two
// chunks in turn. Both come kAheadK chunks early, so that several KiB of W per wave
// are under way all the time. The loads of whole chunks have no condition (past the
// last one it is loaded again): a branch around a load makes the compiler wait for
// it as if the other way had been taken. The part of a chunk at the end of a row that
// is no multiple of 128 is read first, element by element where it leaves the row.
//
// Bound by reading W. Every workgroup reads all of h from L2 as well, so more than 32
// tokens take two row blocks a wave (us with one and two, W of 131072 x 4096: 1 token
// 211 and 226, 32 tokens 224 and 233, 64 tokens 254 and 241, 128 tokens 296 and 262;
// 48 tokens, 256000 x 3584: 451 and 411). Non-temporal loads of W are slower (48
// tokens: 533): the two halves of a 128-byte line come by two loads.
constexpr int kChunkK = 128;                       // k per chunk: four matrix steps
constexpr int kHld = kChunkK + 8;                  // elements of a token's chunk in LDS

// Eight elements of a row at p. ALIGN: bytes that every row starts at a multiple of:
// 16, 4 or 2. Odd rows of a 2-byte aligned matrix are read as aligned words and
// shifted: the element behind p + 7 is read with them.
template <int ALIGN>
__device__ __forceinline__ bf16x8 load_k8(const uint16_t* p) {
  typedef u32x4 __attribute__((aligned(4))) u32x4_word;
  if constexpr (ALIGN == 16) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4*>(p));
  } else if constexpr (ALIGN == 4) {
    return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4_word*>(p));
  } else {
    const bool odd = (reinterpret_cast<uintptr_t>(p) & 2) != 0;
    const uint16_t* q = odd ? p - 1 : p;
    const u32x4 v = *reinterpret_cast<const u32x4_word*>(q);
    const uint32_t e = *reinterpret_cast<const uint32_t*>(odd ? q + 8 : q + 6);
    const uint32_t sh = odd ? 16 : 0;
    return __builtin_bit_cast(bf16x8, u32x4{__builtin_amdgcn_alignbit(v[1], v[0], sh),
                                            __builtin_amdgcn_alignbit(v[2], v[1], sh),
                                            __builtin_amdgcn_alignbit(v[3], v[2], sh),
                                            __builtin_amdgcn_alignbit(e, v[3], sh)});
  }
}
// The same at k of a row of H elements, zero past it.
template <int ALIGN>
__device__ __forceinline__ bf16x8 load_k8_end(const uint16_t* row, int64_t k, int64_t H) {
  typedef __attribute__((ext_vector_type(8))) uint16_t u16x8;
  if (ALIGN != 2 && k + 8 <= H) return load_k8<ALIGN>(row + k);
  u16x8 v;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = k + e < H ? row[k + e] : uint16_t(0);
  return __builtin_bit_cast(bf16x8, v);
}

template <int NT, int RB>
union FewSmem {
  uint16_t h[2][16 * NT][kHld];
  float z[16 * NT][64 * RB + 4];
};
// Lanes of a token in the epilogues of such a tile (48 tokens: whole waves idle).
template <int NT>
constexpr int kFewLanes = NT == 3 ? 4 : 256 / (16 * NT);

// The tile's logits in sm.z: 64 rows from v0 of the V rows of W, tokens 0 .. N - 1 of h.
template <int NT, int ALIGN, int RB>
__device__ __forceinline__ void few_logits(const uint16_t* __restrict__ h,
                                           const uint16_t* __restrict__ W, int64_t N, int64_t H,
                                           int64_t V, int64_t v0, FewSmem<NT, RB>& sm) {
  constexpr int kAheadK = NT == 8 ? 1 : NT >= 3 ? 2 : 3, R = kAheadK + 1;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int r = lane & 15, kg = (lane >> 4) * 8;
  const uint16_t* wrow[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int64_t v = v0 + i * 64 + w * 16 + r;
    wrow[i] = W + (v < V ? v : V - 1) * H;
  }
  // h: load p of a thread is 16 bytes of token 16 p + tid / 16 at k = 8 (tid % 16)
  const int hr = tid >> 4, hk = (tid & 15) * 8;
  const uint16_t* hrow[NT];
#pragma unroll
  for (int p = 0; p < NT; ++p) hrow[p] = h + (16 * p + hr < N ? 16 * p + hr : N - 1) * H;
  bf16x8 a[R][4][RB], b[R][NT];
  auto load = [&](bf16x8 (&fa)[4][RB], bf16x8 (&fb)[NT], int64_t k0) {
#pragma unroll
    for (int p = 0; p < NT; ++p) fb[p] = load_k8<ALIGN>(hrow[p] + k0 + hk);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) fa[s][i] = load_k8<ALIGN>(wrow[i] + k0 + s * 32 + kg);
  };
  auto keep = [&](const bf16x8 (&fb)[NT], int half) {
#pragma unroll
    for (int p = 0; p < NT; ++p) *reinterpret_cast<bf16x8*>(&sm.h[half][16 * p + hr][hk]) = fb[p];
  };
  f32x4 acc[RB][NT];
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const bf16x8 (&fa)[4][RB], int half) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const bf16x8 f = *reinterpret_cast<const bf16x8*>(&sm.h[half][16 * j + r][s * 32 + kg]);
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[s][i], f, acc[i][j], 0, 0, 0);
      }
  };
  const int64_t full = H / kChunkK, end = full * kChunkK;
  auto chunk_k = [&](int64_t c) { return (c < full ? c : full - 1) * kChunkK; };
  if (end < H) {                                   // the end of the rows
    bf16x8 ea[4][RB], eb[NT];
#pragma unroll
    for (int p = 0; p < NT; ++p) eb[p] = load_k8_end<ALIGN>(hrow[p], end + hk, H);
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int s = 0; s < 4; ++s) ea[s][i] = load_k8_end<ALIGN>(wrow[i], end + s * 32 + kg, H);
    keep(eb, 1);
    __syncthreads();
    multiply(ea, 1);
  }
  if (full > 0) {
#pragma unroll
    for (int u = 0; u < kAheadK; ++u) load(a[u], b[u], chunk_k(u));
    keep(b[0], 0);
    __syncthreads();
    for (int64_t c0 = 0; c0 < full; c0 += R) {
#pragma unroll
      for (int u = 0; u < R; ++u) {
        load(a[(u + kAheadK) % R], b[(u + kAheadK) % R], chunk_k(c0 + u + kAheadK));
        const int half = int(c0 + u) & 1;
        if (c0 + u < full) multiply(a[u], half);
        keep(b[(u + 1) % R], half ^ 1);
        __syncthreads();
      }
    }
  }
  __syncthreads();
  // acc[i][j][e]: row 64 i + 16 w + 4 (lane / 16) + e, token 16 j + lane % 16
#pragma unroll
  for (int i = 0; i < RB; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
      *reinterpret_cast<f32x4*>(&sm.z[16 * j + r][64 * i + 16 * w + (lane >> 4) * 4]) = acc[i][j];
  __syncthreads();
}

template <int NT, bool SOFTCAP, int ALIGN, int RB>
__global__ __launch_bounds__(256) void k_lp_few(const uint16_t* __restrict__ h,
                                                const uint16_t* __restrict__ W,
                                                const int64_t* __restrict__ labels, int64_t N,
                                                int64_t H, int64_t V, Warp warp, LpOut out) {
  __shared__ __attribute__((aligned(16))) FewSmem<NT, RB> sm;
  const int64_t v0 = int64_t(blockIdx.x) * (64 * RB);
  few_logits<NT, ALIGN, RB>(h, W, N, H, V, v0, sm);
  constexpr int TPT = kFewLanes<NT>, E = 64 / TPT;
  const int t = threadIdx.x / TPT, q = threadIdx.x % TPT;
  if (t >= 16 * NT) return;
#pragma unroll 1
  for (int i = 0; i < RB; ++i) {
    const int64_t at = v0 + 64 * i;
    if (at >= V) break;
    float z[E];
#pragma unroll
    for (int e = 0; e < E; ++e) z[e] = sm.z[t][64 * i + q * E + e];
    tile_epilogue<TPT, SOFTCAP>(z, q, t, N, labels, at, int(V - at < 64 ? V - at : 64), V, warp,
                                out);
  }
}

// ---- float32 --------------------------------------------------------------------------
// 64 vocabulary rows x 64 tokens a workgroup, a wave 32 x 32 of it in 2 x 2 blocks
// of v_mfma_f32_16x16x4_f32 (32 tokens: a wave 32 x 16). Both operands go through LDS
// in 32-k chunks, two halves in turn, loaded two chunks early without conditions (see
// the few tokens' loads); a lane reads four k of a row at once and feeds them to four
// instructions (both operands in the same order). Bound by the matrix instruction where
// the tiles fill the chip, otherwise by one tile's latency.
constexpr int kF32Ld = 36;                         // floats per row of a chunk in LDS
constexpr int kZLd = 68;

constexpr int kF32K = 32;                          // k per chunk

template <int TN>
union F32Stage {
  struct { float a[64][kF32Ld], b[TN][kF32Ld]; } half[2];
  float z[TN][kZLd];
};
struct F32Regs {
  float a[2][4], b[2][4];
};

// The chunks of k0 .. k1 - 1: whole(k, r) loads one without conditions, end(k, r) what
// is left behind them, with zeros past k1 (it goes first); keep(r, half) puts it into
// LDS, multiply(half) adds its products. Ends with a barrier.
template <class Whole, class End, class Keep, class Multiply>
__device__ __forceinline__ void f32_chunks(int64_t k0, int64_t k1, Whole whole, End end, Keep keep,
                                           Multiply multiply) {
  const int64_t full = (k1 - k0) / kF32K, rest = k0 + full * kF32K;
  F32Regs r[2];
  if (rest < k1) {
    end(rest, r[0]);
    keep(r[0], 1);
    __syncthreads();
    multiply(1);
  }
  if (full > 0) {
    auto at = [&](int64_t c) { return k0 + (c < full ? c : full - 1) * kF32K; };
    whole(at(0), r[0]);
    whole(at(1), r[1]);
    keep(r[0], 0);
    __syncthreads();
    for (int64_t c0 = 0; c0 < full; c0 += 2) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        whole(at(c0 + u + 2), r[u]);
        if (c0 + u < full) multiply(u);
        keep(r[u ^ 1], u ^ 1);
        __syncthreads();
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ f32x4 as_f32x4(const float (&f)[4]) {
  return f32x4{f[0], f[1], f[2], f[3]};
}

// 64 rows from v0 of the V rows of W x TN rows from t0 of the N rows of h, in st.z.
template <int TN>
__device__ __forceinline__ void f32_logits(const float* __restrict__ W,
                                           const float* __restrict__ h, int64_t v0, int64_t V,
                                           int64_t t0, int64_t N, int64_t H, F32Stage<TN>& st) {
  constexpr int NB = TN / 32;                      // rows of h a thread loads, column blocks a wave
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lr = tid >> 3, lc = (tid & 7) * 4;     // rows lr, lr + 32, column lc of a chunk
  const float* ar[2];
  const float* br[NB];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t v = v0 + lr + 32 * i, t = t0 + lr + 32 * i;
    ar[i] = W + (v < V ? v : V - 1) * H;
    if (i < NB) br[i] = h + (t < N ? t : N - 1) * H;
  }
  f32x4 acc[2][NB];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < NB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = (w & 1) * 32, wn = (w >> 1) * 16 * NB, r = lane & 15, kg = (lane >> 4) * 4;
  f32_chunks(
      0, H,
      [&](int64_t k, F32Regs& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          unpack_chunk<float>(load_raw(ar[i] + k + lc), f.a[i]);
          if (i < NB) unpack_chunk<float>(load_raw(br[i] + k + lc), f.b[i]);
        }
      },
      [&](int64_t k, F32Regs& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          load_chunk(ar[i], k + lc, H, f.a[i]);
          if (i < NB) load_chunk(br[i], k + lc, H, f.b[i]);
        }
      },
      [&](const F32Regs& f, int half) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          *reinterpret_cast<f32x4*>(&st.half[half].a[lr + 32 * i][lc]) = as_f32x4(f.a[i]);
          if (i < NB)
            *reinterpret_cast<f32x4*>(&st.half[half].b[lr + 32 * i][lc]) = as_f32x4(f.b[i]);
        }
      },
      [&](int half) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          f32x4 fa[2], fb[NB];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            fa[i] = *reinterpret_cast<const f32x4*>(&st.half[half].a[wm + 16 * i + r][p * 16 + kg]);
            if (i < NB)
              fb[i] = *reinterpret_cast<const f32x4*>(&st.half[half].b[wn + 16 * i + r][p * 16 + kg]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int j = 0; j < NB; ++j)
                acc[i][j] =
                    __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i][e], fb[j][e], acc[i][j], 0, 0, 0);
        }
      });
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<f32x4*>(&st.z[wn + 16 * j + r][wm + 16 * i + kg]) = acc[i][j];
  __syncthreads();
}

template <int TN, bool SOFTCAP>
__global__ __launch_bounds__(256) void k_lp_f32(const float* __restrict__ h,
                                                const float* __restrict__ W,
                                                const int64_t* __restrict__ labels, int64_t N,
                                                int64_t H, int64_t V, Warp warp, LpOut out) {
  __shared__ __attribute__((aligned(16))) F32Stage<TN> st;
  constexpr int TPT = 256 / TN, E = 64 / TPT;
  const int64_t v0 = int64_t(blockIdx.x) * 64, t0 = int64_t(blockIdx.y) * TN;
  f32_logits<TN>(W, h, v0, V, t0, N, H, st);
  const int tl = threadIdx.x / TPT, q = threadIdx.x % TPT;
  float v[E];
#pragma unroll
  for (int e = 0; e < E; ++e) v[e] = st.z[tl][q * E + e];
  tile_epilogue<TPT, SOFTCAP>(v, q, t0 + tl, N, labels, v0, int(V - v0 < 64 ? V - v0 : 64), V,
                              warp, out);
}

// ---- the joins --------------------------------------------------------------------------
struct JoinArgs {
  LpOut in;
  int64_t parts, list0, lists, list_rows, V;       // lists list0 .. lists - 1
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
  uint64_t* first;            // [top_k][first_ld] keys of the lists before list0, or null
  int64_t first_ld;
  float* tau;
};

// Token t's scalars at its position o, from M, S, D.
__device__ __forceinline__ void write_token(const JoinArgs& a, int64_t t, int64_t o, bool live,
                                            float M, float S, float D) {
  const float ls = logf(S);
  if (a.lse) a.lse[o] = live ? M + ls : 0.f;
  if (a.entropy) a.entropy[o] = live ? ls - D / S : 0.f;
  if (a.labels) {
    const int64_t y = a.labels[t];
    a.logp[o] = !live ? 0.f : (y < 0 || y >= a.V) ? NAN : minus(a.in.zt[t], M) - ls;
  }
}
__device__ __forceinline__ void write_alternative(const JoinArgs& a, int64_t o, int k, float x,
                                                  int64_t id, float M, float ls) {
  a.top_logp[o * a.top_k + k] = id >= 0 ? minus(x, M) - ls : -INFINITY;
  a.top_ids[o * a.top_k + k] = id;
}

// (m, s, d) joined into (M, S, D). A part of NaN logits alone has the max -inf and a sum
// of NaN, which stays.
__device__ __forceinline__ void join_part(float& M, float& S, float& D, float m, float s, float d) {
  if (m == -INFINITY && s == 0.f) return;
  const float Mn = fmaxf(M, m);
  const float da = below(M, Mn), db = below(m, Mn);
  const float a = exp2f(da * kLog2e), b = exp2f(db * kLog2e);
  // spelled out: what is contracted decides the last bit
  D = fmaf(b, fmaf(db, s, d), a * fmaf(da, S, D));
  S = fmaf(s, b, S * a);
  M = Mn;
}

// The joins over tiles of many tokens add a token's parts up in one order, whatever the
// threads they have for it: chain c takes parts c, c + kChains, ... in order, then chain c
// joins chain c + half for half = kChains / 2 ... 1. A token's values are then the same
// bits in calls of any count of tokens (another join, other threads). With chains of as
// many as the threads, one row in forty of 131072 logits got another last bit.
constexpr int kChains = 256;

// Thread g of G: its chains c = g (mod G), joined as far as they lie in this thread.
template <int G>
__device__ __forceinline__ void join_chains(const LpOut& in, int64_t parts, int64_t t, int g,
                                            float& M, float& S, float& D) {
  constexpr int C = kChains / G, A = C >= 4 ? 1 : 4 / C;   // four loads in flight at least
  float cm[C], cs[C], cd[C];
#pragma unroll
  for (int u = 0; u < C; ++u) { cm[u] = -INFINITY; cs[u] = 0.f; cd[u] = 0.f; }
  for (int64_t p0 = g; p0 < parts; p0 += A * kChains) {
    float2 ms[A][C];
    float d[A][C];
#pragma unroll
    for (int x = 0; x < A; ++x)
#pragma unroll
      for (int u = 0; u < C; ++u) {
        const int64_t p = p0 + x * kChains + u * G, at = (p < parts ? p : p0) * in.sp + t * in.st;
        ms[x][u] = in.part[at];
        d[x][u] = in.pd[at];
      }
#pragma unroll
    for (int x = 0; x < A; ++x)
#pragma unroll
      for (int u = 0; u < C; ++u)
        if (p0 + x * kChains + u * G < parts)
          join_part(cm[u], cs[u], cd[u], ms[x][u].x, ms[x][u].y, d[x][u]);
  }
#pragma unroll
  for (int h = C / 2; h > 0; h /= 2)
#pragma unroll
    for (int u = 0; u < h; ++u) join_part(cm[u], cs[u], cd[u], cm[u + h], cs[u + h], cd[u + h]);
  M = cm[0]; S = cs[0]; D = cd[0];
}

// The chains of a wave's lanes: lane l joins lane l + half for half = 32 ... 1. Every lane
// gets lane 0's.
__device__ __forceinline__ void join_lanes(float& M, float& S, float& D) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto lower_upper = [&](auto swap) {              // both lanes of a pair join alike
    const auto m = swap(__float_as_uint(M)), s = swap(__float_as_uint(S)),
               d = swap(__float_as_uint(D));
    M = __uint_as_float(m[0]); S = __uint_as_float(s[0]); D = __uint_as_float(d[0]);
    join_part(M, S, D, __uint_as_float(m[1]), __uint_as_float(s[1]), __uint_as_float(d[1]));
  };
  lower_upper([](uint32_t x) { return __builtin_amdgcn_permlane32_swap(x, x, false, false); });
  lower_upper([](uint32_t x) { return __builtin_amdgcn_permlane16_swap(x, x, false, false); });
  // within 16 lanes: from the lane `half` further on, for the lower ones
  join_part(M, S, D, dpp_move<kDppDown + 8>(M), dpp_move<kDppDown + 8>(S), dpp_move<kDppDown + 8>(D));
  join_part(M, S, D, dpp_move<kDppDown + 4>(M), dpp_move<kDppDown + 4>(S), dpp_move<kDppDown + 4>(D));
  join_part(M, S, D, dpp_move<kDppDown + 2>(M), dpp_move<kDppDown + 2>(S), dpp_move<kDppDown + 2>(D));
  join_part(M, S, D, dpp_move<kDppDown + 1>(M), dpp_move<kDppDown + 1>(S), dpp_move<kDppDown + 1>(D));
  auto first = [](float x) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), 0)); };
  M = first(M); S = first(S); D = first(D);
#endif
}

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
__device__ __forceinline__ int64_t key_id(uint64_t k) { return int64_t(uint32_t(~uint32_t(k))); }
__device__ __forceinline__ uint64_t max_u64(uint64_t a, uint64_t b) { return a > b ? a : b; }

// Many tokens and at most one alternative: all parts and lists, or (TAU_ONLY) the lists
// of the first tiles, for a token's largest key. JT tokens a workgroup and G threads for
// each, thread g taking every G-th part and list, then the threads pairwise. 32 tokens
// read whole lines of every part; below 4096 tokens that leaves most CUs idle, and 16
// (below 1024: 4) tokens a workgroup are faster.
template <bool SOFTCAP, bool TAU_ONLY, int JT, int G>
__global__ __launch_bounds__(JT * G) void k_lp_join(JoinArgs a) {
  constexpr int kT = JT * G;
  __shared__ uint64_t keys[kT / 2];
  __shared__ float4 grp[kT / 2];
  const int tid = threadIdx.x, tk = tid % JT, g = tid / JT;
  const int64_t t = int64_t(blockIdx.x) * JT + tk;
  int64_t n_live = a.N;
  if (a.count) { const int64_t c = *a.count; n_live = c < n_live ? c : n_live; }
  const bool live = t < n_live;
  const int K = a.top_k;
  float M = -INFINITY, S = 0.f, D = 0.f;
  if (!TAU_ONLY && live) join_chains<G>(a.in, a.parts, t, g, M, S, D);
  uint64_t top = 0;
  if (K > 0 && live) {
#pragma unroll 4
    for (int64_t l = a.list0 + g; l < a.lists; l += G) {
      const int64_t at = l * a.in.cl + t * a.in.ct;
      top = max_u64(top, rank_key(a.in.cv[at], l * a.list_rows + a.in.ci[at]));
    }
  }
  for (int half = G / 2; half > 0; half >>= 1) {
    // threads half .. 2 half - 1 of each token hand theirs to 0 .. half - 1
    const int slot = tid % (half * JT);
    if (g >= half && g < 2 * half) {
      grp[slot] = make_float4(M, S, D, 0.f);
      keys[slot] = top;
    }
    __syncthreads();
    if (g < half) {
      const float4 f = grp[slot];
      join_part(M, S, D, f.x, f.y, f.z);
      top = max_u64(top, keys[slot]);
    }
    __syncthreads();
  }
  if (g != 0 || t >= a.N) return;
  if (TAU_ONLY) {
    a.first[t] = top;                              // 0 of no list
    a.tau[t] = top != 0 ? key_value(top) : -INFINITY;
    return;
  }
  const int64_t o = a.idx ? int64_t(a.idx[t]) : t;
  const bool shown = live && (!a.labels || a.labels[t] != a.ignore_index);
  write_token(a, t, o, shown, M, S, D);
  if (K > 0) {
    const bool has = shown && top != 0;
    write_alternative(a, o, 0, has ? warp_logit<SOFTCAP>(a.warp, key_value(top)) : 0.f,
                      has ? key_id(top) : -1, M, logf(S));
  }
}

// Lists of tiles without a tau, more than one alternative (up to 1024 lists; TAU_ONLY:
// those of the first tiles, for the top_k keys and the top_k-th logit): G threads a token,
// a list each, held in registers (the candidates of a token lie together). The
// top_k-th largest of the lists' largest keys bounds the alternatives, and at most top_k
// lists reach it: their keys from the bound up go to LDS, where each counts the larger
// ones. With 20 alternatives (us, and by sorted lists): 529 rows over 307 lists
// 21 and 112, 272 over 194 12 and 87, 456 over 16 13 and 43. "Sorted lists": a thread's
// lists sorted and merged in registers, then the threads' pairwise through LDS; for the
// first tiles of 2000 rows over 32000 with 20 alternatives that made the call 284 us, this
// 236.
template <int PER, int KC>    // K <= KC
struct DenseList {
  uint64_t group[64];          // the largest key of each PER threads
  uint64_t bound[2];           // the top_k-th largest of those, and of the threads' keys; or 1
  int count[2];
  uint64_t list[KC * (KC > PER ? KC : PER)];       // K threads' keys, K groups' threads
  uint64_t few[KC * (KC * KC / 64 + 1)];           // K groups' keys of the list
  uint64_t won[KC];
};

template <bool SOFTCAP, bool TAU_ONLY, int G, int KC>             // kc = KC
__global__ __launch_bounds__(G < 256 ? 256 : G) void k_lp_join_dense(JoinArgs a) {
  constexpr int JT = G < 256 ? 256 / G : 1, PER = G / 64;
  constexpr int GC = G < kChains ? G : kChains;    // threads with a chain
  __shared__ DenseList<PER, KC> sel[JT];
  __shared__ float red[3][JT][GC];
  const int tid = threadIdx.x, tk = tid / G, g = tid % G;
  const int64_t t = int64_t(blockIdx.x) * JT + tk;
  int64_t n_live = a.N;
  if (a.count) { const int64_t c = *a.count; n_live = c < n_live ? c : n_live; }
  const bool live = t < n_live;
  const int K = a.top_k;
  DenseList<PER, KC>& st = sel[tk];
  row_u32x4 rv[KC / 4];
  uint32_t ri[KC / 4];
  bool on = live && g < a.lists;
  if (on) {
    const int64_t at = t * a.in.ct + g * a.in.cl;
#pragma unroll
    for (int i = 0; i < KC / 4; ++i) rv[i] = load_raw(a.in.cv + at + 4 * i);
#pragma unroll
    for (int i = 0; i < KC / 4; ++i) ri[i] = reinterpret_cast<const uint32_t*>(a.in.ci + at)[i];
  }
  float M = -INFINITY, S = 0.f, D = 0.f;
  if (!TAU_ONLY && live && g < GC)                 // parts <= G: see run_join_dense
    for (int64_t p = g; p < a.parts; p += kChains) {
      const int64_t at = p * a.in.sp + t * a.in.st;
      const float2 ms = a.in.part[at];
      join_part(M, S, D, ms.x, ms.y, a.in.pd[at]);
    }
  uint64_t key[KC], best = 0;
#pragma unroll
  for (int k = 0; k < KC; ++k) {
    const float v = __uint_as_float(rv[k / 4][k % 4]);
    on = on && v > -INFINITY;                      // nothing behind the first such place
    key[k] = on ? rank_key(v, g * a.list_rows + ((ri[k / 4] >> (8 * (k % 4))) & 255))
                : 0;
    best = max_u64(best, key[k]);
  }
  if constexpr (!TAU_ONLY) {
    if (g < GC) { red[0][tk][g] = M; red[1][tk][g] = S; red[2][tk][g] = D; }
  }
  const uint32_t hi = group_all<PER>(uint32_t(best >> 32), MaxOp());
  const uint32_t lo = group_all<PER>(uint32_t(best >> 32) == hi ? uint32_t(best) : 0u, MaxOp());
  if (g % PER == 0) st.group[g / PER] = (uint64_t(hi) << 32) | lo;
  if (g < KC) st.won[g] = 0;
  if (g < 2) { st.bound[g] = 1; st.count[g] = 0; }
  __syncthreads();
  if (g < 64) {
    const uint64_t x = st.group[g];
    int larger = 0;
    for (int i = 0; i < 64; ++i) larger += st.group[i] > x ? 1 : 0;
    if (x != 0 && larger == K - 1) st.bound[0] = x;
  }
  __syncthreads();
  if (best >= st.bound[0]) st.list[atomicAdd(&st.count[0], 1)] = best;
  __syncthreads();
  int n = st.count[0];
  for (int i = g; i < n; i += G) {
    const uint64_t x = st.list[i];
    int larger = 0;
    for (int o = 0; o < n; ++o) larger += st.list[o] > x ? 1 : 0;
    if (larger == K - 1) st.bound[1] = x;
  }
  __syncthreads();
  const uint64_t bound = st.bound[1];
  if (best >= bound) {
#pragma unroll
    for (int k = 0; k < KC; ++k)
      if (key[k] >= bound) st.list[atomicAdd(&st.count[1], 1)] = key[k];
  }
  __syncthreads();
  n = st.count[1];
  const uint64_t* keys = st.list;
  if (a.lists < 64) {
    // few lists leave that bound low (fewer than top_k none at all): the same once more
    // over the keys in 64 groups, of at most 16
    if (g < 64) {
      uint64_t x = 0;
      for (int i = g; i < n; i += 64) x = max_u64(x, st.list[i]);
      st.group[g] = x;
    }
    if (g == 0) { st.bound[0] = 1; st.count[0] = 0; }
    __syncthreads();
    if (g < 64) {
      const uint64_t x = st.group[g];
      int larger = 0;
      for (int i = 0; i < 64; ++i) larger += st.group[i] > x ? 1 : 0;
      if (x != 0 && larger == K - 1) st.bound[0] = x;
    }
    __syncthreads();
    for (int i = g; i < n; i += G)
      if (st.list[i] >= st.bound[0]) st.few[atomicAdd(&st.count[0], 1)] = st.list[i];
    __syncthreads();
    n = st.count[0];
    keys = st.few;
  }
  for (int i = g; i < n; i += G) {
    const uint64_t x = keys[i];
    int larger = 0;
    for (int o = 0; o < n; ++o) larger += keys[o] > x ? 1 : 0;
    if (larger < K) st.won[larger] = x;
  }
  __syncthreads();
  if (g >= 64) return;
  if constexpr (!TAU_ONLY) {
    auto join = [&](float& m, float& s, float& d, int c) {
      join_part(m, s, d, red[0][tk][c], red[1][tk][c], red[2][tk][c]);
    };
    if constexpr (GC == 256) {
      float m = red[0][tk][g + 64], s = red[1][tk][g + 64], d = red[2][tk][g + 64];
      join(M, S, D, g + 128);
      join(m, s, d, g + 192);
      join_part(M, S, D, m, s, d);
    } else if constexpr (GC == 128) {
      join(M, S, D, g + 64);
    }
    join_lanes(M, S, D);
  }
  if (g >= K || t >= a.N) return;
  if constexpr (TAU_ONLY) {
    a.first[g * a.first_ld + t] = st.won[g];       // of no list: 0
    if (g == K - 1) a.tau[t] = st.won[g] != 0 ? key_value(st.won[g]) : -INFINITY;
    return;
  }
  const int64_t o = a.idx ? int64_t(a.idx[t]) : t;
  const bool shown = live && (!a.labels || a.labels[t] != a.ignore_index);
  if (g == 0) write_token(a, t, o, shown, M, S, D);
  const uint64_t x = st.won[g];
  const bool has = shown && x != 0;
  write_alternative(a, o, g, has ? warp_logit<SOFTCAP>(a.warp, key_value(x)) : 0.f,
                    has ? key_id(x) : -1, M, logf(S));
}

// Many tokens, lists of tiles with a tau, few of which hold anything: 16 tokens a
// workgroup, 32 threads for each. Every candidate goes to a list in LDS, with the
// top_k of the tiles before, and the top_k of those are selected (join_sparse.h); a list
// that overflows is filled again from its own top_k-th key on. 1946 rows over 186 lists
// with 5 alternatives 13 us, 6144 rows over 1984 lists with 8 50 us.
constexpr int kSparseTokens = 16;

struct WorkgroupEnv {
  __device__ __forceinline__ void sync() const { __syncthreads(); }
  __device__ __forceinline__ bool any(bool x) const { return __syncthreads_or(x) != 0; }
  __device__ __forceinline__ int add(int* p) const { return atomicAdd(p, 1); }
};

template <bool SOFTCAP>
__global__ __launch_bounds__(512) void k_lp_join_sparse(JoinArgs a) {
  constexpr int JT = kSparseTokens, G = kSparseG;
  __shared__ SparseKeys<JT> st;
  __shared__ float4 grp[G / 2 * JT];
  const int tid = threadIdx.x, tk = tid % JT, g = tid / JT;
  const int64_t t = int64_t(blockIdx.x) * JT + tk;
  int64_t n_live = a.N;
  if (a.count) { const int64_t c = *a.count; n_live = c < n_live ? c : n_live; }
  const bool live = t < n_live;
  const int K = a.top_k;
  float M = -INFINITY, S = 0.f, D = 0.f;
  if (live) join_chains<G>(a.in, a.parts, t, g, M, S, D);
  const int64_t keys = K + (a.lists - a.list0) * a.in.kc;
  sparse_top(st, tk, g, K, keys, WorkgroupEnv(), [&](auto push) {
    if (!live) return;
    if (g < K) {
      const uint64_t key = a.first[g * a.first_ld + t];
      if (key != 0) push(key);
    }
    for (int64_t l = a.list0 + g; l < a.lists; l += 4 * G) {
      float v[4][2];
      uint8_t row[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {              // the first two of four lists at a time
        const int64_t at = (l + u * G < a.lists ? l + u * G : l) * a.in.cl + t * a.in.ct;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int64_t i = at + (k < a.in.kc ? k : 0) * a.in.ck;
          v[u][k] = a.in.cv[i];
          row[u][k] = a.in.ci[i];
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (l + u * G >= a.lists || !(v[u][0] > -INFINITY)) continue;
        const int64_t at = (l + u * G) * a.in.cl + t * a.in.ct, v0 = (l + u * G) * a.list_rows;
        push(rank_key(v[u][0], v0 + row[u][0]));
        if (a.in.kc < 2 || !(v[u][1] > -INFINITY)) continue;
        push(rank_key(v[u][1], v0 + row[u][1]));
        for (int k = 2; k < a.in.kc; ++k) {
          const float x = a.in.cv[at + k * a.in.ck];
          if (!(x > -INFINITY)) break;
          push(rank_key(x, v0 + a.in.ci[at + k * a.in.ck]));
        }
      }
    }
  });
  for (int half = G / 2; half > 0; half >>= 1) {
    const int slot = tid % (half * JT);
    if (g >= half && g < 2 * half) grp[slot] = make_float4(M, S, D, 0.f);
    __syncthreads();
    if (g < half) {
      const float4 f = grp[slot];
      join_part(M, S, D, f.x, f.y, f.z);
    }
    __syncthreads();
  }
  if (g == 0) grp[tk] = make_float4(M, S, D, 0.f);
  __syncthreads();
  if (t >= a.N) return;
  const float4 f = grp[tk];
  const int64_t o = a.idx ? int64_t(a.idx[t]) : t;
  const bool shown = live && (!a.labels || a.labels[t] != a.ignore_index);
  if (g == 0) write_token(a, t, o, shown, f.x, f.y, f.z);
  if (g < K) {
    const uint64_t k = st.won[tk][g];
    const bool has = shown && k != 0;
    write_alternative(a, o, g, has ? warp_logit<SOFTCAP>(a.warp, key_value(k)) : 0.f,
                      has ? key_id(k) : -1, f.x, logf(f.y));
  }
}

// A workgroup joins one token of 64-row tiles. The top_k of any grouped keys lie in
// the top_k groups of the largest keys, so the alternatives are found in two or three
// selections: of tiles (of threads, each with several tiles, and then of their tiles
// beyond 2048 tiles), then of the logits of those tiles. A key is a logit's order and
// then the lower id, so keys are distinct. Each selection is a chain of a few barriers
// and bound by that: 1 row over 2048 tiles with 8 alternatives 12 us, 48 over 4000 tiles
// with 20 25 us, 257 over 79 tiles with 3 8 us.
constexpr int kFewThreads = 1024;
constexpr int kSelMax = 2 * kFewThreads;           // keys of a selection

struct Select {
  uint64_t group[64];          // the largest key of each 16 threads
  uint64_t bound;              // the K-th largest of those, or 1
  int count;
  uint64_t list[kSelMax];      // the keys from the bound up
  uint64_t won[kLpTop];        // the K largest, in order; 0 behind the last
};

// The K <= 32 largest of the workgroup's keys (two a thread) in st.won: at least K
// keys reach the K-th largest of the 64 groups' largest, and usually few more; those
// are gathered and each counts the larger ones. Ends with a barrier.
__device__ __forceinline__ void select_keys(uint64_t a, uint64_t b, int K, Select& st) {
  const int tid = threadIdx.x;
  const uint64_t m = max_u64(a, b);
  const uint32_t hi = group_all<16>(uint32_t(m >> 32), MaxOp());
  const uint32_t lo = group_all<16>(uint32_t(m >> 32) == hi ? uint32_t(m) : 0u, MaxOp());
  if ((tid & 15) == 0) st.group[tid >> 4] = (uint64_t(hi) << 32) | lo;
  if (tid < kLpTop) st.won[tid] = 0;
  if (tid == 0) { st.count = 0; st.bound = 1; }
  __syncthreads();
  if (tid < 64) {
    const uint64_t k = st.group[tid];
    int above = 0;
    for (int i = 0; i < 64; ++i) above += st.group[i] > k ? 1 : 0;
    if (k != 0 && above == K - 1) st.bound = k;
  }
  __syncthreads();
  const uint64_t bound = st.bound;
  if (a >= bound) st.list[atomicAdd(&st.count, 1)] = a;     // any order: they are ranked
  if (b >= bound) st.list[atomicAdd(&st.count, 1)] = b;
  __syncthreads();
  const int n = st.count;
  for (int i = tid; i < n; i += kFewThreads) {
    const uint64_t k = st.list[i];
    int above = 0;
    for (int o = 0; o < n && above < K; ++o) above += st.list[o] > k ? 1 : 0;
    if (above < K) st.won[above] = k;
  }
  __syncthreads();
}

template <bool SOFTCAP>
__global__ __launch_bounds__(kFewThreads) void k_lp_join_few(JoinArgs a) {
  constexpr int kWaves = kFewThreads / 64;
  __shared__ float red[3][kWaves];
  __shared__ Select st;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t = blockIdx.x;
  const bool live = !a.labels || a.labels[t] != a.ignore_index;
  const float2* part = a.in.part + t * a.in.st;
  const float* pd = a.in.pd + t * a.in.st;
  const float* zmax = a.in.zmax + t * a.in.st;
  const int K = a.top_k;
  float M = -INFINITY, S = 0.f, D = 0.f;
  uint64_t best[2] = {0, 0};                       // this thread's tiles, or the best of them
  const bool direct = a.parts <= kSelMax;
  auto tile_key = [&](int64_t p) -> uint64_t { return p < a.parts ? rank_key(zmax[p], p) : 0; };
  for (int64_t p = tid; p < a.parts; p += 2 * kFewThreads) {
    const int64_t p1 = p + kFewThreads < a.parts ? p + kFewThreads : p;
    const float2 m0 = part[p], m1 = part[p1];
    const float d0 = pd[p], d1 = pd[p1];
    if (K > 0) {
      const uint64_t k0 = tile_key(p), k1 = tile_key(p + kFewThreads);
      best[0] = max_u64(best[0], direct ? k0 : max_u64(k0, k1));
      if (direct) best[1] = k1;
    }
    join_part(M, S, D, m0.x, m0.y, d0);
    if (p1 != p) join_part(M, S, D, m1.x, m1.y, d1);
  }
  const float Mw = wave_all(M, MaxOp());
  const float dl = below(M, Mw), f = exp2f(dl * kLog2e);
  D = wave_all(f * fmaf(dl, S, D), AddOp());
  S = wave_all(S == 0.f ? 0.f : S * f, AddOp());
  if (lane == 0) { red[0][w] = Mw; red[1][w] = S; red[2][w] = D; }
  if (K > 0) {
    select_keys(best[0], best[1], K, st);
    if (!direct) {
      // the tiles of the threads that won: key_id % kFewThreads names the thread
      const int per = int((a.parts + kFewThreads - 1) / kFewThreads);
      uint64_t c[2] = {0, 0};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int i = tid + j * kFewThreads;
        if (i < K * per && st.won[i / per] != 0)
          c[j] = tile_key(key_id(st.won[i / per]) % kFewThreads + int64_t(i % per) * kFewThreads);
      }
      __syncthreads();                             // the winners are read
      select_keys(c[0], c[1], K, st);
    }
    // the logits of the K tiles
    uint64_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = tid + j * kFewThreads;
      if (i < K * 64 && st.won[i / 64] != 0) {
        const int64_t v = key_id(st.won[i / 64]) * 64 + i % 64;
        if (v < a.V) c[j] = rank_key(a.in.z[t * a.V + v], v);
      }
    }
    __syncthreads();
    select_keys(c[0], c[1], K, st);
  } else {
    __syncthreads();
  }
  if (tid >= (K > 0 ? K : 1)) return;
  M = -INFINITY; S = 0.f; D = 0.f;
  for (int i = 0; i < kWaves; ++i) join_part(M, S, D, red[0][i], red[1][i], red[2][i]);
  if (tid == 0) write_token(a, t, t, live, M, S, D);
  if (K > 0) {
    const uint64_t m = st.won[tid];
    const bool has = live && m != 0;
    write_alternative(a, t, tid, has ? warp_logit<SOFTCAP>(a.warp, key_value(m)) : 0.f,
                      has ? key_id(m) : -1, M, logf(S));
  }
}

// ---- the logit gradient -------------------------------------------------------------------
// With a = dL/dlogp, b = dL/dentropy, l = x - lse and p = exp(l):
//   dL/dx_v = a [v = y] - p (a + b (l + entropy))
// so G = (ca [v = y] + p (c0 + c1 l)) dx/dz with ca = a, c0 = -(a + b entropy),
// c1 = -b, formed once per live token in the gathered order. A token outside the
// vocabulary gets NaN: its gradients fail closed, as the head's loss does.
//
// G goes to the products as bf16, off by up to 2^-8 of itself: a pair of bf16, which
// float32 gradients use, takes the gradients of 3687 rows of 4096 over 131072 from 8.9 to
// 15.4 ms. That adds up where it matters most: the G of the given tokens is by far the
// largest of its row, the dW row of a frequent token is the sum of many of them, often of
// either sign, and what all rows of W share cancels in dH only against it. So what rounding
// those left is kept in float32. It is added to dH's float32 sums (times W's row of the
// token) and, a weighted lookup gradient over the same rows, to the float32 dW rows of the
// tokens, which the products leave beside dW for it; both are then rounded once. That
// takes 7 us of 562 (a training step of 2048 rows of 1024 over 32000) and 30 of 12190 (4096
// of 4096 over 131072) more than a repair of the rounded dW alone, and leaves dH and dW off
// by 0.00166 of their norm, as much as rounding the exact ones does (0.0024 and 0.0022 so).
__global__ __launch_bounds__(256) void k_lp_coef(
    const int32_t* __restrict__ idx, const int64_t* __restrict__ labels,
    const int64_t* __restrict__ count, int64_t N, int64_t V, int64_t ignore_index,
    const float* __restrict__ lse, const float* __restrict__ ent, const float* __restrict__ ga,
    const float* __restrict__ gb, float* __restrict__ lse_g, float* __restrict__ c0,
    float* __restrict__ c1, float* __restrict__ ca) {
  const int64_t r = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (r >= N || r >= *count) return;
  const int64_t t = idx[r], y = labels[r];
  float a = ga ? ga[t] : 0.f;
  const float b = gb ? gb[t] : 0.f, s = gb ? ent[t] : 0.f;
  if (y != ignore_index && (y < 0 || y >= V)) a = NAN;
  lse_g[r] = lse[t];
  c0[r] = -(a + b * s);
  c1[r] = -b;
  ca[r] = a;
}

// What rounding x to bf16 leaves of it; nothing of infinities and NaN.
__device__ __forceinline__ float bf16_rest(float x) {
  const float r = x - bf16_to_f32(f32_to_bf16(x));
  return fabsf(r) < INFINITY ? r : 0.f;
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
  float* rest;                // !SPLIT: what rounding the given token's G leaves

  static constexpr int kTokBytes = 6144;
  __device__ __forceinline__ void stage(char* tok, int64_t n0, int wave, int lane) const {
    stage_tokens<2>(tok, labels, n0, N, wave, lane);
    stage_tokens<1>(tok + 2048, lse, n0, N, wave, lane);
    stage_tokens<1>(tok + 3 * 1024, c0, n0, N, wave, lane);
    stage_tokens<1>(tok + 4096, c1, n0, N, wave, lane);
    stage_tokens<1>(tok + 5120, ca, n0, N, wave, lane);
  }

  __device__ __forceinline__ void operator()(Acc& acc, int64_t m0, int64_t n0, int wm, int wn,
                                             int lane, char* smem, const char* tok) const {
    const int64_t* lab = reinterpret_cast<const int64_t*>(tok);
    const float* lse_t = reinterpret_cast<const float*>(tok + 2048);
    const float* c0_t = reinterpret_cast<const float*>(tok + 3 * 1024);
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
          if (!SPLIT) rest[n0 + tl] = bf16_rest(tp.val[j]);
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

// Few live tokens: the same G from the few-token kernel's logits. The coefficients
// come straight from the call's arrays.
struct FewGrad {
  const int32_t* idx;
  const int64_t* labels;      // gathered, as h is
  const int64_t* count;
  const float* lse;
  const float* ent;
  const float* ga;
  const float* gb;
  float* rest;
  uint16_t* g;
  int64_t V, v0, gblk;        // v0: the chunk's first vocabulary row
};

template <int NT, bool SOFTCAP>
__global__ __launch_bounds__(256) void k_lp_few_grad(const uint16_t* __restrict__ h,
                                                     const uint16_t* __restrict__ W, int64_t N,
                                                     int64_t H, int64_t vcur, Warp warp,
                                                     FewGrad a) {
  __shared__ __attribute__((aligned(16))) FewSmem<NT, 1> sm;
  const int64_t c0 = int64_t(blockIdx.x) * 64;     // the chunk's column
  few_logits<NT, 16, 1>(h, W, N, H, vcur, c0, sm);
  constexpr int TPT = kFewLanes<NT>, E = 64 / TPT;
  const int t = threadIdx.x / TPT, q = threadIdx.x % TPT;
  const int64_t live = *a.count;
  if (t >= live || t >= N) return;
  const int64_t o = a.idx[t], y = a.labels[t], at = c0 + q * E;
  const float ca = (y < 0 || y >= a.V) ? NAN : a.ga ? a.ga[o] : 0.f;
  const float cb = a.gb ? a.gb[o] : 0.f, l0 = a.lse[o];
  const float k0 = -(ca + cb * (a.gb ? a.ent[o] : 0.f));
  float g[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float z = sm.z[t][q * E + e], l = warp_logit<SOFTCAP>(warp, z) - l0;
    float x = __builtin_amdgcn_exp2f(l * kLog2e) * fmaf(-cb, l, k0);
    const bool target = y == a.v0 + at + e && at + e < vcur;
    x = (target ? x + ca : x) * warp_slope<SOFTCAP>(warp, z);
    if (target) a.rest[t] = bf16_rest(x);
    g[e] = at + e < vcur ? x : 0.f;
  }
  // 4 (or 8) adjacent columns lie in one block of 32; dH reads whole runs of 8, so the
  // zeros behind the last row are stored too
  constexpr int RUN = E < 8 ? E : 8;
#pragma unroll
  for (int e = 0; e < E; e += RUN) {
    if (at + e >= (vcur + 7) / 8 * 8) break;
    uint32_t* to = reinterpret_cast<uint32_t*>(a.g + gemm::blocked_offset(t, at + e, a.gblk));
#pragma unroll
    for (int i = 0; i < RUN; i += 2) to[i / 2] = pack_bf16x2(g[e + i], g[e + i + 1]);
  }
}

// float32: G^T[v - v0][t] of one vocabulary chunk, zero for ignored tokens and for
// the columns N <= t < ldg.
template <int TN, bool SOFTCAP>
__global__ __launch_bounds__(256) void k_lp_f32_grad(
    const float* __restrict__ h, const float* __restrict__ W, const int64_t* __restrict__ labels,
    int64_t N, int64_t H, int64_t V, int64_t ignore_index, Warp warp,
    const float* __restrict__ lse, const float* __restrict__ ent, const float* __restrict__ ga,
    const float* __restrict__ gb, int64_t v0, int64_t vcur, int64_t ldg, float* __restrict__ gt) {
  __shared__ __attribute__((aligned(16))) F32Stage<TN> st;
  const int64_t m0 = int64_t(blockIdx.x) * 64, t0 = int64_t(blockIdx.y) * TN;
  f32_logits<TN>(W + v0 * H, h, m0, vcur, t0, N, H, st);
  const int tl = threadIdx.x % TN;
  const int64_t t = t0 + tl;
  if (t >= ldg) return;
  const int64_t y = t < N ? labels[t] : ignore_index;
  const bool live = t < N && y != ignore_index;
  float ca = 0.f, cb = 0.f, k0 = 0.f, l0 = 0.f;
  if (live) {
    ca = (y < 0 || y >= V) ? NAN : ga ? ga[t] : 0.f;
    cb = gb ? gb[t] : 0.f;
    k0 = -(ca + cb * (gb ? ent[t] : 0.f));
    l0 = lse[t];
  }
  for (int r = threadIdx.x / TN; r < 64; r += 256 / TN) {
    if (m0 + r >= vcur) break;
    float v = 0.f;
    if (live) {
      const float zz = st.z[tl][r], l = warp_logit<SOFTCAP>(warp, zz) - l0;
      v = exp2f(l * kLog2e) * fmaf(-cb, l, k0);
      if (v0 + m0 + r == y) v += ca;
      v *= warp_slope<SOFTCAP>(warp, zz);
    }
    gt[(m0 + r) * ldg + t] = v;
  }
}

// float32 products of a chunk's G^T [rows][ldg] on the float32 matrix instruction,
// 64 x 64 tiles as above:
//   DW:  C[m][n] = sum_t G^T[m][t] h[t][n]     (m vocabulary rows, K = tokens)
//   !DW: C[t][n] = sum_m G^T[m][t] W[m][n]     (K = the chunk's vocabulary rows)
// B (and for dH also A) is stored with its row contiguous across K: a chunk goes to
// LDS as [k][64]. A workgroup makes one tile of a segment of K (dH has few tiles and a
// long K; each segment leaves a partial product of its own). Both products run in one
// grid: 257 x 515 over 5003 46 us (50 in two), 512 x 1024 over 32000 585 us (115
// TFLOP/s).
struct F32Product {
  const float* b;
  int64_t M, K, kseg;
  int accumulate;
  float* c;
  int64_t seg_stride;
};
struct F32ProductStage {
  float a[2][64 * kF32Ld], b[2][kF32K * kZLd];     // 64 kF32Ld > kF32K kZLd
};

template <bool DW>
__device__ __forceinline__ void f32_product(const float* __restrict__ gt, int64_t ldg, int64_t H,
                                            const F32Product& q, int64_t index,
                                            F32ProductStage& st) {
  const int64_t M = q.M, K = q.K, mt = (M + 63) / 64, nt = (H + 63) / 64;
  const float* __restrict__ B = q.b;
  float (&sa)[2][64 * kF32Ld] = st.a;
  float (&sb)[2][kF32K * kZLd] = st.b;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t m0 = index % mt * 64, n0 = index / mt % nt * 64, z = index / (mt * nt);
  const int64_t k0 = z * q.kseg, k1 = K - k0 < q.kseg ? K : k0 + q.kseg;
  float* __restrict__ C = q.c + z * q.seg_stride;
  // [k][64] chunks: rows tid / 16, + 16, columns 4 (tid % 16); [64][k] as f32_logits
  const int kr = tid >> 4, kc = (tid & 15) * 4, lr = tid >> 3, lc = (tid & 7) * 4;
  const float* ar[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t m = m0 + lr + 32 * i, c = m0 + kc < ldg ? m0 + kc : 0;
    ar[i] = DW ? gt + (m < M ? m : M - 1) * ldg + lc : gt + (kr + 16 * i) * ldg + c;
  }
  auto load_a = [&](int64_t k, F32Regs& f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) unpack_chunk<float>(load_raw(ar[i] + (DW ? k : k * ldg)), f.a[i]);
  };
  auto end = [&](int64_t k, F32Regs& f) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t kk = k + kr + 16 * i;
      if constexpr (DW) {
        load_chunk(ar[i] - lc, k + lc, k1, f.a[i]);
      } else {
        load_chunk(gt + (kk < k1 ? kk : k1 - 1) * ldg, m0 + kc, kk < k1 ? M : 0, f.a[i]);
      }
      load_chunk(B + (kk < k1 ? kk : k1 - 1) * H, n0 + kc, kk < k1 ? H : 0, f.b[i]);
    }
  };
  f32x4 acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  const int wm = (w & 1) * 32, wn = (w >> 1) * 32, r = lane & 15, kg = (lane >> 4) * 4;
  auto keep = [&](const F32Regs& f, int half) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* pa = sa[half] + (DW ? (lr + 32 * i) * kF32Ld + lc : (kr + 16 * i) * kZLd + kc);
      *reinterpret_cast<f32x4*>(pa) = as_f32x4(f.a[i]);
      *reinterpret_cast<f32x4*>(sb[half] + (kr + 16 * i) * kZLd + kc) = as_f32x4(f.b[i]);
    }
  };
  auto multiply = [&](int half) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      float fa[2][4], fb[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int kk = p * 16 + kg + e;
          fa[i][e] = sa[half][DW ? (wm + 16 * i + r) * kF32Ld + kk : kk * kZLd + wm + 16 * i + r];
          fb[i][e] = sb[half][kk * kZLd + wn + 16 * i + r];
        }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[i][e], fb[j][e], acc[i][j], 0, 0, 0);
    }
  };
  // B's columns: 16 bytes where the tile lies in the row, otherwise one by one, those
  // past the row (their products are not stored) from its last
  const bool inside = n0 + 64 <= H;
  const float* b0 = B + (inside ? n0 + kc : 0);
  int col[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) col[e] = int(n0 + kc + e < H ? n0 + kc + e : H - 1);
  if (inside) {
    f32_chunks(k0, k1, [&](int64_t k, F32Regs& f) {
      load_a(k, f);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        unpack_chunk<float>(load_raw(b0 + (k + kr + 16 * i) * H), f.b[i]);
    }, end, keep, multiply);
  } else {
    f32_chunks(k0, k1, [&](int64_t k, F32Regs& f) {
      load_a(k, f);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) f.b[i][e] = b0[(k + kr + 16 * i) * H + col[e]];
    }, end, keep, multiply);
  }
  // acc[i][j][e]: row 16 i + 4 (lane / 16) + e, column 16 j + lane % 16
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t m = m0 + wm + 16 * i + kg + e;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int64_t n = n0 + wn + 16 * j + r;
        if (m < M && n < H) {
          float* c = C + m * H + n;
          *c = q.accumulate ? *c + acc[i][j][e] : acc[i][j][e];
        }
      }
    }
}

// dH's tiles, then dW's.
__global__ __launch_bounds__(256) void k_f32_products(const float* __restrict__ gt, int64_t ldg,
                                                      int64_t H, F32Product dh, F32Product dw,
                                                      int64_t dh_tiles) {
  __shared__ __attribute__((aligned(16))) F32ProductStage st;
  const int64_t i = blockIdx.x;
  if (i < dh_tiles) f32_product<false>(gt, ldg, H, dh, i, st);
  else f32_product<true>(gt, ldg, H, dw, i - dh_tiles, st);
}

// dH (+)= the segments' partial products, in an order of their count alone: 8 groups of
// 32 threads add every 8th segment, then the groups' sums in order.
__global__ __launch_bounds__(256) void k_f32_dh_sum(const float* __restrict__ part, int segs,
                                                    int64_t n, int accumulate,
                                                    float* __restrict__ dH) {
  __shared__ float red[8][32];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t i = int64_t(blockIdx.x) * 32 + c;
  float v = 0.f;
  if (i < n) {
#pragma unroll 8
    for (int z = g; z < segs; z += 8) v += part[z * n + i];
  }
  red[g][c] = v;
  __syncthreads();
  if (g > 0 || i >= n) return;
  v = accumulate ? dH[i] : 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) v += red[k][c];
  dH[i] = v;
}

unsigned cdiv(int64_t a, int64_t b) { return unsigned((a + b - 1) / b); }

template <int I>
using Int = std::integral_constant<int, I>;

// Whether the float32 tiles take 32 tokens instead of 64: where the last 64 would be half
// empty, or where there are too few tiles for the chip (us of a training step with 64 and
// 32: 257 tokens of 515 over 5003 114 and 106, 20 of 1024 over 32000 167 and 140, 300 of
// 515 over 1003 66 and 55; the other way 512 of 1024 over 32000 1148 and 1188).
bool f32_narrow(int64_t N, int64_t V) {
  return (N - 1) % 64 < 32 || ((N + 63) / 64) * ((V + 63) / 64) <= 256;
}

template <bool SOFTCAP, bool TAU_ONLY>
hipError_t run_join_dense(const LpPlan& q, const JoinArgs& j, const Launcher& L) {
  auto run = [&](auto g, auto kc) {
    constexpr int G = decltype(g)::value, T = G < 256 ? 256 : G;
    hipLaunchKernelGGL((k_lp_join_dense<SOFTCAP, TAU_ONLY, G, decltype(kc)::value>),
                       dim3(cdiv(j.N, T / G)), dim3(T), 0, L.stream, j);
  };
  auto by_kc = [&](auto g) {
    if (q.kc == 8) run(g, Int<8>{});
    else if (q.kc == 16) run(g, Int<16>{});
    else run(g, Int<32>{});
  };
  // a thread a list, and two lists a part: no more parts than threads
  if (j.lists > 1024 || (!TAU_ONLY && 2 * j.parts > j.lists + 1)) return hipErrorInvalidValue;
  L.pre(kLpJoin);
  if (j.lists <= 64) by_kc(Int<64>{});
  else if (j.lists <= 128) by_kc(Int<128>{});
  else if (j.lists <= 256) by_kc(Int<256>{});
  else if (j.lists <= 512) by_kc(Int<512>{});
  else by_kc(Int<1024>{});
  L.post(kLpJoin);
  return hipGetLastError();
}

template <bool SOFTCAP, bool TAU_ONLY>
hipError_t run_join(const LpPlan& q, const JoinArgs& j, const Launcher& L) {
  // lists without a tau and more than one alternative go to run_join_dense
  if (q.tiles && (TAU_ONLY || !j.first) && j.top_k > 1) return hipErrorInvalidValue;
  L.pre(kLpJoin);
  if (!q.tiles) {
    hipLaunchKernelGGL(k_lp_join_few<SOFTCAP>, dim3(unsigned(j.N)), dim3(kFewThreads), 0,
                       L.stream, j);
  } else if (!TAU_ONLY && j.first) {
    hipLaunchKernelGGL(k_lp_join_sparse<SOFTCAP>, dim3(cdiv(j.N, kSparseTokens)), dim3(512), 0,
                       L.stream, j);
  } else {
    auto run = [&](auto jt) {
      constexpr int JT = decltype(jt)::value;
      hipLaunchKernelGGL((k_lp_join<SOFTCAP, TAU_ONLY, JT, 1024 / JT>), dim3(cdiv(j.N, JT)),
                         dim3(1024), 0, L.stream, j);
    };
    if (j.N >= 4096) run(Int<32>{});
    else if (j.N >= 1024) run(Int<16>{});
    else run(Int<4>{});
  }
  L.post(kLpJoin);
  return hipGetLastError();
}

template <bool SOFTCAP>
hipError_t run_few(const LpArgs& a, const Warp& warp, const LpOut& out, const Launcher& L) {
  const auto* h = static_cast<const uint16_t*>(a.h);
  const auto* W = static_cast<const uint16_t*>(a.W);
  auto go = [&](auto nt) {
    constexpr int NT = decltype(nt)::value, RB = NT >= 3 ? 2 : 1;
    const dim3 grid(cdiv(a.V, kLpRows * RB));
    auto run = [&](auto align) {
      hipLaunchKernelGGL((k_lp_few<NT, SOFTCAP, decltype(align)::value, RB>), grid, dim3(256), 0,
                         L.stream, h, W, a.tokens, a.N, a.H, a.V, warp, out);
    };
    if (a.H % 8 == 0) run(Int<16>{});
    else if (a.H % 2 == 0) run(Int<4>{});
    else run(Int<2>{});
  };
  L.pre(kLpTiles);
  if (a.N <= 16) go(Int<1>{});
  else if (a.N <= 32) go(Int<2>{});
  else if (a.N <= 48) go(Int<3>{});
  else if (a.N <= 64) go(Int<4>{});
  else go(Int<8>{});
  L.post(kLpTiles);
  return hipGetLastError();
}

template <bool SOFTCAP>
hipError_t logprobs(const LpPlan& q, const LpArgs& a, char* ws, const Launcher& L) {
  const Warp warp = make_warp(a.softcap, a.temperature);
  LpOut out{reinterpret_cast<float2*>(ws + q.off_part), reinterpret_cast<float*>(ws + q.off_pd),
            reinterpret_cast<float*>(ws + q.off_zt), reinterpret_cast<float*>(ws + q.off_cv),
            reinterpret_cast<uint8_t*>(ws + q.off_ci), reinterpret_cast<float*>(ws + q.off_zmax),
            q.top_k && !q.tiles ? reinterpret_cast<float*>(ws + q.off_z) : nullptr,
            q.sp, q.st, q.cl, q.ck, q.ct, int(q.kc), q.top_k};
  JoinArgs j{out, q.parts, 0, q.lists, q.list_rows, a.V, a.N, nullptr, nullptr, a.tokens,
             a.ignore_index, q.top_k, warp, a.logp, a.entropy, a.lse, a.top_logp, a.top_ids,
             nullptr, q.nc, nullptr};
  hipError_t e = hipSuccess;
  if (a.dtype == FLCE_F32 || q.few) {
    if (a.status)
      e = a.tokens ? launch_token_status(a.tokens, a.N, a.V, a.ignore_index, a.status, L)
                   : launch_token_status(nullptr, 0, a.V, a.ignore_index, a.status, L);
    if (e != hipSuccess) return e;
  }
  if (q.few) {
    e = run_few<SOFTCAP>(a, warp, out, L);
    return e == hipSuccess ? run_join<SOFTCAP, false>(q, j, L) : e;
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
      auto run = [&](auto tn) {
        constexpr int TN = decltype(tn)::value;
        hipLaunchKernelGGL((k_lp_f32<TN, SOFTCAP>), dim3(cdiv(a.V, 64), cdiv(c.N, TN)), dim3(256),
                           0, L.stream, static_cast<const float*>(a.h) + t0 * a.H,
                           static_cast<const float*>(a.W), c.labels, c.N, a.H, a.V, warp, out);
      };
      f32_narrow(c.N, a.V) ? run(Int<32>{}) : run(Int<64>{});
      L.post(kLpTiles);
      e = hipGetLastError();
      if (e == hipSuccess) e = run_join<SOFTCAP, false>(q, c, L);
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
  if (e == hipSuccess && q.gather && q.n_chunks > 1) e = launch_chunk_counts(p, ag, false, L);
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
      jc.count = q.n_chunks > 1 ? ag.ccnt + c : &ag.sc->n_valid;
    } else {
      at_token(jc, t0);
    }
    const int64_t pre = lp_first_tiles(q, jc.N);
    // More than one alternative: in tiles without a bound (the first group, at most 512,
    // or all where there is none: fewer than 512) the candidates of a token lie together,
    // for k_lp_join_dense. In the others up to 8 are all that the join reads of a list.
    const bool dense = q.top_k > 1;
    LpOut lone = out, to = out;
    if (dense) lone.cl = q.kc, lone.ck = 1, lone.ct = (pre > 0 ? 2 * pre : q.lists) * q.kc;
    if (q.top_k <= 8) to.kc = q.top_k;
    // vocabulary rows [v0, v1) of the chunk's live tokens
    auto tiles = [&](int64_t v0, int64_t v1, const LpOut& to, const float* tau) {
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
        return run(EpiLp<SOFTCAP, true>{jc.labels, jc.N, a.V, v0, warp, to, tau});
      return run(EpiLp<SOFTCAP, false>{jc.labels, jc.N, a.V, v0, warp, to, nullptr});
    };
    // Alternatives: the first tiles of the vocabulary alone, whole rounds of the
    // chip, give every token a bound tau that few logits of the others exceed;
    // their epilogues then have next to nothing to extract.
    if (pre > 0) {
      jc.tau = reinterpret_cast<float*>(ws + q.off_tau);
      jc.first = reinterpret_cast<uint64_t*>(ws + q.off_first);
      e = tiles(0, pre * kBM, lone, nullptr);
      jc.in = lone;
      jc.lists = 2 * pre;
      if (e == hipSuccess)
        e = dense ? run_join_dense<false, true>(q, jc, L) : run_join<false, true>(q, jc, L);
      if (e == hipSuccess) e = tiles(pre * kBM, a.V, to, jc.tau);
      jc.in = to;
      jc.list0 = 2 * pre;
      jc.lists = q.lists;
    } else {
      e = tiles(0, a.V, lone, nullptr);
      jc.in = lone;
    }
    if (e == hipSuccess)
      e = dense && pre == 0 ? run_join_dense<SOFTCAP, false>(q, jc, L)
                            : run_join<SOFTCAP, false>(q, jc, L);
  }
  return e;
}

}  // namespace

hipError_t launch_logprobs(const LpPlan& q, const LpArgs& a, char* ws, const Launcher& L) {
  return a.softcap > 0.f ? logprobs<true>(q, a, ws, L) : logprobs<false>(q, a, ws, L);
}

hipError_t launch_lp_f32_products(const Plan& p, const Args& a, int64_t chunk, const Launcher& L) {
  const int64_t v0 = chunk * p.vchunk, vcur = gemm::chunk_rows(p, chunk);
  float* dH = static_cast<float*>(a.dH);
  const int64_t kseg = lp_f32_segment(p), segs = (vcur + kseg - 1) / kseg;
  const F32Product dh{static_cast<const float*>(a.W) + v0 * p.H, p.N, vcur, kseg,
                      segs == 1 && chunk > 0 ? 1 : 0, segs == 1 ? dH : a.dh_part, p.N * p.H};
  const F32Product dw{static_cast<const float*>(a.h), vcur, p.N, p.N, a.accumulate_dW,
                      static_cast<float*>(a.dW) + v0 * p.H, 0};
  const int64_t nt = cdiv(p.H, 64), dh_tiles = cdiv(p.N, 64) * nt * segs;
  L.pre(kGemmDWDH);
  hipLaunchKernelGGL(k_f32_products, dim3(unsigned(dh_tiles + cdiv(vcur, 64) * nt)), dim3(256), 0,
                     L.stream, static_cast<const float*>(a.g), p.ldg, p.H, dh, dw, dh_tiles);
  L.post(kGemmDWDH);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || segs == 1) return e;
  L.pre(kDhReduce);
  hipLaunchKernelGGL(k_f32_dh_sum, dim3(cdiv(p.N * p.H, 32)), dim3(256), 0, L.stream, a.dh_part,
                     int(segs), p.N * p.H, chunk > 0 ? 1 : 0, dH);
  L.post(kDhReduce);
  return hipGetLastError();
}

hipError_t launch_lp_coefficients(const Plan& p, const Args& a, const LpGradArgs& g,
                                  const Launcher& L) {
  // few tokens and float32: formed where they are used
  if (p.dtype != FLCE_BF16 || lp_few_backward(p)) return hipSuccess;
  if (!p.compact) return hipErrorInvalidValue;
  L.pre(kLpJoin);
  hipLaunchKernelGGL(k_lp_coef, dim3(cdiv(p.N, 256)), dim3(256), 0, L.stream,
                     a.idx, a.yc, &a.sc->n_valid, p.N, p.V, a.ignore_index, g.lse, g.entropy, g.grad_logp, g.grad_entropy, g.lse_g, g.c0, g.c1, g.ca);
  L.post(kLpJoin);
  return hipGetLastError();
}

hipError_t launch_lp_gradient(const Plan& p, const Args& a, const LpGradArgs& g, int64_t chunk,
                              const Launcher& L) {
  const int64_t v0 = chunk * p.vchunk, vcur = gemm::chunk_rows(p, chunk);
  const Warp warp = make_warp(a.softcap, g.temperature);
  if (p.dtype == FLCE_F32) {
    auto run = [&](auto tn, auto cap) {
      constexpr int TN = decltype(tn)::value;
      hipLaunchKernelGGL((k_lp_f32_grad<TN, decltype(cap)::value>),
                         dim3(cdiv(vcur, 64), cdiv(p.ldg, TN)), dim3(256), 0, L.stream,
                         static_cast<const float*>(a.h), static_cast<const float*>(a.W), a.labels,
                         p.N, p.H, p.V, a.ignore_index, warp, g.lse, g.entropy, g.grad_logp,
                         g.grad_entropy, v0, vcur, p.ldg, static_cast<float*>(a.g));
    };
    auto by_cap = [&](auto tn) {
      a.softcap > 0.f ? run(tn, std::true_type{}) : run(tn, std::false_type{});
    };
    L.pre(kGradLogits);
    f32_narrow(p.N, vcur) ? by_cap(Int<32>{}) : by_cap(Int<64>{});
    L.post(kGradLogits);
    return hipGetLastError();
  }
  if (!p.compact) return hipErrorInvalidValue;
  if (lp_few_backward(p)) {
    const FewGrad f{a.idx, a.yc, &a.sc->n_valid, g.lse, g.entropy, g.grad_logp, g.grad_entropy,
                    g.rest, static_cast<uint16_t*>(a.g), p.V, v0, gemm::g_block(p)};
    auto go = [&](auto nt) {
      constexpr int NT = decltype(nt)::value;
      const auto* h = static_cast<const uint16_t*>(a.hc);
      const auto* W = static_cast<const uint16_t*>(a.W) + v0 * p.H;
      if (a.softcap > 0.f)
        hipLaunchKernelGGL((k_lp_few_grad<NT, true>), dim3(cdiv(vcur, 64)), dim3(256), 0, L.stream,
                           h, W, p.N, p.H, vcur, warp, f);
      else
        hipLaunchKernelGGL((k_lp_few_grad<NT, false>), dim3(cdiv(vcur, 64)), dim3(256), 0,
                           L.stream, h, W, p.N, p.H, vcur, warp, f);
    };
    L.pre(kGradLogits);
    if (p.N <= 16) go(Int<1>{});
    else if (p.N <= 32) go(Int<2>{});
    else if (p.N <= 64) go(Int<4>{});
    else go(Int<8>{});
    L.post(kGradLogits);
    return hipGetLastError();
  }
  constexpr int NF = gemm::kFormN;
  const gemm::Launch l = gemm::backward_launch(p, chunk, 0);
  auto run = [&](auto cap, auto split) {
    const EpiLpGrad<decltype(cap)::value, decltype(split)::value> epi{
        a.yc, g.lse_g, g.c0, g.c1, g.ca, p.N, p.V, v0, vcur, gemm::g_block(p), warp,
        static_cast<uint16_t*>(a.g), p.vchunk * p.ldg, g.rest};
    return run_gemm<NF, NF, kDynN>(l, a, epi, kGradLogits, L, &a.sc->n_valid);
  };
  using Y = std::true_type;
  using No = std::false_type;
  if (p.g_parts == 2) return a.softcap > 0.f ? run(Y{}, Y{}) : run(No{}, Y{});
  return a.softcap > 0.f ? run(Y{}, No{}) : run(No{}, No{});
}

}  // namespace flce
