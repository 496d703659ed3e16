// Sampling a token of each row of logits z [N][V] with temperature, top-k, top-p and min-p
// from one given uniform number a row:
//   x_i = softcap(z_i) / T,  w_i = exp(x_i - max x)
//   ranks: largest z first, equal ones by lowest index
//   kept: rank < k; then mass of the kept ranks above < p * mass of all kept; then w >= min_p
//   token = the first index i with sum over kept j <= i of w_j  >  u * sum over kept w_j
//
// All three filters keep the first ranks, so the kept set is a threshold: the keys above
// tau and the first m of those equal to it, in index order (a key is the logit's bits in an
// order of unsigned numbers). tau comes from a radix selection, by counts for top-k and by
// masses for top-p.
//
// Weights are whole numbers: w in 64-bit floating point times 2^S, rounded, with S as large
// as V weights' sum leaves in 62 bits (45 for 131072). Sums of whole numbers do not depend
// on their order, so the LDS atomics and the split over threads leave the same bits on
// every run, and which token a uniform number falls on is decided to 2^-S of the largest
// weight, not to a float's 2^-24 of the sum.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "flce_internal.h"
#include "ops_plan.h"
#include "row_io.h"
#include "wave_ops.h"

namespace flce {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBins = 2048;
constexpr double kLog2eD = 1.4426950408889634074;

__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);     // -0 is 0
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;       // order_key(-inf)

// 2^t for t in (-1022, 0]: 2^n 2^f with |f| <= 1/2, the exponential's series to f^11 (what
// it leaves out is below 2^-47).
__device__ __forceinline__ double exp2_neg(double t) {
  const double n = __builtin_rint(t), y = (t - n) * 0.69314718055994530942;
  double s = 1.0 / 39916800;
  s = fma(s, y, 1.0 / 3628800);
  s = fma(s, y, 1.0 / 362880);
  s = fma(s, y, 1.0 / 40320);
  s = fma(s, y, 1.0 / 5040);
  s = fma(s, y, 1.0 / 720);
  s = fma(s, y, 1.0 / 120);
  s = fma(s, y, 1.0 / 24);
  s = fma(s, y, 1.0 / 6);
  s = fma(s, y, 0.5);
  s = fma(s, y, 1.0);
  s = fma(s, y, 1.0);
  return __builtin_ldexp(s, int(n));
}

// A row's weights.
struct Weights {
  double cap, inv_cap, xmax, scale;                // scale: log2(e) / T
  float zmax;
  int S;
  double min_p;
  __device__ __forceinline__ double warp(float z) const {
    return cap > 0.0 ? cap * tanh(double(z) * inv_cap) : double(z);
  }
  // w of a logit, at most 1; zero below 2^-(S + 1), for -inf, and next to a logit of +inf.
  __device__ __forceinline__ double weight(float z) const {
    if (z == zmax) return 1.0;
    if (z == -INFINITY) return 0.0;                // also where a softcap makes it finite
    const double t = (warp(z) - xmax) * scale;
    return t > -(S + 1.0) ? exp2_neg(t) : 0.0;
  }
  __device__ __forceinline__ uint64_t fixed(double w) const {
    // w 2^S + 2^52 has its whole part, rounded to nearest, in its low 52 bits
    return __builtin_bit_cast(uint64_t, __builtin_ldexp(w, S) + 4503599627370496.0) &
           0xfffffffffffffull;
  }
  __device__ __forceinline__ uint64_t mass(float z) const { return fixed(weight(z)); }
  // ... after min-p
  __device__ __forceinline__ uint64_t kept(float z) const {
    const double w = weight(z);
    return w >= min_p ? fixed(w) : 0;
  }
};

struct Shared {
  uint64_t hist[kBins];
  uint64_t wave_sum[kWaves];
  uint32_t wave_cnt[kWaves];
  uint64_t above;
  uint32_t bin;
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) {
  const uint32_t lo = __shfl_up(uint32_t(v), d), hi = __shfl_up(uint32_t(v >> 32), d);
  return uint64_t(hi) << 32 | lo;
}
// Sum over the lanes up to this one.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t o = shfl_up64(v, d);
    if (lane >= d) v += o;
  }
  return v;
}
__device__ __forceinline__ uint64_t wave_sum(uint64_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t lo = __shfl_xor(uint32_t(v), d), hi = __shfl_xor(uint32_t(v >> 32), d);
    v += uint64_t(hi) << 32 | lo;
  }
  return v;
}

// The row's elements [lo, hi) dealt to `count` threads in 16-byte chunks, f(z) for each.
template <class T, class F>
__device__ __forceinline__ void for_each(const T* row, int64_t lo, int64_t hi, int t, int count,
                                         F f) {
  constexpr int E = kPerChunk<T>;
  for (int64_t c = lo + int64_t(t) * E; c < hi; c += int64_t(count) * E) {
    float v[E];
    load_chunk(row, c, hi, v);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (c + e < hi) f(v[e], c + e);
  }
}

// With the histogram's bins, highest first, summed up: the bin in which the sum passes
// `target` (above < target <= above + bin; target 1 .. total), in sm.bin, sm.above. If
// target is a share (by p of the total), it is formed here. Returns the target.
__device__ __forceinline__ uint64_t find_bin(Shared& sm, uint64_t target, double p, bool share) {
  constexpr int kEach = kBins / kThreads;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  __syncthreads();
  uint64_t v[kEach], sum = 0;
#pragma unroll
  for (int i = 0; i < kEach; ++i) sum += v[i] = sm.hist[kBins - 1 - (tid * kEach + i)];
  const uint64_t incl = wave_scan(sum, lane);
  if (lane == 63) sm.wave_sum[w] = incl;
  __syncthreads();
  uint64_t before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    if (i < w) before += sm.wave_sum[i];
    total += sm.wave_sum[i];
  }
  if (share) {
    const double r = __builtin_ceil(p * double(total));
    target = r >= double(total) ? total : r >= 1.0 ? uint64_t(r) : 1;
  }
  uint64_t at = before + incl - sum;
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    if (at < target && target <= at + v[i]) {
      sm.bin = kBins - 1 - (tid * kEach + i);
      sm.above = at;
    }
    at += v[i];
  }
  __syncthreads();
  return target;
}

// The key tau at which the sum of add(z) over the row's keys, highest first, passes
// `target`, and the sum above it. extra: added once for key extra_key.
template <class T, class Add>
__device__ __forceinline__ uint32_t select_key(const T* row, int64_t V, Shared& sm,
                                               uint64_t& target, double p, bool share,
                                               uint64_t& above, uint32_t extra_key,
                                               uint64_t extra, Add add) {
  uint32_t prefix = 0, mask = 0;
  above = 0;
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0, bits = digit < 2 ? 11 : 10;
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    auto count = [&](uint32_t key, uint64_t v) {
      if (v && (key & mask) == prefix)
        atomicAdd(reinterpret_cast<unsigned long long*>(
                      &sm.hist[(key >> shift) & ((1u << bits) - 1)]),
                  static_cast<unsigned long long>(v));
    };
    for_each(row, 0, V, threadIdx.x, kThreads, [&](float z, int64_t) {
      const uint32_t key = order_key(z);
      if ((key & mask) == prefix) count(key, add(z, key));
    });
    if (threadIdx.x == 0) count(extra_key, extra);
    target = find_bin(sm, target - above, p, share && digit == 0) + above;
    prefix |= sm.bin << shift;
    mask |= ((1u << bits) - 1) << shift;
    above += sm.above;
    __syncthreads();
  }
  return prefix;
}

// A workgroup a row.
template <class T>
__global__ __launch_bounds__(kThreads) void k_sample(SampleArgs a) {
  __shared__ Shared sm;
  constexpr int E = kPerChunk<T>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = blockIdx.x, V = a.V;
  const T* row = static_cast<const T*>(a.logits) + r * a.ld;

  // the largest logit; a row of -inf alone or with a NaN has no token
  uint32_t best = 0;
  bool nan = false;
  for_each(row, 0, V, tid, kThreads, [&](float z, int64_t) {
    if (z != z) nan = true;
    else best = MaxOp()(best, order_key(z));
  });
  best = wave_all(best, MaxOp());
  if (lane == 0) {
    sm.wave_cnt[wave] = best;
    sm.wave_sum[wave] = 0;
  }
  __syncthreads();
  if (nan) sm.wave_sum[wave] = 1;
  __syncthreads();
  best = 0;
  nan = false;
#pragma unroll
  for (int i = 0; i < kWaves; ++i) {
    best = MaxOp()(best, sm.wave_cnt[i]);
    nan |= sm.wave_sum[i] != 0;
  }
  __syncthreads();                                 // read before they are written again
  if (nan || best <= kKeyNegInf) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logp) a.logp[r] = nan ? NAN : -INFINITY;
    }
    return;
  }

  const float T_ = a.temperature.at(r);
  int64_t k = a.top_k.at(r);
  if (k <= 0 || k > V) k = V;
  if (!(T_ > 0.f)) k = 1;
  Weights wt;
  wt.cap = a.softcap;
  wt.inv_cap = a.softcap > 0.f ? 1.0 / a.softcap : 0.0;
  wt.zmax = key_value(best);
  wt.xmax = wt.warp(wt.zmax);
  wt.scale = T_ > 0.f ? kLog2eD / double(T_) : 0.0;
  wt.S = a.weight_bits;
  wt.min_p = fmin(fmax(double(a.min_p.at(r)), 0.0), 1.0);
  const double p = fmax(double(a.top_p.at(r)), 0.0);

  uint32_t tau = 0;
  uint64_t m = ~0ull >> 1;                         // keys equal to tau that are kept
  if (k == 1) {
    tau = best;
    m = 1;
  } else if (k < V) {
    uint64_t above, target = uint64_t(k);
    tau = select_key(row, V, sm, target, 0.0, false, above, 0u, 0ull,
                     [](float, uint32_t) { return uint64_t(1); });
    m = uint64_t(k) - above;
  }
  if (k > 1 && p < 1.0) {
    uint64_t above, target = 0;
    const uint64_t w_tau = tau ? wt.mass(key_value(tau)) : 0;
    const uint32_t tau_k = tau;
    tau = select_key(row, V, sm, target, p, true, above, tau_k, tau_k ? m * w_tau : 0,
                     [&](float z, uint32_t key) { return key > tau_k ? wt.mass(z) : 0; });
    const uint64_t w = wt.mass(key_value(tau));
    const uint64_t need = (target - above + w - 1) / w;
    m = tau == tau_k && m < need ? m : need;
  }
  // masses and counts of equal keys before a place: the mass kept there
  const uint64_t w_tau = tau ? wt.kept(key_value(tau)) : 0;
  auto mass_at = [&](uint64_t sum, uint64_t ties) { return sum + (ties < m ? ties : m) * w_tau; };

  // the token: the row's sixteenth that holds the target, its sixteenth, and so on
  int64_t lo = 0, len = V;
  uint64_t sum0 = 0, tie0 = 0, target = 0, total = 0;
  bool first = true;
  do {
    const int64_t part = (((len + kWaves - 1) / kWaves) + E - 1) / E * E;
    const int64_t from = lo + wave * part;
    const int64_t to = from + part < lo + len ? from + part : lo + len;
    uint64_t sum = 0;
    uint32_t ties = 0;
    for_each(row, from, to, lane, 64, [&](float z, int64_t) {
      const uint32_t key = order_key(z);
      if (key > tau) sum += wt.kept(z);
      else if (key == tau) ++ties;
    });
    sum = wave_sum(sum);
    ties = uint32_t(wave_sum(ties));
    if (lane == 0) {
      sm.wave_sum[wave] = sum;
      sm.wave_cnt[wave] = ties;
    }
    __syncthreads();
    if (first) {
      uint64_t s = 0, t = 0;
      for (int i = 0; i < kWaves; ++i) {
        s += sm.wave_sum[i];
        t += sm.wave_cnt[i];
      }
      total = mass_at(s, t);
      const double u = fmin(fmax(double(a.uniforms[r]), 0.0), 1.0) * double(total);
      target = u >= double(total) ? total - 1 : uint64_t(u);
      if (target >= total) target = total - 1;
      first = false;
    }
    int64_t next = lo, rest = len;
    for (int i = 0; i < kWaves; ++i) {
      const uint64_t s = sum0 + sm.wave_sum[i], t = tie0 + sm.wave_cnt[i];
      next = lo + i * part;
      rest = lo + len - next < part ? lo + len - next : part;
      if (target < mass_at(s, t)) break;
      sum0 = s;
      tie0 = t;
    }
    lo = next;
    len = rest;
    __syncthreads();
  } while (len > 64);
  if (wave == 0) {
    const float z = lane < len ? to_f32(row[lo + lane]) : -INFINITY;
    const uint32_t key = lane < len ? order_key(z) : 0;
    const uint64_t s = sum0 + wave_scan(lane < len && key > tau ? wt.kept(z) : 0, lane);
    const uint64_t t = tie0 + wave_scan(lane < len && key == tau ? 1 : 0, lane);
    const uint64_t hit = __ballot(target < mass_at(s, t));
    const int at = hit ? __builtin_ctzll(hit) : 0;
    if (lane == at) {
      a.tokens[r] = lo + at;
      if (a.logp) {
        const double x = z == wt.zmax ? 0.0 : (wt.warp(z) - wt.xmax) * wt.scale;
        a.logp[r] = float(x / kLog2eD - log(__builtin_ldexp(double(total), -wt.S)));
      }
    }
  }
}

template <class T>
hipError_t sample(const SampleArgs& a, const Launcher& L) {
  L.pre(kSample);
  hipLaunchKernelGGL(k_sample<T>, dim3(unsigned(a.N)), dim3(kThreads), 0, L.stream, a);
  L.post(kSample);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, const Launcher& L) {
  return a.dtype == FLCE_F32 ? sample<float>(a, L) : sample<Bf16Bits>(a, L);
}

}  // namespace flce
