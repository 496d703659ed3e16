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
//
// A workgroup takes a row. Its waves take contiguous sixteenths of it (segments), so that
// sums by wave are sums by place. The first pass finds the largest logit; what follows
// depends on what can be ruled out before the selection:
// - top-k: the k-th largest of the threads' own maxima is a bound that few logits but the
//   first k pass (where the maxima of each 64 or 128 logits are at hand, from the head's
//   product or, for few long rows, a kernel before this one, those are read in the logits'
//   place, and the parts that reach the bound). Those are collected in LDS, in index
//   order, and everything else is done on the list. min-p alone bounds the list in the same way.
// - top-p without top-k: one pass forms all weights and adds them up by bins of an eighth
//   of a power of two, for each wave; the bin in which the mass passes p is then collected,
//   and the selection runs on that.
// - no filter: one pass sums the weights of each segment.
// The token is then found in the segment that holds it. A list that does not fit (thousands
// of equal logits, or a k near the 1024 threads, whose bound then keeps a good part of a long
// row) or a k above them leaves the row to the selection over the whole row.
//
// Top-p without top-k is bound by the vector units: 256 rows of 131072 float32 take 102 us
// (134 MB; at the memory's rate 26), of which the maximum takes 19, the weights in 64 bits
// 37, collecting and selecting 27, the token 9. A selection over whole rows, three digits of
// counts and three of masses, took 239. Keeping each logit's bin as a byte in LDS, so that
// collecting reads no memory, gave 97, and 2 us more for rows of 32000: not kept. Top-k is
// bound by latency: one row of 131072 18 us (4 of them the maxima), 128 bf16 rows of 32000
// with settings of their own 22 to 30, by the settings drawn.
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
constexpr int kBins = 2048;                        // of a radix selection's digit
constexpr int kMassBins = 384;                     // of weights: eighths of 2^-48 .. 1
constexpr int kWaveList = 256;                     // candidates a wave collects
// A list up to this long is ranked by counting, a longer one by digits (us, 1 row of 131072
// and 256 of 32000 float32: top-50 18 and 24, 23 and 30; top-100 22 and 26, 27 and 31; top-150
// 27 and 27, 31 and 31; top-250 38 and 29, 41 and 32).
constexpr int kSmallList = 256;
constexpr int kMaximaChunks = 4;                   // a thread of k_sample_maxima loads
constexpr double kLog2eD = 1.4426950408889634074;

__device__ __forceinline__ uint32_t order_key(float z) {
  const uint32_t b = __float_as_uint(z + 0.f);     // -0 is 0
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}
constexpr uint32_t kKeyNegInf = 0x007fffffu;       // order_key(-inf)

// 2^(t + up) for t in [-1000, 0]: 2^n 2^f with |f| <= 1/2, and 2^f by the polynomial of
// degree 10 through its values at the Chebyshev points (off by 2^-51).
__device__ __forceinline__ double exp2_neg(double t, int up = 0) {
  const double n = __builtin_rint(t), f = t - n;
  double s = 7.072585949269224e-09;
  s = fma(s, f, 1.0208690299958306e-07);
  s = fma(s, f, 1.321544258792169e-06);
  s = fma(s, f, 1.5252657260200837e-05);
  s = fma(s, f, 0.0001540353044173605);
  s = fma(s, f, 0.0013333558230164974);
  s = fma(s, f, 0.009618129107606888);
  s = fma(s, f, 0.05550410866444772);
  s = fma(s, f, 0.24022650695910097);
  s = fma(s, f, 0.69314718055995);
  s = fma(s, f, 1.0);
  return __builtin_ldexp(s, int(n) + up);
}

// A row's weights. CAP: logits are capped first.
template <bool CAP>
struct Weights {
  double cap, two_inv_cap, xmax, scale;            // scale: log2(e) / T
  int S;
  double min_p, log_min_p;                         // log_min_p: for a first look
  // cap tanh(z / cap) = sign cap (1 - e) / (1 + e), e = exp(-2 |z| / cap): off by a few 2^-53
  // of cap, which is all that a difference to xmax needs. A logit of -inf stays.
  __device__ __forceinline__ double warp(float z) const {
    if constexpr (!CAP) return double(z);
    const double t = fmax(fabs(double(z)) * two_inv_cap * -kLog2eD, -1000.0), e = exp2_neg(t);
    return z == -INFINITY ? -INFINITY : copysign(cap * ((1.0 - e) / (1.0 + e)), double(z));
  }
  // log2 of w of a logit, or -64 where that is lower (w is then zero): so for -inf, and for
  // all others next to one of +inf, whose difference to itself, a NaN, counts as 0.
  __device__ __forceinline__ double log_weight(float z) const {
    return fmax(fmin((warp(z) - xmax) * scale, 0.0), -64.0);
  }
  __device__ __forceinline__ double weight(float z) const { return exp2_neg(log_weight(z)); }
  // w 2^S + 2^52 has its whole part, rounded to nearest, in its low 52 bits
  __device__ __forceinline__ uint64_t whole(double w_s) const {
    return __builtin_bit_cast(uint64_t, w_s + 4503599627370496.0) & 0xfffffffffffffull;
  }
  __device__ __forceinline__ uint64_t fixed_of(double log_w) const {
    return whole(exp2_neg(log_w, S));
  }
  __device__ __forceinline__ uint64_t mass(float z) const { return fixed_of(log_weight(z)); }
  __device__ __forceinline__ bool reaches_min_p(float z) const {
    const double t = log_weight(z);
    return t > log_min_p - 1e-6 && exp2_neg(t) >= min_p;
  }
  // ... after min-p
  __device__ __forceinline__ uint64_t kept(float z) const {
    const double w = weight(z);
    return w >= min_p ? whole(__builtin_ldexp(w, S)) : 0;
  }
};

struct Shared {
  union {
    uint64_t hist[kBins];
    uint64_t mass[kWaves][kMassBins];
  };
  uint32_t key[kWaves * kWaveList], idx[kWaves * kWaveList];   // a list, in index order
  uint64_t wave_sum[kWaves];
  uint32_t wave_cnt[kWaves];
  uint64_t above;
  uint32_t bin, found;
};

// A row in memory.
constexpr int kLaneMost = 8;                       // values of a lane in descend()
template <class T>
struct Row {
  static constexpr int E = kPerChunk<T>;
  const T* p;
  int64_t n;
  __device__ __forceinline__ float at(int64_t i) const { return to_f32(p[i]); }
  // The chunk at c (a multiple of E) of [.., hi), without a condition on the load: at the
  // end of the range, or behind it, the range's last E values are read instead. Value e is
  // that of index i + e, and belongs to the chunk for e >= the result.
  __device__ __forceinline__ int chunk(int64_t c, int64_t hi, float (&v)[E], int64_t& i) const {
    i = c + E <= hi ? c : hi - E;
    unpack_chunk<T>(load_raw(p + i), v);
    return c - i < E ? int(c - i) : E;
  }
  // f(u, values, index of the first, the first that counts) for the chunks u = 0 .. U - 1 of
  // each turn that lane t of `count` takes of [lo, hi), all under way at once, and end() behind
  // every turn; lo is a multiple of E. What whole turns leave goes chunk by chunk.
  template <int U, class F, class End>
  __device__ __forceinline__ void turns(int64_t lo, int64_t hi, int t, int count, F f,
                                        End end) const {
    const int64_t step = int64_t(count) * E;
    if (hi < E) {                                  // fewer values than a chunk: -inf behind them
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = e < hi ? at(e) : -INFINITY;
      f(0, v, int64_t(0), lo == 0 && t == 0 ? 0 : E);
      end();
      return;
    }
    int64_t base = lo;
    const T* q = p + lo + int64_t(t) * E;
#pragma unroll 1
    for (; base + U * step <= hi; base += U * step, q += U * step) {
      row_u32x4 raw[U];
#pragma unroll
      for (int u = 0; u < U; ++u) raw[u] = load_raw(q + u * step);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[E];
        unpack_chunk<T>(raw[u], v);
        f(u, v, base + (u * count + t) * int64_t(E), 0);
      }
      end();
    }
#pragma unroll 1
    for (; base < hi; base += step) {
      float v[E];
      int64_t i;
      const int e0 = chunk(base + t * int64_t(E), hi, v, i);
      f(0, v, i, e0);
      end();
    }
  }
  template <int U = 4, class F>
  __device__ __forceinline__ void each(int64_t lo, int64_t hi, int t, int count, F f) const {
    turns<U>(lo, hi, t, count, [&](int, const float (&v)[E], int64_t i, int e0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= e0) f(v[e], i + e);
    }, [] {});
  }
};

// The list in LDS.
struct List {
  static constexpr int E = 1;
  const uint32_t* key;
  int64_t n;
  __device__ __forceinline__ float at(int64_t i) const { return key_value(key[i]); }
  template <class F>
  __device__ __forceinline__ void each(int64_t lo, int64_t hi, int t, int count, F f) const {
    for (int64_t i = lo + t; i < hi; i += count) f(key_value(key[i]), i);
  }
};

// The sum of the waves' sm.wave_sum before wave w, and of all.
__device__ __forceinline__ uint64_t before_wave(const Shared& sm, int w, uint64_t& total) {
  const int lane = threadIdx.x & 63;
  const uint64_t v = lane < kWaves ? sm.wave_sum[lane] : 0, s = wave_scan64(v);
  total = from_lane64(s, kWaves - 1);
  return from_lane64(s - v, __builtin_amdgcn_readfirstlane(w));
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
  const uint64_t incl = wave_scan64(sum);
  if (lane == 63) sm.wave_sum[w] = incl;
  __syncthreads();
  uint64_t total;
  const uint64_t before = before_wave(sm, w, total);
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

// The key tau at which the sum of add(z) over the source's keys, highest first, passes
// `target`, and the sum above it. extra: added once for key extra_key. The keys share
// their bits above the lowest `bits`, which are those of `prefix`.
template <class Src, class Add>
__device__ __forceinline__ uint32_t select_key(const Src& src, Shared& sm,
                                               uint64_t& target, double p, bool share,
                                               uint64_t& above, uint32_t extra_key,
                                               uint64_t extra, Add add, int left = 32,
                                               uint32_t prefix = 0) {
  uint32_t mask = left < 32 ? ~0u << left : 0;
  above = 0;
  bool first = true;
#pragma unroll 1
  while (left > 0) {
    const int bits = left < 11 ? left : 11, shift = left - bits;
    left = shift;
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    auto count = [&](uint32_t key, uint64_t v) {
      if (v && (key & mask) == prefix)
        atomicAdd(reinterpret_cast<unsigned long long*>(
                      &sm.hist[(key >> shift) & ((1u << bits) - 1)]),
                  static_cast<unsigned long long>(v));
    };
    src.each(0, src.n, threadIdx.x, kThreads, [&](float z, int64_t) {
      const uint32_t key = order_key(z);
      if ((key & mask) == prefix) count(key, add(z, key));
    });
    if (threadIdx.x == 0) count(extra_key, extra);
    target = find_bin(sm, target - above, p, share && first) + above;
    first = false;
    prefix |= sm.bin << shift;
    mask |= ((1u << bits) - 1) << shift;
    above += sm.above;
    __syncthreads();
  }
  return prefix;
}

// What is kept of a row's keys: those above tau and the first m equal to it, of both those
// whose weight is at least min-p.
struct Kept {
  uint32_t tau = 0;
  uint64_t m = ~0ull >> 1;
};

// top-k and then top-p over a source that holds at least the first k ranks.
template <class Src, bool CAP>
__device__ __forceinline__ Kept select(const Src& src, Shared& sm, const Weights<CAP>& wt, int64_t k,
                                       double p) {
  Kept s;
  if (k < src.n) {
    uint64_t above, target = uint64_t(k);
    s.tau = select_key(src, sm, target, 0.0, false, above, 0u, 0ull,
                       [](float, uint32_t) { return uint64_t(1); });
    s.m = uint64_t(k) - above;
  }
  if (p < 1.0) {
    uint64_t above, target = 0;
    const uint64_t w_tau = s.tau ? wt.mass(key_value(s.tau)) : 0;
    const uint32_t tau_k = s.tau;
    s.tau = select_key(src, sm, target, p, true, above, tau_k, tau_k ? s.m * w_tau : 0,
                       [&](float z, uint32_t key) { return key > tau_k ? wt.mass(z) : 0; });
    const uint64_t w = wt.mass(key_value(s.tau));
    const uint64_t need = (target - above + w - 1) / w;
    s.m = s.tau == tau_k && s.m < need ? s.m : need;
  }
  return s;
}

// Where the target lies: the mass and the count of keys equal to tau before [lo, lo + len).
struct Place {
  int64_t lo, len;
  uint64_t sum, ties;
};

__device__ __forceinline__ uint64_t target_of(float uniform, uint64_t total) {
  const double u = fmin(fmax(double(uniform), 0.0), 1.0) * double(total);
  const uint64_t t = u >= double(total) ? total - 1 : uint64_t(u);
  return t < total ? t : total - 1;
}

// With every wave's kept mass and ties of part i of `at` in sm.wave_sum[i], sm.wave_cnt[i]:
// the part that holds the target. total = 0: first call, which forms total and target.
__device__ __forceinline__ int enter(Place& at, int64_t part, Shared& sm, const Kept& s,
                                     uint64_t w_tau, float uniform, uint64_t& total,
                                     uint64_t& target) {
  auto mass_at = [&](uint64_t sum, uint64_t ties) { return sum + (ties < s.m ? ties : s.m) * w_tau; };
  __syncthreads();
  // lane i: up to and with part i
  const int lane = threadIdx.x & 63;
  const uint64_t a0 = lane < kWaves ? sm.wave_sum[lane] : 0, c0 = lane < kWaves ? sm.wave_cnt[lane] : 0;
  const uint64_t a = at.sum + wave_scan64(a0), c = at.ties + wave_scan64(c0);
  __syncthreads();
  if (total == 0) {
    total = from_lane64(mass_at(a, c), 63);
    target = target_of(uniform, total);
  }
  const uint64_t past = __ballot(lane < kWaves && mass_at(a, c) <= target);
  const int part_of = __popcll(past) < kWaves ? __popcll(past) : kWaves - 1;
  at.sum = from_lane64(a - a0, part_of);
  at.ties = from_lane64(c - c0, part_of);
  at.lo += part_of * part;
  at.len -= part_of * part;
  if (at.len > part) at.len = part;
  return part_of;
}

// The source's index that the target falls on. A long place is first cut to its sixteenth
// that holds the target; then every lane takes up to kLaneMost consecutive values, and the
// wave whose values hold it finds the lane and the value.
template <class Src, bool CAP>
__device__ __forceinline__ int64_t descend(const Src& src, Place at, Shared& sm,
                                           const Weights<CAP>& wt, const Kept& s, float uniform,
                                           uint64_t& total, uint64_t target) {
  constexpr int E = Src::E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t w_tau = s.tau ? wt.kept(key_value(s.tau)) : 0;
  auto put = [&](uint64_t sum, uint64_t ties) {
    if (lane == 0) {
      sm.wave_sum[wave] = sum;
      sm.wave_cnt[wave] = uint32_t(ties);
    }
  };
  while (at.len > kThreads * kLaneMost) {
    const int64_t part = (((at.len + kWaves - 1) / kWaves) + E - 1) / E * E;
    const int64_t from = at.lo + wave * part, end = at.lo + at.len;
    uint64_t sum = 0;
    uint32_t ties = 0;
    if (from < end)
      src.each(from, from + part < end ? from + part : end, lane, 64, [&](float z, int64_t) {
        const uint32_t key = order_key(z);
        if (key > s.tau) sum += wt.kept(z);
        else if (key == s.tau) ++ties;
      });
    put(wave_sum64(sum), wave_sum64(ties));
    enter(at, part, sm, s, w_tau, uniform, total, target);
  }
  const int64_t per = ((at.len + kThreads - 1) / kThreads + E - 1) / E * E;
  const int64_t end = at.lo + at.len, lo = at.lo + threadIdx.x * per;
  const int64_t hi = lo + per < end ? lo + per : end;
  uint64_t sum = 0, own_ties = 0;
#pragma unroll 1
  for (int64_t i = lo; i < hi; ++i) {
    const float z = src.at(i);
    const uint32_t key = order_key(z);
    if (key > s.tau) sum += wt.kept(z);
    else if (key == s.tau) ++own_ties;
  }
  uint64_t sums = wave_scan64(sum), ties = wave_scan64(own_ties);
  put(from_lane64(sums, 63), from_lane64(ties, 63));
  const int part_of = enter(at, 64 * per, sm, s, w_tau, uniform, total, target);
  if (wave == part_of) {
    auto mass_at = [&](uint64_t a, uint64_t c) { return a + (c < s.m ? c : s.m) * w_tau; };
    sums += at.sum;
    ties += at.ties;
    const uint64_t hit = __ballot(target < mass_at(sums, ties));
    if (lane == (hit ? __builtin_ctzll(hit) : 63)) {
      uint64_t a = sums - sum, c = ties - own_ties;
      int64_t i = lo;
#pragma unroll 1
      for (; i < hi - 1; ++i) {
        const float z = src.at(i);
        const uint32_t key = order_key(z);
        if (key > s.tau) a += wt.kept(z);
        else if (key == s.tau) ++c;
        if (target < mass_at(a, c)) break;
      }
      sm.found = uint32_t(i);
    }
  }
  __syncthreads();
  return sm.found;
}

// The list's index for a list of up to kSmallList that holds the first k ranks: each thread
// counts the ranks above its own, and their mass.
template <bool CAP>
__device__ __forceinline__ int64_t small_list(Shared& sm, int n, const Weights<CAP>& wt, int64_t k,
                                              double p, float uniform, uint64_t& total) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint64_t* mass = sm.hist;
  const float z = tid < n ? key_value(sm.key[tid]) : 0.f;
  const double lw = tid < n ? wt.log_weight(z) : -64.0;
  const uint64_t own = tid < n ? wt.fixed_of(lw) : 0;
  if (tid < kSmallList) mass[tid] = own;
  __syncthreads();
  bool keep = tid < n;
  uint64_t above = 0;
  if (wave * 64 < n) {
    const uint32_t key = tid < n ? sm.key[tid] : 0;
    int rank = 0;
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const uint32_t o = sm.key[j];
      const bool better = o > key || (o == key && j < tid);
      rank += better;
      above += better ? mass[j] : 0;
    }
    keep = keep && rank < k;
  }
  auto block_sum = [&](uint64_t v, uint64_t& before) {      // v: sums along each wave
    if (lane == 63) sm.wave_sum[wave] = v;
    __syncthreads();
    uint64_t all;
    before = before_wave(sm, wave, all);
    __syncthreads();
    return all;
  };
  uint64_t before;
  if (p < 1.0) {
    const uint64_t all = block_sum(wave_scan64(keep ? own : 0), before);
    const double r = __builtin_ceil(p * double(all));
    const uint64_t limit = r >= double(all) ? all : r >= 1.0 ? uint64_t(r) : 1;
    keep = keep && above < limit;
  }
  keep = keep && exp2_neg(lw) >= wt.min_p;
  const uint64_t incl = wave_scan64(keep ? own : 0);
  total = block_sum(incl, before);
  const uint64_t target = target_of(uniform, total);
  const uint64_t upto = before + incl;
  if (keep && own && upto > target && upto - own <= target) sm.found = tid;
  __syncthreads();
  return sm.found;
}

// With `have` indices of each wave, in order, in its place of sm.idx (at most kWaveList are
// there): all of them and their keys from the front on. Returns how many, or -1 if a wave
// found more than its place holds.
template <class T>
__device__ __forceinline__ int close_gaps(const Row<T>& row, Shared& sm, int have) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t* idx = sm.idx + wave * kWaveList;
  if (lane == 0) sm.wave_sum[wave] = uint64_t(have);
  __syncthreads();
  uint64_t n;
  const int start = int(before_wave(sm, wave, n));
  const bool fits = __ballot(lane < kWaves && sm.wave_sum[lane & (kWaves - 1)] > kWaveList) == 0;
  // every wave reads its place before any writes
  uint32_t x[kWaveList / 64];
#pragma unroll
  for (int i = 0; i < kWaveList / 64; ++i) x[i] = idx[i * 64 + lane];
  __syncthreads();
  if (!fits) return -1;
#pragma unroll
  for (int i = 0; i < kWaveList / 64; ++i)
    if (i * 64 + lane < have) {
      sm.idx[start + i * 64 + lane] = x[i];
      sm.key[start + i * 64 + lane] = order_key(row.at(x[i]));
    }
  __syncthreads();
  return int(n);
}

// The row's logits for which take(z, i) holds, in index order, into sm.key and sm.idx. Each
// wave first fills a place of its own from its segment. Returns how many, or -1 if a wave
// found more than its place holds.
template <class T, class Take>
__device__ __forceinline__ int collect(const Row<T>& row, int64_t seg, Shared& sm, Take take) {
  constexpr int E = Row<T>::E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t from = wave * seg, to = from + seg < row.n ? from + seg : row.n;
  const uint64_t below = (1ull << lane) - 1;
  uint32_t* idx = sm.idx + wave * kWaveList;
  constexpr int U = 32 / E;                        // a bit a value
  int have = 0;
  uint32_t mine = 0;
  int64_t at[U];
  if (from < to)
    row.template turns<U>(from, to, lane, 64, [&](int u, const float (&v)[E], int64_t i, int e0) {
      at[u] = i;
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (e >= e0 && take(v[e])) mine |= 1u << (u * E + e);
    }, [&] {
      if (__ballot(mine != 0) != 0) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t m = (mine >> (u * E)) & ((1u << E) - 1);
          if (__ballot(m != 0) == 0) continue;
          int before = 0, all = 0;
#pragma unroll 1
          for (int e = 0; e < E; ++e) {
            const uint64_t b = __ballot((m >> e) & 1);
            before += __popcll(b & below);
            all += __popcll(b);
          }
          for (int to_ = have + before; m != 0; m &= m - 1, ++to_)
            if (to_ < kWaveList) idx[to_] = uint32_t(at[u] + __builtin_ctz(m));
          have += all;
        }
        mine = 0;
      }
    });
  return close_gaps(row, sm, have);
}

// The row's keys of at least `bound` in the parts whose maxima reach it, as collect(): wave w
// looks at the parts from w bseg on.
template <class T>
__device__ __forceinline__ int collect_parts(const Row<T>& row, const SampleArgs& a,
                                             const float* maxima, int64_t bseg, uint32_t bound,
                                             Shared& sm) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t below = (1ull << lane) - 1;
  uint32_t* idx = sm.idx + wave * kWaveList;
  const int64_t first = wave * bseg, last = first + bseg < a.blocks ? first + bseg : a.blocks;
  int have = 0;
  for (int64_t b0 = first; b0 < last; b0 += 64) {
    const bool in = b0 + lane < last;
    uint64_t parts = __ballot(in && order_key(in ? maxima[b0 + lane] : 0.f) >= bound);
    for (; parts != 0; parts &= parts - 1) {
      const int64_t at = (b0 + __builtin_ctzll(parts)) * a.block;
      for (int64_t i = at + lane; i - lane < at + a.block; i += 64) {
        const bool take = i < row.n && order_key(row.at(i < row.n ? i : 0)) >= bound;
        const uint64_t hits = __ballot(take);
        const int to = have + __popcll(hits & below);
        if (take && to < kWaveList) idx[to] = uint32_t(i);
        have += __popcll(hits);
      }
    }
  }
  return close_gaps(row, sm, have);
}

// The same in any order within a wave's place, which keep their gaps: wave w's are
// sm.wave_cnt[w] from w kWaveList on. False if a wave found more than its place holds.
template <class T, class Take>
__device__ __forceinline__ bool gather(const Row<T>& row, int64_t seg, Shared& sm, Take take) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t from = wave * seg, to = from + seg < row.n ? from + seg : row.n;
  if (lane == 0) sm.wave_cnt[wave] = 0;
  if (from < to)
    row.template each<8>(from, to, lane, 64, [&](float z, int64_t) {
      if (take(z)) {
        const uint32_t at = atomicAdd(&sm.wave_cnt[wave], 1u);
        if (at < kWaveList) sm.key[wave * kWaveList + at] = order_key(z);
      }
    });
  __syncthreads();
  return __ballot(sm.wave_cnt[lane & (kWaves - 1)] > uint32_t(kWaveList)) == 0;
}

// What gather() left, as a source without an order.
struct Gathered {
  const Shared& sm;
  int64_t n;
  template <class F>
  __device__ __forceinline__ void each(int64_t, int64_t, int t, int, F f) const {
    const int lane = t & 63, wave = t >> 6;
    for (uint32_t i = lane; i < sm.wave_cnt[wave]; i += 64)
      f(key_value(sm.key[wave * kWaveList + i]), int64_t(0));
  }
};

// A key that at least k of the threads' maxima reach (0 if fewer have one): the k-th
// largest's upper 22 bits.
__device__ __forceinline__ uint32_t bound_of_maxima(uint32_t own, int64_t k, Shared& sm) {
  uint32_t prefix = 0, mask = 0;
  uint64_t above = 0;
#pragma unroll 1
  for (int digit = 0; digit < 2; ++digit) {
    const int shift = digit == 0 ? 21 : 10;
    for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    if (own > kKeyNegInf && (own & mask) == prefix)
      atomicAdd(reinterpret_cast<unsigned long long*>(&sm.hist[(own >> shift) & (kBins - 1)]), 1ull);
    if (threadIdx.x == 0) sm.bin = kBins;
    find_bin(sm, uint64_t(k) - above, 0.0, false);
    if (sm.bin == kBins) return 0;                 // fewer than k (at the first digit)
    prefix |= sm.bin << shift;
    mask |= uint32_t(kBins - 1) << shift;
    above += sm.above;
    __syncthreads();
  }
  return prefix;
}

// A workgroup a row.
template <class T, bool CAP>
__global__ __launch_bounds__(kThreads) void k_sample(SampleArgs a) {
  __shared__ Shared sm;
  constexpr int E = kPerChunk<T>;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t r = blockIdx.x;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.ld, a.V};
  const int64_t V = a.V, part = (V + kWaves - 1) / kWaves, seg = (part + E - 1) / E * E;
  const int64_t from = wave * seg, to = from + seg < V ? from + seg : V;

  const float T_ = a.temperature.at(r), uniform = a.uniforms[r];
  int64_t k = a.top_k.at(r);
  if (k <= 0 || k > V) k = V;
  if (!(T_ > 0.f)) k = 1;

  // the largest logit; a row of -inf alone or with a NaN has no token
  float most = -INFINITY;
  bool nan = false;
  // fewer parts than k bound nothing: then the threads' own maxima, of which there are more
  // (one capped bf16 row of 56291, 440 parts: top-500 85 -> 38 us, top-900 91 -> 43; where the
  // list then overflows, top-1000, 90 -> 104)
  const bool few_parts = k > a.blocks && k <= kThreads && k < V;
  const float* maxima = a.maxima && !few_parts ? a.maxima + r * a.blocks : nullptr;
  const int64_t bseg = (a.blocks + kWaves - 1) / kWaves;
  if (maxima) {
    for (int64_t b = wave * bseg + lane; b < (wave + 1) * bseg && b < a.blocks; b += 64) {
      nan |= maxima[b] != maxima[b];
      most = fmaxf(most, maxima[b]);
    }
  } else if (from < to) {
    row.template turns<8>(from, to, lane, 64, [&](int, const float (&v)[E], int64_t, int e0) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        nan |= v[e] != v[e];
        // each value in one thread's maximum: bound_of_maxima counts them
        most = fmaxf(most, e >= e0 ? v[e] : -INFINITY);
      }
    }, [] {});
  }
  const uint32_t own = order_key(most);            // key of -inf: nothing
  uint32_t best = wave_all(own, MaxOp());
  const uint64_t any_nan = __ballot(nan);
  if (lane == 0) {
    sm.wave_cnt[wave] = best;
    sm.wave_sum[wave] = any_nan;
  }
  __syncthreads();
  best = wave_all(sm.wave_cnt[lane & (kWaves - 1)], MaxOp());
  nan = __ballot(sm.wave_sum[lane & (kWaves - 1)] != 0) != 0;
  __syncthreads();                                 // read before they are written again
  if (nan || best <= kKeyNegInf) {
    if (tid == 0) {
      a.tokens[r] = -1;
      if (a.logp) a.logp[r] = nan ? NAN : -INFINITY;
    }
    return;
  }

  Weights<CAP> wt;
  wt.cap = a.softcap;
  wt.two_inv_cap = a.softcap > 0.f ? 2.0 / a.softcap : 0.0;
  wt.xmax = wt.warp(key_value(best));
  // not 0 for an infinite temperature: -inf times it is to stay -inf
  wt.scale = T_ > 0.f ? fmax(kLog2eD / double(T_), 1e-300) : 0.0;
  wt.S = a.weight_bits;
  wt.min_p = fmin(fmax(double(a.min_p.at(r)), 0.0), 1.0);
  wt.log_min_p = wt.min_p > 0.0 ? fmax(log2(wt.min_p), -63.0) : -63.0;
  const double p = fmax(double(a.top_p.at(r)), 0.0);

  uint64_t total = 0, target = 0;
  int64_t token = -1;
  if (k == 1 && maxima) {                          // the first of the largest
    const int n = collect_parts(row, a, maxima, bseg, best, sm);
    if (n > 0) token = sm.idx[0];
    total = 1ull << wt.S;
  }
  if (k == 1 && token < 0) {
    if (maxima || own == best) {
      uint32_t first = ~0u;
      row.each(from, to, lane, 64, [&](float z, int64_t i) {
        if (order_key(z) == best && uint32_t(i) < first) first = uint32_t(i);
      });
      sm.idx[tid] = first;
    } else {
      sm.idx[tid] = ~0u;
    }
    __syncthreads();
    uint32_t first = sm.idx[lane];
#pragma unroll 1
    for (int i = 1; i < kWaves; ++i) first = MinOp()(first, sm.idx[i * 64 + lane]);
    token = wave_all(first, MinOp());
    total = 1ull << wt.S;
  } else if (k > 1 && (k < V || (p >= 1.0 && wt.min_p > 0.0))) {
    // a list of all that may be kept
    int n;
    if (k < V) {
      const uint32_t bound = k <= kThreads ? bound_of_maxima(own, k, sm) : 0u;
      n = !bound ? -1
          : maxima ? collect_parts(row, a, maxima, bseg, bound, sm)
                   : collect(row, seg, sm, [&](float z) { return order_key(z) >= bound; });
    } else {
      n = collect(row, seg, sm, [&](float z) { return wt.reaches_min_p(z); });
    }
    if (n >= 0) {
      int64_t at;
      if (n <= kSmallList) {
        at = small_list(sm, n, wt, k, p, uniform, total);
      } else {
        const List list{sm.key, n};
        const Kept s = select(list, sm, wt, k, p);
        at = descend(list, Place{0, n, 0, 0}, sm, wt, s, uniform, total, target);
      }
      token = sm.idx[at];
    }
  } else if (k > 1 && p < 1.0) {
    // weights by bins of an eighth of a power of two, each wave its own
    for (int i = tid; i < kWaves * kMassBins; i += kThreads) (&sm.mass[0][0])[i] = 0;
    __syncthreads();
    // 0: the largest weights; the last holds all below 2^-47.9
    auto bin_of = [](double t) {
      const int b = int(t * -8.0);
      return b < kMassBins - 1 ? b : kMassBins - 1;
    };
    if (from < to)
      row.each(from, to, lane, 64, [&](float z, int64_t) {
        const double t = wt.log_weight(z);
        const uint64_t w = wt.fixed_of(t);
        if (w)
          atomicAdd(reinterpret_cast<unsigned long long*>(&sm.mass[wave][bin_of(t)]),
                    static_cast<unsigned long long>(w));
      });
    __syncthreads();
    // the bin in which the sum passes p of all
    uint64_t mine = 0;
    if (tid < kMassBins)
      for (int i = 0; i < kWaves; ++i) mine += sm.mass[i][tid];
    const uint64_t incl = wave_scan64(mine);
    if (lane == 63) sm.wave_sum[wave] = incl;
    __syncthreads();
    uint64_t all;
    const uint64_t before = before_wave(sm, wave, all);
    const double share = __builtin_ceil(p * double(all));
    const uint64_t limit = share >= double(all) ? all : share >= 1.0 ? uint64_t(share) : 1;
    const uint64_t upto = before + incl;
    if (tid < kMassBins && upto >= limit && upto - mine < limit) {
      sm.bin = tid;
      sm.above = upto - mine;
    }
    __syncthreads();
    const int p_bin = sm.bin;
    const uint64_t above_bin = sm.above;
    int bin = p_bin;
    if (wt.min_p > 0.0) {
      // what min-p leaves lies in higher bins alone: it is all kept
      if (bin_of(wt.log_min_p) + 1 < bin) bin = -1;
    }
    int n;
    if (bin < 0) {
      n = collect(row, seg, sm, [&](float z) { return wt.reaches_min_p(z); });
      if (n >= 0) {
        const List list{sm.key, n};
        const int64_t at = descend(list, Place{0, n, 0, 0}, sm, wt, Kept{}, uniform, total, target);
        token = sm.idx[at];
      }
    } else {
      // each segment's mass in the bins above is kept, unless min-p's border is near
      const bool clean = !(wt.min_p > 0.0) || bin_of(wt.log_min_p) - 1 > bin;
      uint64_t sum = 0;
      if (clean) {
        for (int i = lane; i < bin; i += 64) sum += sm.mass[wave][i];
        sum = wave_sum64(sum);
      }
      if (clean && gather(row, seg, sm, [&](float z) { return bin_of(wt.log_weight(z)) == bin; })) {
        const Gathered in_bin{sm, 0};
        uint32_t least = ~0u, most = 0;
        in_bin.each(0, 0, tid, kThreads, [&](float z, int64_t) {
          least = MinOp()(least, order_key(z));
          most = MaxOp()(most, order_key(z));
        });
        least = wave_all(least, MinOp());
        most = wave_all(most, MaxOp());
        if (lane == 0) sm.wave_sum[wave] = uint64_t(most) << 32 | least;
        __syncthreads();
        const uint64_t ends = sm.wave_sum[lane & (kWaves - 1)];
        least = wave_all(uint32_t(ends), MinOp());
        most = wave_all(uint32_t(ends >> 32), MaxOp());
        const int differ = 32 - __builtin_clz((least ^ most) | 1u);
        Kept s;
        uint64_t above, goal = limit - above_bin;
        s.tau = select_key(in_bin, sm, goal, 0.0, false, above, 0u, 0ull,
                           [&](float z, uint32_t) { return wt.mass(z); }, differ,
                           differ < 32 ? most >> differ << differ : 0u);
        const uint64_t w = wt.mass(key_value(s.tau));
        s.m = (goal - above + w - 1) / w;
        // the kept mass and ties of each segment
        uint64_t in = 0;
        uint32_t ties = 0;
        in_bin.each(0, 0, tid, kThreads, [&](float z, int64_t) {
          const uint32_t key = order_key(z);
          if (key > s.tau) in += wt.mass(z);
          else if (key == s.tau) ++ties;
        });
        in = wave_sum64(in) + sum;
        ties = uint32_t(wave_sum64(ties));
        __syncthreads();                           // the counts are read
        if (lane == 0) {
          sm.wave_sum[wave] = in;
          sm.wave_cnt[wave] = ties;
        }
        Place at{0, V, 0, 0};
        enter(at, seg, sm, s, w, uniform, total, target);
        token = descend(row, at, sm, wt, s, uniform, total, target);
      }
    }
  }
  if (token < 0) {                                 // no filter, or a list that does not fit
    const Kept s = k < V || p < 1.0 ? select(row, sm, wt, k, p) : Kept{};
    token = descend(row, Place{0, V, 0, 0}, sm, wt, s, uniform, total, target);
  }
  if (tid == 0) {
    a.tokens[r] = token;
    if (a.logp) {
      const double x = k == 1 ? 0.0 : fmin((wt.warp(row.at(token)) - wt.xmax) * wt.scale, 0.0);
      a.logp[r] = float(x / kLog2eD - log(__builtin_ldexp(double(total), -wt.S)));
    }
  }
}

// The maxima of each 16 chunks of the rows: 64 float32 or 128 bf16 logits, NaN where one is.
// Where a few rows are long a workgroup a row leaves most CUs idle, and reads the row twice.
template <class T>
__global__ __launch_bounds__(256) void k_sample_maxima(SampleArgs a, float* __restrict__ maxima) {
  constexpr int E = kPerChunk<T>, U = kMaximaChunks;
  const int64_t r = blockIdx.y;
  const Row<T> row{static_cast<const T*>(a.logits) + r * a.ld, a.V};
  const int64_t c0 = (int64_t(blockIdx.x) * (256 * U) + threadIdx.x) * E;
  float v[U][E];
  int64_t i[U];
  int e0[U];
#pragma unroll
  for (int u = 0; u < U; ++u) e0[u] = row.chunk(c0 + u * 256 * E, a.V, v[u], i[u]);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e) m = MaxNanOp()(m, e >= e0[u] ? v[u][e] : -INFINITY);
    m = group_all<16>(m, MaxNanOp());
    const int64_t part = (c0 + u * 256 * E) / (16 * E);
    if (threadIdx.x % 16 == 0 && part < a.blocks) maxima[r * a.blocks + part] = m;
  }
}

template <class T>
hipError_t sample(SampleArgs a, float* maxima, const Launcher& L) {
  if (maxima && a.blocks && !a.maxima) {
    constexpr int64_t kCols = 256 * kMaximaChunks * kPerChunk<T>;
    L.pre(kSample);
    hipLaunchKernelGGL(k_sample_maxima<T>, dim3(unsigned((a.V + kCols - 1) / kCols), unsigned(a.N)),
                       dim3(256), 0, L.stream, a, maxima);
    L.post(kSample);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    a.maxima = maxima;
  }
  L.pre(kSample);
  hipLaunchKernelGGL((a.softcap > 0.f ? k_sample<T, true> : k_sample<T, false>), dim3(unsigned(a.N)), dim3(kThreads), 0, L.stream, a);
  L.post(kSample);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, float* maxima, const Launcher& L) {
  return a.dtype == FLCE_F32 ? sample<float>(a, maxima, L) : sample<Bf16Bits>(a, maxima, L);
}

}  // namespace flce
