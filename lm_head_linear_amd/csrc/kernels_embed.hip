// Embedding lookup with scaling, out_i = round(scale W[tok_i]), and its
// gradient dW[v] (+)= round(scale sum of dout_i over tok_i = v).
//
// The lookup reads and writes a row per token and is bound by that.
//
// The gradient sorts the tokens (stable, so equal ids keep their order), and a
// wave then adds up the rows of a window of sorted tokens over a slice of
// columns, one id after another: each row of dout is read once, a dW row whose
// tokens lie in one window is written once, and the sums are float32 in a fixed
// order. An id whose tokens reach past a window leaves a float32 partial row per
// window; a second pass adds those up in window order. Atomic adds would need
// float32 rows of the whole table and would not give the same bits twice.
//
// The sort: least significant digit first, 8 bits a pass. A wave ranks 64 keys
// at a time by ballots over the digit's bits, counting in a table of its own,
// so equal digits keep their order. Up to kSortLocal tokens one workgroup sorts
// in LDS; more go through one histogram, scan and scatter pass per digit over
// many workgroups.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "flce_internal.h"
#include "ops_plan.h"
#include "row_io.h"

namespace flce {
namespace {

// ---- lookup ---------------------------------------------------------------------
// A wave per unit of 128 chunks (2 KiB) of one row.
constexpr int kUnitChunks = 128;

template <class T>
__global__ __launch_bounds__(256) void k_embed(const int64_t* __restrict__ tokens,
                                               const T* __restrict__ W, int64_t N, int64_t H,
                                               int64_t V, int64_t padding, float scale,
                                               T* __restrict__ out, int64_t ldo, int64_t units) {
  constexpr int E = kPerChunk<T>;
  const int lane = threadIdx.x & 63;
  const int64_t u = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (u >= N * units) return;
  const int64_t row = u / units, c0 = (u - row * units) * kUnitChunks * E;
  const int64_t tok = tokens[row];
  const bool pad = tok == padding, bad = !pad && (tok < 0 || tok >= V);
  const T* src = W + (pad || bad ? 0 : tok) * H;
  float f[2][E];
#pragma unroll
  for (int k = 0; k < 2; ++k) load_chunk(src, c0 + (k * 64 + lane) * E, H, f[k]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int e = 0; e < E; ++e) f[k][e] = bad ? NAN : pad ? 0.f : f[k][e] * scale;
    store_chunk(out + row * ldo, c0 + (k * 64 + lane) * E, H, f[k]);
  }
}

// *status = FLCE_ERR_LABEL if any token is neither the padding index nor in
// [0, V). One workgroup.
__global__ __launch_bounds__(1024) void k_token_status(const int64_t* __restrict__ tokens,
                                                       int64_t N, int64_t V, int64_t padding,
                                                       int32_t* __restrict__ status) {
  int bad = 0;
  for (int64_t i = threadIdx.x; i < N; i += 1024) {
    const int64_t t = tokens[i];
    bad |= t != padding && (t < 0 || t >= V);
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *status = bad ? FLCE_ERR_LABEL : FLCE_OK;
}

// ---- the sort -------------------------------------------------------------------
constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;

// A token's key: its id, or V for one that has no row (padding, or outside the
// table), which sorts behind all others.
__device__ __forceinline__ uint32_t token_key(int64_t t, int64_t V, int64_t padding) {
  return (t == padding || t < 0 || t >= V) ? uint32_t(V) : uint32_t(t);
}

// The rank of this lane's digit among the wave's keys so far: the count of equal
// digits in earlier rounds (cnt, this wave's table) plus those of lower lanes.
// Dead lanes take no part. Every lane of the wave calls it.
__device__ __forceinline__ uint32_t wave_rank(uint32_t d, bool live, uint32_t* cnt, int lane) {
  uint64_t same = __ballot(live);
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint64_t m = __ballot((d >> b) & 1);
    same &= ((d >> b) & 1) ? m : ~m;
  }
  const uint32_t lower = __popcll(same & ((1ull << lane) - 1));
  uint32_t base = 0;
  // the table is read and written by different lanes of the wave: keep the order
  if (live) base = cnt[d];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  if (live && lower == 0) cnt[d] = base + __popcll(same);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  return base + lower;
}

// cnt[w][d] (the waves' digit counts) replaced by where wave w's first key of
// digit d goes, `base` of digit d (by thread d < 256) added: exclusive sums over
// digits, then over waves. `base` null: the digits one behind another.
__device__ __forceinline__ void digit_offsets(uint32_t (*cnt)[256], uint32_t* wsum,
                                              const uint32_t* base) {
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t total = 0;
  if (tid < 256)
    for (int i = 0; i < kSortWaves; ++i) total += cnt[i][tid];
  uint32_t inc = total;
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t o = __shfl_up(inc, off);
    if (lane >= off) inc += o;
  }
  if (tid < 256 && lane == 63) wsum[w] = inc;
  __syncthreads();
  if (tid < 256) {
    uint32_t at = inc - total;
    for (int i = 0; i < w; ++i) at += wsum[i];
    if (base) at = base[tid];
    for (int i = 0; i < kSortWaves; ++i) {
      const uint32_t n = cnt[i][tid];
      cnt[i][tid] = at;
      at += n;
    }
  }
  __syncthreads();
}

// Up to kSortLocal tokens, in one workgroup: R keys a thread.
template <int R>
__global__ __launch_bounds__(kSortThreads) void k_sort_local(
    const int64_t* __restrict__ tokens, int64_t N, int64_t V, int64_t padding, int bits,
    uint32_t* __restrict__ skey, uint32_t* __restrict__ spos, int32_t* __restrict__ status) {
  __shared__ uint32_t key[kSortThreads * R];
  __shared__ uint16_t pos[kSortThreads * R];
  __shared__ uint32_t cnt[kSortWaves][256];
  __shared__ uint32_t wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t k[R], p[R], dest[R];
  int bad = 0;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (w * R + r) * 64 + lane;         // wave w: R consecutive runs of 64
    p[r] = uint32_t(i);
    k[r] = 0;
    if (i < N) {
      const int64_t t = tokens[i];
      k[r] = token_key(t, V, padding);
      bad |= t != padding && k[r] == uint32_t(V);
    }
  }
  bad = __syncthreads_or(bad);
  if (status && tid == 0) *status = bad ? FLCE_ERR_LABEL : FLCE_OK;
  for (int shift = 0; shift < bits; shift += 8) {
    for (int i = tid; i < kSortWaves * 256; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
      dest[r] = wave_rank((k[r] >> shift) & 255, (w * R + r) * 64 + lane < N, cnt[w], lane);
    __syncthreads();
    digit_offsets(cnt, wsum, nullptr);
#pragma unroll
    for (int r = 0; r < R; ++r)
      if ((w * R + r) * 64 + lane < N) {
        const uint32_t to = cnt[w][(k[r] >> shift) & 255] + dest[r];
        key[to] = k[r];
        pos[to] = uint16_t(p[r]);
      }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int i = (w * R + r) * 64 + lane;
      if (i < N) { k[r] = key[i]; p[r] = pos[i]; }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = (w * R + r) * 64 + lane;
    if (i < N) { skey[i] = k[r]; spos[i] = p[r]; }
  }
}

// Many workgroups, kSortBlock keys each (kSortRounds a thread). `first`: the keys
// come from the tokens, their positions are their order.
constexpr int kSortRounds = int(kSortBlock) / kSortThreads;

__device__ __forceinline__ void read_keys(uint32_t (&k)[kSortRounds], uint32_t (&p)[kSortRounds],
                                          const int64_t* tokens, const uint32_t* key,
                                          const uint32_t* pos, int64_t N, int64_t V,
                                          int64_t padding) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int64_t i = int64_t(blockIdx.x) * kSortBlock + (w * kSortRounds + r) * 64 + lane;
    k[r] = p[r] = 0;
    if (i < N) {
      k[r] = tokens ? token_key(tokens[i], V, padding) : key[i];
      p[r] = tokens ? uint32_t(i) : pos[i];
    }
  }
}

// hist[d][block] = keys of digit d in the block.
__global__ __launch_bounds__(kSortThreads) void k_sort_hist(
    const int64_t* __restrict__ tokens, const uint32_t* __restrict__ key, int64_t N, int64_t V,
    int64_t padding, int shift, uint32_t* __restrict__ hist) {
  __shared__ uint32_t cnt[256];
  if (threadIdx.x < 256) cnt[threadIdx.x] = 0;
  __syncthreads();
  for (int64_t i = int64_t(blockIdx.x) * kSortBlock + threadIdx.x;
       i < N && i < (int64_t(blockIdx.x) + 1) * kSortBlock; i += kSortThreads) {
    const uint32_t k = tokens ? token_key(tokens[i], V, padding) : key[i];
    atomicAdd(&cnt[(k >> shift) & 255], 1u);       // a count: its order does not matter
  }
  __syncthreads();
  if (threadIdx.x < 256) hist[int64_t(threadIdx.x) * gridDim.x + blockIdx.x] = cnt[threadIdx.x];
}

// Exclusive sums over the n counts, in place. One workgroup.
__global__ __launch_bounds__(kSortThreads) void k_sort_scan(uint32_t* __restrict__ hist,
                                                            int64_t n) {
  __shared__ uint32_t wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  uint32_t before = 0;
  for (int64_t i0 = 0; i0 < n; i0 += kSortThreads) {
    const int64_t i = i0 + tid;
    const uint32_t x = i < n ? hist[i] : 0;
    uint32_t inc = x;
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t o = __shfl_up(inc, off);
      if (lane >= off) inc += o;
    }
    if (lane == 63) wsum[w] = inc;
    __syncthreads();
    uint32_t at = before + inc - x, all = 0;
    for (int j = 0; j < kSortWaves; ++j) {
      at += j < w ? wsum[j] : 0;
      all += wsum[j];
    }
    if (i < n) hist[i] = at;
    before += all;
    __syncthreads();
  }
}

__global__ __launch_bounds__(kSortThreads) void k_sort_scatter(
    const int64_t* __restrict__ tokens, const uint32_t* __restrict__ key,
    const uint32_t* __restrict__ pos, int64_t N, int64_t V, int64_t padding, int shift,
    const uint32_t* __restrict__ hist, uint32_t* __restrict__ okey, uint32_t* __restrict__ opos) {
  __shared__ uint32_t cnt[kSortWaves][256];
  __shared__ uint32_t base[256], wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  for (int i = tid; i < kSortWaves * 256; i += kSortThreads) (&cnt[0][0])[i] = 0;
  if (tid < 256) base[tid] = hist[int64_t(tid) * gridDim.x + blockIdx.x];
  __syncthreads();
  uint32_t k[kSortRounds], p[kSortRounds], rank[kSortRounds];
  read_keys(k, p, tokens, key, pos, N, V, padding);
  const int64_t i0 = int64_t(blockIdx.x) * kSortBlock + w * kSortRounds * 64 + lane;
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    rank[r] = wave_rank((k[r] >> shift) & 255, i0 + r * 64 < N, cnt[w], lane);
  __syncthreads();
  digit_offsets(cnt, wsum, base);
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r)
    if (i0 + r * 64 < N) {
      const uint32_t to = cnt[w][(k[r] >> shift) & 255] + rank[r];
      okey[to] = k[r];
      opos[to] = p[r];
    }
}

// ---- the sums ---------------------------------------------------------------------
// A lane's E values of a slice: 8 columns of either dout type.
constexpr int kLaneCols = 8;
constexpr int kSliceCols = 64 * kLaneCols;

template <class T>
__device__ __forceinline__ void load_cols(const T* row, int64_t c, int64_t n, float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    load_chunk(row, c, n, f);
  } else {
    float a[4], b[4];
    load_chunk(row, c, n, a);
    load_chunk(row, c + 4, n, b);
#pragma unroll
    for (int e = 0; e < 4; ++e) { f[e] = a[e]; f[4 + e] = b[e]; }
  }
}
template <class T>
__device__ __forceinline__ void store_cols(T* row, int64_t c, int64_t n, const float (&f)[8]) {
  if constexpr (sizeof(T) == 2) {
    store_chunk(row, c, n, f);
  } else {
    float a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) { a[e] = f[e]; b[e] = f[4 + e]; }
    store_chunk(row, c, n, a);
    store_chunk(row, c + 4, n, b);
  }
}

// dW[v] = scale acc, added to what is there when `accumulate`.
template <class G>
__device__ __forceinline__ void write_row(G* dW, int64_t v, int64_t H, int64_t c, float scale,
                                          int accumulate, const float (&acc)[8]) {
  float f[8];
  if (accumulate) {
    load_cols(dW + v * H, c, H, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = fmaf(acc[e], scale, f[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = acc[e] * scale;
  }
  store_cols(dW + v * H, c, H, f);
}

// A wave: the sorted tokens [w win, w win + win) over kSliceCols columns. The
// partial rows of window w: part[2 w] of an id that reaches into it from the
// window before, part[2 w + 1] of one that starts in it and reaches past it.
constexpr int kInFlight = 8;                       // rows loaded before they are added

template <class T, class G>
__global__ __launch_bounds__(256) void k_embed_sum(
    const uint32_t* __restrict__ skey, const uint32_t* __restrict__ spos,
    const T* __restrict__ dout, int64_t ldd, int64_t N, int64_t H, int64_t V, int win,
    int64_t slices, float scale, int accumulate, G* __restrict__ dW, float* __restrict__ part) {
  const int lane = threadIdx.x & 63;
  const int64_t u = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wd = u / slices, c = (u - wd * slices) * kSliceCols + lane * kLaneCols;
  const int64_t i0 = wd * win;
  if (i0 >= N) return;
  const int n = int(N - i0 < win ? N - i0 : win);
  // an id that reaches in from the window before: its first run is a partial row
  auto key_at = [&](int64_t i) -> uint32_t { return __builtin_amdgcn_readfirstlane(skey[i]); };
  uint32_t cur = key_at(i0);
  bool head = i0 > 0 && key_at(i0 - 1) == cur;
  float acc[8] = {};
  auto flush = [&](bool tail) {
    if (cur >= uint32_t(V)) return;                // no row: padding, or a bad id
    if (head || tail) store_cols(part + (2 * wd + (head ? 0 : 1)) * H, c, H, acc);
    else write_row(dW, int64_t(cur), H, c, scale, accumulate, acc);
  };
  for (int b = 0; b < n; b += kInFlight) {
    float f[kInFlight][8];
    uint32_t key[kInFlight];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      const int64_t i = i0 + (b + r < n ? b + r : n - 1);
      key[r] = key_at(i);
      if (key[r] >= uint32_t(V)) continue;         // the rows behind the last id
      load_cols(dout + int64_t(__builtin_amdgcn_readfirstlane(spos[i])) * ldd, c, H, f[r]);
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      if (b + r >= n || key[r] >= uint32_t(V)) continue;
      if (key[r] != cur) {
        flush(false);
        cur = key[r];
        head = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += f[r][e];
    }
    if (key[kInFlight - 1] >= uint32_t(V)) break;  // nothing but such rows from here on
  }
  flush(i0 + n < N && key_at(i0 + n) == cur);
}

// The ids that reach past the window they start in: their partial rows added up
// in window order. A wave per window and slice; most have none and leave.
template <class G>
__global__ __launch_bounds__(256) void k_embed_join(const uint32_t* __restrict__ skey, int64_t N,
                                                    int64_t H, int64_t V, int win, int64_t slices,
                                                    float scale, int accumulate,
                                                    G* __restrict__ dW,
                                                    const float* __restrict__ part) {
  const int lane = threadIdx.x & 63;
  const int64_t u = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wd = u / slices, c = (u - wd * slices) * kSliceCols + lane * kLaneCols;
  const int64_t i0 = wd * win, i1 = i0 + win;
  if (i1 >= N) return;                             // the last window: nothing behind it
  const uint32_t key = skey[i1 - 1];
  if (key >= uint32_t(V) || skey[i1] != key) return;
  if (skey[i0] == key && i0 > 0 && skey[i0 - 1] == key) return;   // it started earlier
  float acc[8];
  load_cols(part + (2 * wd + 1) * H, c, H, acc);
  for (int64_t x = wd + 1;; ++x) {
    float f[8];
    load_cols(part + 2 * x * H, c, H, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] += f[e];
    const int64_t end = (x + 1) * win;
    if (end >= N || skey[end] != key) break;
  }
  write_row(dW, int64_t(key), H, c, scale, accumulate, acc);
}

template <int R>
void sort_local(const EmbedGradArgs& a, int bits, const Launcher& L) {
  hipLaunchKernelGGL(k_sort_local<R>, dim3(1), dim3(kSortThreads), 0, L.stream, a.tokens, a.N, a.V,
                     a.padding, bits, a.key[0], a.pos[0], a.status);
}

template <class T, class G>
hipError_t sums(const EmbedGradArgs& a, const uint32_t* key, const uint32_t* pos,
                const Launcher& L) {
  const int64_t slices = (a.H + kSliceCols - 1) / kSliceCols;
  const int64_t waves = (a.N + a.window - 1) / a.window * slices;
  const dim3 grid(unsigned((waves + 3) / 4));
  G* dW = static_cast<G*>(a.dW);
  L.pre(kEmbedGrad);
  hipLaunchKernelGGL((k_embed_sum<T, G>), grid, dim3(256), 0, L.stream, key, pos,
                     static_cast<const T*>(a.dout), a.ld_dout, a.N, a.H, a.V, int(a.window),
                     slices, a.scale, a.accumulate, dW, a.part);
  L.post(kEmbedGrad);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.N <= a.window) return e;
  L.pre(kEmbedGrad);
  hipLaunchKernelGGL(k_embed_join<G>, grid, dim3(256), 0, L.stream, key, a.N, a.H, a.V,
                     int(a.window), slices, a.scale, a.accumulate, dW, a.part);
  L.post(kEmbedGrad);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_embedding(const EmbedArgs& a, const Launcher& L) {
  const int64_t e = a.dtype == FLCE_BF16 ? 8 : 4;
  const int64_t units = (a.H + kUnitChunks * e - 1) / (kUnitChunks * e);
  const dim3 grid(unsigned((a.N * units + 3) / 4));
  L.pre(kEmbed);
  if (a.dtype == FLCE_BF16)
    hipLaunchKernelGGL(k_embed<Bf16Bits>, grid, dim3(256), 0, L.stream, a.tokens,
                       static_cast<const Bf16Bits*>(a.W), a.N, a.H, a.V, a.padding, a.scale,
                       static_cast<Bf16Bits*>(a.out), a.ld_out, units);
  else
    hipLaunchKernelGGL(k_embed<float>, grid, dim3(256), 0, L.stream, a.tokens,
                       static_cast<const float*>(a.W), a.N, a.H, a.V, a.padding, a.scale,
                       static_cast<float*>(a.out), a.ld_out, units);
  L.post(kEmbed);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess || !a.status) return r;
  return launch_token_status(a.tokens, a.N, a.V, a.padding, a.status, L);
}

hipError_t launch_token_status(const int64_t* tokens, int64_t N, int64_t V, int64_t padding,
                               int32_t* status, const Launcher& L) {
  L.pre(kEmbedSort);
  hipLaunchKernelGGL(k_token_status, dim3(1), dim3(1024), 0, L.stream, tokens, N, V, padding,
                     status);
  L.post(kEmbedSort);
  return hipGetLastError();
}

hipError_t launch_embedding_backward(const EmbedGradArgs& a, const Launcher& L) {
  hipError_t e = hipSuccess;
  if (!a.accumulate) {
    const size_t es = a.grad_dtype == FLCE_BF16 ? 2 : 4;
    e = launch_zero_bytes(a.dW, size_t(a.V) * a.H * es, L);
    if (e != hipSuccess) return e;
  }
  int bits = 1;
  while (bits < 32 && (int64_t(1) << bits) <= a.V) ++bits;   // keys 0 .. V
  int at = 0;
  if (a.N <= kSortLocal) {
    L.pre(kEmbedSort);
    if (a.N <= kSortThreads) sort_local<1>(a, bits, L);
    else if (a.N <= 4 * kSortThreads) sort_local<4>(a, bits, L);
    else sort_local<16>(a, bits, L);
    L.post(kEmbedSort);
    e = hipGetLastError();
  } else {
    if (a.status) e = launch_token_status(a.tokens, a.N, a.V, a.padding, a.status, L);
    const int64_t nb = (a.N + kSortBlock - 1) / kSortBlock;
    const dim3 grid{unsigned(nb)};
    for (int shift = 0; e == hipSuccess && shift < bits; shift += 8) {
      const int64_t* tok = shift == 0 ? a.tokens : nullptr;
      L.pre(kEmbedSort);
      hipLaunchKernelGGL(k_sort_hist, grid, dim3(kSortThreads), 0, L.stream, tok, a.key[at], a.N,
                         a.V, a.padding, shift, a.hist);
      hipLaunchKernelGGL(k_sort_scan, dim3(1), dim3(kSortThreads), 0, L.stream, a.hist, 256 * nb);
      hipLaunchKernelGGL(k_sort_scatter, grid, dim3(kSortThreads), 0, L.stream, tok, a.key[at],
                         a.pos[at], a.N, a.V, a.padding, shift, a.hist, a.key[1 - at],
                         a.pos[1 - at]);
      L.post(kEmbedSort);
      e = hipGetLastError();
      at = 1 - at;
    }
  }
  if (e != hipSuccess) return e;
  if (a.dtype == FLCE_F32) return sums<float, float>(a, a.key[at], a.pos[at], L);
  if (a.grad_dtype == FLCE_F32) return sums<Bf16Bits, float>(a, a.key[at], a.pos[at], L);
  return sums<Bf16Bits, Bf16Bits>(a, a.key[at], a.pos[at], L);
}

}  // namespace flce
