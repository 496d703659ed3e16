// Embedding lookup with scaling, out_i = round(scale W[tok_i]), and its
// gradient dW[v] (+)= round(scale sum of dout_i over tok_i = v).
//
// The lookup reads and writes a row per token and is bound by that (bf16, 16384 rows of
// 4096 of a table of 131072, frequent ids repeated: 40 us, 268 MB).
//
// The gradient sorts the tokens (stable, so equal ids keep their order), and the
// rows of 64 or 256 sorted tokens are then added up over a slice of columns by a
// workgroup, one id after another: each row of dout is read once, a dW row whose
// tokens lie in one window is written once, and the sums are float32 in a fixed
// order. An id whose tokens reach past a window leaves a float32 partial row per
// window; a second pass adds those up in window order. Atomic adds would need
// float32 rows of the whole table and would not give the same bits twice.
//
// The sort: least significant digit first, 8 bits a pass. A wave ranks 64 keys
// at a time by ballots over the digit's bits, counting in a table of its own,
// so equal digits keep their order. A workgroup sorts a chunk of kSortChunk
// tokens in LDS. Up to kSortMerge tokens the sorted chunks are merged in one
// step: a key's place is its place in its chunk plus, found by bisection in LDS,
// the keys of each other chunk that go before it. More tokens go through one
// histogram, scan and scatter pass per digit over many workgroups. (One
// workgroup sorting 16384 tokens in LDS by itself took 163 us.)
//
// The gradient is bound by writing dW and reading dout. The same 16384 rows: 9 us for
// the chunks, 168 us for the merge, which clears the 1.07 GB of dW beside it (6.4 TB/s),
// 62 us for the sums and 5 us for the ids that cross windows. Added to a dW that is
// there, the clearing falls away.
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

// The sort keeps a few CUs busy for some 20 us: the other workgroups of its two
// launches clear dW meanwhile, 64 KiB each.
struct Clear {
  uint4* p;
  int64_t n16;                // 16-byte pieces in all
  int64_t first;              // the launch's first 64 KiB piece
};
__device__ __forceinline__ void clear_piece(const Clear& f, int64_t piece) {
  const uint4 z = {0u, 0u, 0u, 0u};
  const int64_t i = (f.first + piece) * 4096 + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + 1024 * k < f.n16) f.p[i + 1024 * k] = z;
}

// Chunk blockIdx.x of kSortChunk tokens, a key a thread; the workgroups behind the
// chunks clear.
__global__ __launch_bounds__(kSortThreads) void k_sort_chunks(
    const int64_t* __restrict__ tokens, int64_t N, int64_t V, int64_t padding, int bits,
    uint32_t* __restrict__ skey, uint32_t* __restrict__ spos, int64_t chunks, Clear fill) {
  if (blockIdx.x >= chunks) {
    clear_piece(fill, blockIdx.x - chunks);
    return;
  }
  static_assert(kSortThreads == kSortChunk, "a key a thread");
  __shared__ uint32_t key[kSortThreads], pos[kSortThreads];
  __shared__ uint32_t cnt[kSortWaves][256];
  __shared__ uint32_t wsum[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t i0 = int64_t(blockIdx.x) * kSortChunk;
  const bool live = i0 + tid < N;
  uint32_t k = live ? token_key(tokens[i0 + tid], V, padding) : 0, p = uint32_t(i0 + tid);
  for (int shift = 0; shift < bits; shift += 8) {
    for (int i = tid; i < kSortWaves * 256; i += kSortThreads) (&cnt[0][0])[i] = 0;
    __syncthreads();
    const uint32_t rank = wave_rank((k >> shift) & 255, live, cnt[w], lane);
    __syncthreads();
    digit_offsets(cnt, wsum, nullptr);
    if (live) {
      const uint32_t to = cnt[w][(k >> shift) & 255] + rank;
      key[to] = k;
      pos[to] = p;
    }
    __syncthreads();
    if (live) { k = key[tid]; p = pos[tid]; }
  }
  if (live) { skey[i0 + tid] = k; spos[i0 + tid] = p; }
}

// The sorted chunks merged, a key of chunk blockIdx.x a thread. Equal keys of an
// earlier chunk go before, those of a later one behind. C: chunks held, in LDS;
// places past the last key hold the largest value.
template <int C>
__global__ __launch_bounds__(kSortThreads) void k_sort_merge(
    const uint32_t* __restrict__ ikey, const uint32_t* __restrict__ ipos, int64_t N,
    uint32_t* __restrict__ okey, uint32_t* __restrict__ opos, int64_t chunks, Clear fill) {
  if (blockIdx.x >= chunks) {
    clear_piece(fill, blockIdx.x - chunks);
    return;
  }
  __shared__ __attribute__((aligned(16))) uint32_t key[C * kSortChunk];
  const int held = int(chunks + 3) / 4 * 4;
#pragma unroll 4
  for (int i = 4 * threadIdx.x; i < held * int(kSortChunk); i += 4 * kSortThreads) {
    uint4 v = {0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu};
    if (i + 4 <= N) {
      v = *reinterpret_cast<const uint4*>(ikey + i);
    } else {
      if (i < N) v.x = ikey[i];
      if (i + 1 < N) v.y = ikey[i + 1];
      if (i + 2 < N) v.z = ikey[i + 2];
    }
    *reinterpret_cast<uint4*>(key + i) = v;
  }
  __syncthreads();
  const int c = blockIdx.x;
  const int64_t at = int64_t(c) * kSortChunk + threadIdx.x;
  if (at >= N) return;
  const uint32_t k = key[at];
  uint32_t place = threadIdx.x;
  for (int b = 0; b < held; b += 4) {              // four bisections at a time
    uint32_t lo[4], less[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      lo[u] = 0;
      less[u] = b + u < c ? k + 1 : k;             // keys below this go before
    }
#pragma unroll
    for (int step = int(kSortChunk); step > 0; step >>= 1)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t m = lo[u] + step;
        if (m <= kSortChunk && key[(b + u) * kSortChunk + m - 1] < less[u]) lo[u] = m;
      }
#pragma unroll
    for (int u = 0; u < 4; ++u) place += b + u == c ? 0 : lo[u];
  }
  okey[place] = k;
  opos[place] = ipos[at];
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
// A wave's slice of kSliceCols columns, 8 a lane: 8 adjacent ones (FULL, a slice within
// the row), or every 64th (the slice at the row's end: loads past it read the row's
// last value, stores there are left out).
constexpr int kSliceCols = 512;

template <bool FULL>
struct Slice {
  int64_t c0, H;
  int lane;
  __device__ __forceinline__ int64_t col(int e) const {
    const int64_t c = c0 + e * 64 + lane;
    return c < H ? c : H - 1;
  }
  template <class T>
  __device__ __forceinline__ void load(const T* row, float (&f)[8]) const {
    if constexpr (!FULL) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = to_f32(row[col(e)]);
    } else if constexpr (sizeof(T) == 2) {
      unpack_chunk<T>(load_raw(row + c0 + lane * 8), f);
    } else {
      float a[4], b[4];
      unpack_chunk<T>(load_raw(row + c0 + lane * 8), a);
      unpack_chunk<T>(load_raw(row + c0 + lane * 8 + 4), b);
#pragma unroll
      for (int e = 0; e < 4; ++e) { f[e] = a[e]; f[4 + e] = b[e]; }
    }
  }
  template <class T>
  __device__ __forceinline__ void store(T* row, const float (&f)[8]) const {
    if constexpr (!FULL) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c0 + e * 64 + lane < H) row[c0 + e * 64 + lane] = from_f32<T>(f[e]);
    } else if constexpr (sizeof(T) == 2) {
      *reinterpret_cast<row_u32x4_any*>(row + c0 + lane * 8) = pack_chunk<T>(f);
    } else {
      const float a[4] = {f[0], f[1], f[2], f[3]}, b[4] = {f[4], f[5], f[6], f[7]};
      *reinterpret_cast<row_u32x4_any*>(row + c0 + lane * 8) = pack_chunk<T>(a);
      *reinterpret_cast<row_u32x4_any*>(row + c0 + lane * 8 + 4) = pack_chunk<T>(b);
    }
  }
  __device__ __forceinline__ int slot(int e) const { return FULL ? lane * 8 + e : e * 64 + lane; }
};

struct SumArgs {
  const uint32_t* skey;
  const uint32_t* spos;
  const void* dout;
  const float* weight;        // WEIGHT: row i counts weight[i] times, and what is added
  const uint32_t* slot;       //   to are the float32 rows slot[id] - 1 of keep, not dW
  const float* keep;
  int64_t ldd, N, H, V, slices;
  float scale;
  void* dW;
  float* part;
};

// A workgroup: 8 SW sorted tokens over a slice, SW of them a wave, in order. A wave
// writes the rows of the ids that begin and end in its SW; its first run, if the id
// began before, and its last, if the id goes on, stay in LDS, where the wave in which
// an id began adds up what the others left of it. What reaches past the workgroup's
// tokens goes to memory: part[2 w] of an id that began before workgroup w's tokens,
// part[2 w + 1] of one that begins there and goes on. ADD: the dW row is added to; it
// is loaded with the rows of dout, so that no id waits for its own.
constexpr int kSumWaves = 8;
constexpr int kInFlight = 8;                       // rows loaded before they are added

struct SumEdges {
  float run[2][kSumWaves][kSliceCols];             // first runs, last runs
  int whole[kSumWaves];                            // a wave's tokens are one run of an id
};                                                 //   that began before and goes on

template <class T, class G, bool WEIGHT, bool ADD, int SW, bool FULL>
__device__ __forceinline__ void sum_slice(const SumArgs& a, int64_t wd, const Slice<FULL>& sl,
                                          SumEdges& edge) {
  const int lane = sl.lane;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t H = a.H, N = a.N;
  G* dW = static_cast<G*>(a.dW);
  const T* dout = static_cast<const T*>(a.dout);
  const int64_t i0 = (wd * kSumWaves + w) * SW;
  const int n = i0 >= N ? 0 : int(N - i0 < SW ? N - i0 : SW);
  const uint32_t none = uint32_t(a.V);
  // the wave's keys, positions and weights in its lanes; the keys beside them
  const int li = lane & (SW - 1);
  const int64_t il = n > 0 ? i0 + (li < n ? li : n - 1) : 0;
  const uint32_t keys = n > 0 ? a.skey[il] : none, poss = n > 0 ? a.spos[il] : 0;
  const float wgts = WEIGHT && keys < none ? a.weight[poss] : 1.f;
  const uint32_t slots = WEIGHT && keys < none ? a.slot[keys] - 1 : 0;
  const uint32_t before = i0 > 0 && n > 0 ? a.skey[i0 - 1] : none;
  const uint32_t behind = n == SW && i0 + n < N ? a.skey[i0 + n] : none;
  auto uni = [](uint32_t x) -> uint32_t { return __builtin_amdgcn_readfirstlane(x); };
  auto key_of = [&](int q) -> uint32_t { return __builtin_amdgcn_readlane(keys, q); };
  uint32_t cur = key_of(0);
  bool head = cur < none && uni(before) == cur;
  const uint32_t last = n > 0 ? key_of(SW - 1) : none;
  const bool tail = last < none && uni(behind) == last;
  float acc[8] = {}, old[8] = {};
  auto write = [&](uint32_t key) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = ADD ? fmaf(acc[e], a.scale, old[e]) : acc[e] * a.scale;
    sl.store(dW + int64_t(key) * H, f);
  };
  auto leave = [&](int which) {                    // the run so far, to LDS
#pragma unroll
    for (int e = 0; e < 8; ++e) edge.run[which][w][sl.slot(e)] = acc[e];
  };
#pragma unroll 1
  for (int q = 0; q < SW; q += kInFlight) {
    if (q >= n || key_of(q) >= none) break;        // the rest has no rows
    float f[kInFlight][8], g[ADD ? kInFlight : 1][8];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      sl.load(dout + int64_t(uint32_t(__builtin_amdgcn_readlane(poss, q + r))) * a.ldd, f[r]);
      if constexpr (ADD) {
        const uint32_t key = key_of(q + r);
        if constexpr (WEIGHT)
          sl.load(a.keep + int64_t(uint32_t(__builtin_amdgcn_readlane(slots, q + r))) * H, g[r]);
        else
          sl.load(dW + int64_t(key < none ? key : 0) * H, g[r]);
      }
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      const uint32_t key = key_of(q + r);
      if (q + r >= n || key >= none) continue;
      if (key != cur) {
        if (head) leave(0);
        else write(cur);
        cur = key;
        head = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = 0.f;
      }
      const float x = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wgts), q + r));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        acc[e] = WEIGHT ? fmaf(x, f[r][e], acc[e]) : acc[e] + f[r][e];
        if constexpr (ADD) old[e] = g[r][e];
      }
    }
  }
  if (cur < none) {
    if (head) leave(0);
    else if (tail) leave(1);
    else write(cur);
  }
  if (lane == 0) edge.whole[w] = tail && head;     // head still set: no other id came
  __syncthreads();
  // wave w: the id that began in it and goes on; wave 0 also the one begun before.
  // True if it goes on past the workgroup.
  auto join = [&](int from, bool began) {
    int x = began ? from + 1 : 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = began ? edge.run[1][from][sl.slot(e)] : 0.f;
    for (; x < kSumWaves; ++x) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += edge.run[0][x][sl.slot(e)];
      if (!edge.whole[x]) break;
    }
    return x == kSumWaves;
  };
  const bool began_before = w == 0 && n > 0 && uni(before) < none && uni(before) == key_of(0);
  if (began_before) {
    join(0, false);
    sl.store(a.part + 2 * wd * H, acc);
  }
  if (tail && !edge.whole[w]) {
    if (join(w, true)) sl.store(a.part + (2 * wd + 1) * H, acc);
    else write(last);                              // `old` is still the row of `last`
  }
}

template <class T, class G, bool WEIGHT, bool ADD, int SW>
__global__ __launch_bounds__(64 * kSumWaves) void k_embed_sum(SumArgs a) {
  __shared__ SumEdges edge;
  const int lane = threadIdx.x & 63;
  const int64_t wd = blockIdx.x / a.slices, c0 = (blockIdx.x - wd * a.slices) * kSliceCols;
  if (c0 + kSliceCols <= a.H)
    sum_slice<T, G, WEIGHT, ADD, SW, true>(a, wd, Slice<true>{c0, a.H, lane}, edge);
  else
    sum_slice<T, G, WEIGHT, ADD, SW, false>(a, wd, Slice<false>{c0, a.H, lane}, edge);
}

// The ids that reach past the workgroup's tokens they begin in: their partial rows
// added up in order. A wave per workgroup's tokens and slice; most have none.
template <class G, bool WEIGHT, bool ADD, bool FULL>
__device__ __forceinline__ void join_slice(const SumArgs& a, int64_t win, int64_t wd,
                                           const Slice<FULL>& sl) {
  const int64_t H = a.H, i0 = wd * win, i1 = i0 + win;
  const uint32_t none = uint32_t(a.V);
  if (i1 >= a.N) return;                           // the last one: nothing behind it
  const uint32_t key = a.skey[i1 - 1];
  if (key >= none || a.skey[i1] != key) return;
  if (a.skey[i0] == key && i0 > 0 && a.skey[i0 - 1] == key) return;   // it began earlier
  G* row = static_cast<G*>(a.dW) + int64_t(key) * H;
  float acc[8], old[8] = {};
  sl.load(a.part + (2 * wd + 1) * H, acc);
  if constexpr (WEIGHT) sl.load(a.keep + int64_t(a.slot[key] - 1) * H, old);
  else if constexpr (ADD) sl.load(row, old);
  // those behind that begin with this id, their rows loaded eight at a time
  const int64_t windows = (a.N + win - 1) / win;
  bool more = true;
#pragma unroll 1
  for (int64_t x = wd + 1; more; x += kInFlight) {
    float f[kInFlight][8];
    uint32_t first[kInFlight];
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      const int64_t y = x + r < windows ? x + r : wd;
      first[r] = x + r < windows ? a.skey[y * win] : none;
      sl.load(a.part + 2 * y * H, f[r]);           // not added unless it is this id's
    }
#pragma unroll
    for (int r = 0; r < kInFlight; ++r) {
      more = more && first[r] == key;
      if (more) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[r][e];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) acc[e] = ADD ? fmaf(acc[e], a.scale, old[e]) : acc[e] * a.scale;
  sl.store(row, acc);
}

template <class G, bool WEIGHT, bool ADD>
__global__ __launch_bounds__(256) void k_embed_join(SumArgs a, int64_t win) {
  const int lane = threadIdx.x & 63;
  const int64_t u = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t wd = u / a.slices, c0 = (u - wd * a.slices) * kSliceCols;
  if (c0 + kSliceCols <= a.H) join_slice<G, WEIGHT, ADD>(a, win, wd, Slice<true>{c0, a.H, lane});
  else join_slice<G, WEIGHT, ADD>(a, win, wd, Slice<false>{c0, a.H, lane});
}

template <class T, class G, bool WEIGHT = false>
hipError_t sums(const EmbedGradArgs& a, const uint32_t* key, const uint32_t* pos,
                const Launcher& L) {
  const int64_t slices = (a.H + kSliceCols - 1) / kSliceCols, win = embed_window(a.N);
  const int64_t windows = (a.N + win - 1) / win;
  const SumArgs s{key, pos, a.dout, a.weight, a.slot, a.keep, a.ld_dout, a.N, a.H, a.V, slices,
                  a.scale, a.dW, a.part};
  auto run = [&](auto add) {
    constexpr bool ADD = decltype(add)::value;
    const dim3 grid(unsigned(windows * slices)), block(64 * kSumWaves);
    L.pre(kEmbedGrad);
    if (win == kSumWaves * 8)
      hipLaunchKernelGGL((k_embed_sum<T, G, WEIGHT, ADD, 8>), grid, block, 0, L.stream, s);
    else
      hipLaunchKernelGGL((k_embed_sum<T, G, WEIGHT, ADD, 32>), grid, block, 0, L.stream, s);
    L.post(kEmbedGrad);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || windows == 1) return e;
    L.pre(kEmbedGrad);
    hipLaunchKernelGGL((k_embed_join<G, WEIGHT, ADD>), dim3(unsigned((windows * slices + 3) / 4)),
                       dim3(256), 0, L.stream, s, win);
    L.post(kEmbedGrad);
    return hipGetLastError();
  };
  if constexpr (!WEIGHT)
    if (!a.accumulate) return run(std::false_type{});
  return run(std::true_type{});
}

// slot[v] = 1 + the sorted position of id v's first token; of ids without one it stays.
__global__ __launch_bounds__(256) void k_token_slots(const uint32_t* __restrict__ skey, int64_t N,
                                                     uint32_t none, uint32_t* __restrict__ slot) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= N) return;
  const uint32_t k = skey[i];
  if (k < none && (i == 0 || skey[i - 1] != k)) slot[k] = uint32_t(i) + 1;
}

// The tokens sorted into list *list of the workspace's two; `bytes` at `clear` are set to
// zero on the way.
hipError_t sort_tokens(const EmbedGradArgs& a, void* clear, size_t bytes, const Launcher& L,
                       int* list) {
  hipError_t e = hipSuccess;
  // cleared beside the sort as far as it is whole 16-byte pieces, else before it
  const bool beside = a.N <= kSortMerge && (reinterpret_cast<uintptr_t>(clear) & 15u) == 0;
  const size_t with = beside ? bytes / 16 * 16 : 0;
  e = launch_zero_bytes(static_cast<char*>(clear) + with, bytes - with, L);
  if (e != hipSuccess) return e;
  int bits = 1;
  while (bits < 32 && (int64_t(1) << bits) <= a.V) ++bits;   // keys 0 .. V
  int at = 0;
  if (a.N <= kSortMerge) {
    const int64_t chunks = (a.N + kSortChunk - 1) / kSortChunk;
    Clear fill{static_cast<uint4*>(clear), int64_t(with / 16), 0};
    const int64_t pieces = (fill.n16 + 4095) / 4096;
    const int64_t first = chunks > 1 && pieces > 512 ? 512 : pieces;
    L.pre(kEmbedSort);
    hipLaunchKernelGGL(k_sort_chunks, dim3(unsigned(chunks + first)), dim3(kSortThreads), 0,
                       L.stream, a.tokens, a.N, a.V, a.padding, bits, a.key[0], a.pos[0], chunks,
                       fill);
    fill.first = first;
    auto merge = [&](auto c) {
      hipLaunchKernelGGL(k_sort_merge<decltype(c)::value>, dim3(unsigned(chunks + pieces - first)),
                         dim3(kSortThreads), 0, L.stream, a.key[0], a.pos[0], a.N, a.key[1],
                         a.pos[1], chunks, fill);
    };
    if (chunks > 1) {
      if (chunks <= 4) merge(std::integral_constant<int, 4>{});
      else if (chunks <= 16) merge(std::integral_constant<int, 16>{});
      else merge(std::integral_constant<int, 32>{});
      at = 1;
    }
    L.post(kEmbedSort);
    e = hipGetLastError();
  } else {
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
  *list = at;
  return e;
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
  if (a.status) e = launch_token_status(a.tokens, a.N, a.V, a.padding, a.status, L);
  int at = 0;
  const size_t bytes = a.accumulate ? 0 : size_t(a.V) * a.H * (a.grad_dtype == FLCE_BF16 ? 2 : 4);
  if (e == hipSuccess) e = sort_tokens(a, a.dW, bytes, L, &at);
  if (e != hipSuccess) return e;
  if (a.dtype == FLCE_F32) return sums<float, float>(a, a.key[at], a.pos[at], L);
  if (a.grad_dtype == FLCE_F32) return sums<Bf16Bits, float>(a, a.key[at], a.pos[at], L);
  return sums<Bf16Bits, Bf16Bits>(a, a.key[at], a.pos[at], L);
}

hipError_t launch_weighted_sort(const EmbedGradArgs& a, const Launcher& L, int* list) {
  const hipError_t e = sort_tokens(a, a.slot, lp_slot_bytes(a.V), L, list);
  if (e != hipSuccess) return e;
  L.pre(kEmbedSort);
  hipLaunchKernelGGL(k_token_slots, dim3(unsigned((a.N + 255) / 256)), dim3(256), 0, L.stream,
                     a.key[*list], a.N, uint32_t(a.V), a.slot);
  L.post(kEmbedSort);
  return hipGetLastError();
}

hipError_t launch_weighted_sums(const EmbedGradArgs& a, int list, const Launcher& L) {
  if (!a.weight || !a.slot || !a.keep || a.dtype != FLCE_BF16 || a.grad_dtype != FLCE_BF16)
    return hipErrorInvalidValue;
  return sums<Bf16Bits, Bf16Bits, true>(a, a.key[list], a.pos[list], L);
}

}  // namespace flce
