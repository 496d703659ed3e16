// The operators around the head's loss: the arguments of their launches and the
// host-side plans of their workspaces. Launches need HIP; the plans do not, so
// the checks build and run on a machine without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#include "flce_plan.h"

namespace flce {

constexpr int kBF16 = 1;      // FLCE_BF16

// ---- dropout -------------------------------------------------------------------------
// The mask (dropout.h): a value stays where its 16 bits are at least the threshold, and
// is multiplied by the scale.
struct DropSpec {
  uint64_t seed, offset;
  const int64_t* step;        // device, added to the offset; may be null
  uint32_t threshold;
  float scale;
};

inline DropSpec make_drop(double p, uint64_t seed, uint64_t offset, const int64_t* step) {
  const double t = p * 65536.0 + 0.5;
  const uint32_t threshold = t < 65535.0 ? uint32_t(t) : 65535u;
  return DropSpec{seed, offset, step, threshold, float(65536.0 / (65536.0 - threshold))};
}

struct DropoutArgs {
  const void* x;
  int64_t ld_x;
  const void* residual;       // may be null
  int64_t ld_res;
  int64_t N, H;
  DropSpec drop;
  void* out;
  int64_t ld_out;
  int dtype;
};

// Blocks of eight columns a thread takes, from kDropMany of them, which keeps grids of
// 2^34 blocks within what one holds. us with four and with one, bf16 with the residual, rows
// that are in no cache: 2^18 blocks 5.3 and 4.4, 2^20 12.4 and 11.6, 2^21 21.8 and 20.2, 2^22
// (8192 x 4096) 39.7 and 37.3, 2^23 80 and 73; float32 2^20 21.2 and 20.1, 2^22 78 and 70.
constexpr int kDropBlocks = 4;
constexpr int64_t kDropMany = int64_t(1) << 20;

// ---- root-mean-square norm ---------------------------------------------------------
struct NormArgs {
  const void* x;
  int64_t ld_x;
  const void* residual;       // null: the norm of x itself, s not written
  int64_t ld_res;
  const void* weight;
  int64_t N, H;
  float eps, offset;
  void* y;
  int64_t ld_y;
  void* s;
  int64_t ld_s;
  float* rstd;                // may be null
  int dtype, weight_dtype;
  const DropSpec* drop = nullptr;  // x's dropout; s is written then also without a residual
};

struct NormBwdArgs {
  const void* dy;
  int64_t ld_dy;
  const void* ds;             // may be null
  int64_t ld_ds;
  const void* s;
  int64_t ld_s;
  const void* weight;
  const float* rstd;
  int64_t N, H;
  float offset;
  void* dx;
  int64_t ld_dx;
  void* dweight;              // may be null: not wanted
  int accumulate;
  int dtype, weight_dtype;
  float* dw_part;             // [norm_shares(N)][H], null without dweight
  // x's dropout: dx is then masked, and the sum's gradient goes to dres (may be null)
  const DropSpec* drop = nullptr;
  void* dres = nullptr;
  int64_t ld_dres = 0;
};

// Workgroups of the norm's backward, each with a share of dw: four per CU.
constexpr int64_t kNormShares = 1024;
inline int64_t norm_shares(int64_t N) { return N < kNormShares ? N : kNormShares; }

// ---- the linear transform in front of the head ---------------------------------------
struct LinearArgs {
  const void* x;
  int64_t ld_x;
  const void* weight;         // [O][I]
  const void* bias;           // may be null
  const void* residual;       // may be null
  int64_t ld_res;
  int64_t N, I, O;
  int activation;
  void* y;
  int64_t ld_y;
  void* slope;                // may be null
  int dtype, y_dtype;
  float* maxima = nullptr;    // [N][linear_max_blocks()], of y without bias and activation
};

struct LinearBwdArgs {
  const void* dy;
  int64_t ld_dy;
  const void* x;
  int64_t ld_x;
  const void* weight;
  const void* slope;          // null: 1
  int64_t N, I, O;
  void* dx;                   // may be null
  int64_t ld_dx;
  void* dweight;              // may be null
  void* dbias;                // may be null
  int accumulate;             // dweight and dbias are added to
  int dtype;
};

// Tiles of 256 x 256 from which a bf16 product runs on the head's tiles, most of a round of the
// 256 CUs. us on these and on smaller ones, forward to 4096 columns (silu, bias, residual,
// slope), by tiles:
//   k  512: 160 44 39, 224 46 51, 256 47 53, 288 83 63, 384 85 77, 512 91 104
//   k 1024: 160 53 51, 224 55 68, 256 57 70, 288 101 84, 384 103 103, 512 111 137
//   k 4096: 128 101 90, 160 103 127, 256 120 172, 288 213 210, 384 219 258, 512 242 345
// and both gradients of I = 2048, N = O: 128 64 55, 160 78 90, 224 114 154, 288 237 243, 384
// 327 384. Little past a whole round a short k would do better on the smaller ones.
constexpr int64_t kLinearLargeTiles = 192;

// Rows up to which a forward takes the kernels that read W once (k_linear_few), and W's rows
// from which bf16 takes the head's (k_linear_wide, up to kFewTokens rows). us of the few rows'
// kernel, the wide one and tiles, bf16, k 1024:
//   W of  4096: 1 row 4.2 7.9 7.3,  16 5.0  8.1 7.7,  48  7.6 18.3  8.7,  64  8.3 20.6 7.4
//   W of  8192: 1 row 5.4 8.3 7.4,  16 6.8  8.6 7.8,  48 11.8 18.3  8.9,  64 13.4 20.6 7.9
//   W of 16384: 1 row 9.5 8.6 8.9,  16 12.7 8.8 9.5,  64 25.5 22.9 10.1, 128 - 37.8 12.9
//   W of 32768: 1 row 20 16 14,     16 26 16 15,      64 46 25 16,       128 - 40 23
//   W of 49152: 1 row 28 21 30,     16 36 22 32,      64 68 36 41,       128 - 50 51
// float32 (no wide one): W of 4096 1 row 5.2 and 10.6 on tiles, 32 8.6 10.7, 64 12.7 11.2; W of
// 16384 15.9 24.6, 32 25.4 26.2, 64 41.7 25.8. Between a W of about 8192 and 40000 rows, and
// near 64 rows of x, tiles would do better.
constexpr int64_t kLinearFew = 64, kLinearWide = 32768;

// Tiles of 128 x 128 from which a product takes those (others: of 64 x 64): one and a half
// rounds of the CUs. us on tiles of 128 and of 64, to 2048 columns, by tiles of 128:
//   bf16, k 512: 128 13.6 8.6, 256 15.5 15.8, 320 25.9 19.6, 448 27.3 24.7, 512 28.9 27.7
//   bf16, k 2048: 128 26 19, 256 29 34, 320 49 42, 448 51 56, 512 55 61
//   bf16, gradients of I = 1024: 128 25 16, 256 33 39, 320 62 58, 448 85 101, 512 102 131
//   float32, k 512: 128 43 27, 256 45 47, 320 83 57, 448 84 76, 512 85 85
//   float32, k 2048: 256 139 159, 320 271 186, 448 273 256, 512 274 289
constexpr int64_t kLinearWholeTiles = 384;
// ... and of float32, below which it takes tiles of 32 x 32. us on tiles of 64 and of 32, to
// 512 columns, by tiles of 128: k 256: 16 9.2 5.3, 32 9.7 7.3, 48 10.1 9.2, 64 10.5 10.9, 128
// 16.5 17.2; k 1024: 16 24 11, 48 25 21, 64 25 26, 128 42 47; gradients of I = 256: 32 26 23,
// 48 44 38, 64 56 58, 128 188 209.
constexpr int64_t kLinearQuarterTiles = 64;

// A gradient's product of rows x cols over k: split along k into segments of `seg` (a multiple
// of a stage) where its tiles leave CUs without work, each a partial product of its own.
struct LinearSplit {
  int64_t segs = 1, seg = 0;
};

struct LinearPlan {
  int64_t dz_rows = 8;        // rows of dz a workgroup forms (and adds up for db)
  int64_t dz_parts = 0;       // workgroups along the rows
  int64_t tile = 0;           // edge of the products' tiles, unless they run on the head's
  LinearSplit dx, dw;
  size_t off_dz = 0, off_part = 0, off_dx = 0, off_dw = 0, total = 0;
};

// The edge of the tiles of a product of n tiles of 128 x 128.
inline int64_t linear_tile(int64_t n, int dtype) {
  if (n >= kLinearWholeTiles) return 128;
  return dtype == kBF16 || n >= kLinearQuarterTiles ? 64 : 32;
}

bool make_linear_plan(int64_t N, int64_t I, int64_t O, int dtype, LinearPlan* p);

// ---- sampling ------------------------------------------------------------------------
// A setting of a call: one value, or a value a row (device).
template <class T>
struct Setting {
  const T* rows;              // null: value
  T value;
#if defined(__HIPCC__)
  __device__ __forceinline__ T at(int64_t r) const { return rows ? rows[r] : value; }
#endif
};

struct SampleArgs {
  const void* logits;         // [N][ld]
  int64_t ld, N, V;
  const float* uniforms;
  Setting<float> temperature, top_p, min_p;
  Setting<int32_t> top_k;
  float softcap;
  int64_t* tokens;
  float* logp;                // may be null
  int dtype;
  int weight_bits;            // S: weights are multiples of 2^-S of the largest
  const float* maxima = nullptr;   // [N][blocks], of equal parts of each row, if at hand
  int64_t blocks = 0, block = 0;   // how many, and a part's length
};

// Bits of a weight so that V of them sum up below 2^63, and at most what one rounding of a
// 64-bit floating-point value to a whole number holds.
inline int sample_weight_bits(int64_t V) {
  int log_v = 0;
  while ((int64_t(1) << log_v) < V) ++log_v;
  return 62 - log_v < 51 ? 62 - log_v : 51;
}

// Rows of given logits whose maxima a kernel of its own forms first (parts of 16 chunks of 16
// bytes): a few long ones, of which top-k or temperature 0 may need no more than those. 0:
// none. top-p alone reads every logit in any case. us without and with it, top-50 and greedy:
//   float32   1 x  32768  15.7 17.4   5.2  7.4      64 x  32768  16.8 19.1   5.7  8.5
//             1 x  49152  19.1 17.2   7.1  7.4      64 x  49152  20.6 18.7   7.6  8.7
//             1 x 131072  23.6 18.1  10.1  7.9      64 x 131072  24.8 23.7  11.3 11.9
//            96 x 131072  28.3 28.1  14.9 16.5      96 x  49152  22.3 19.8   8.8  9.5
//   bf16      1 x  32768  17.2 19.8   6.6  8.6      64 x  32768  18.2 21.5   6.8  9.3
//             1 x  49152  20.2 20.0   8.4  8.4      64 x  49152  21.4 21.0   9.0  9.3
//             1 x 131072  24.1 19.8  10.0  8.5      64 x 131072  25.5 22.5  11.2 10.5
inline int64_t sample_parts(int64_t N, int64_t V, int dtype) {
  const int64_t part = dtype == kBF16 ? 128 : 64;
  return N <= 64 && V >= 49152 ? (V + part - 1) / part : 0;
}

// Logits of the head form: as many rows at a time as fit these bytes. Their maxima add at most
// a 64th: 512 MiB in all.
constexpr int64_t kSampleLogitBytes = int64_t(504) << 20;

struct SamplePlan {
  int64_t rows = 0;
  size_t off_max = 0, total = 0;   // the maxima of 64 logits or more each
};

bool make_sample_plan(int64_t N, int64_t H, int64_t V, int dtype, SamplePlan* p);

// ---- embedding ---------------------------------------------------------------------
// Tokens that one workgroup sorts in LDS, tokens up to which such chunks are
// merged at once, and tokens per workgroup of the digit passes beyond that.
constexpr int64_t kSortChunk = 1024;
constexpr int64_t kSortMerge = 32768;
constexpr int64_t kSortBlock = 8192;
// Sorted tokens whose rows one workgroup adds up: 32 a wave, or 8 where that leaves
// most CUs idle (2048 x 1024 rows: 36 us with 32, 12 us with 8).
inline int64_t embed_window(int64_t N) { return N <= 8192 ? 64 : 256; }

struct EmbedArgs {
  const int64_t* tokens;
  const void* W;
  int64_t N, H, V, padding;
  float scale;
  void* out;
  int64_t ld_out;
  int dtype;
  int32_t* status;            // may be null
};

struct EmbedGradArgs {
  const int64_t* tokens;
  const void* dout;
  int64_t ld_dout, N, H, V, padding;
  float scale;
  void* dW;
  int accumulate;
  int dtype, grad_dtype;
  int32_t* status;            // may be null
  // workspace
  uint32_t* key[2];           // sorted keys and the tokens' positions, twice
  uint32_t* pos[2];
  uint32_t* hist;             // [256][blocks] digit counts (N > kSortMerge)
  float* part;                // [windows][2][H] partial rows
  // weighted form, or null (bf16 only): row i counts weight[i] times, and what the sums
  // are added to are the float32 rows of `keep`: id v's row is slot[v] - 1
  const float* weight;        // [N]
  uint32_t* slot;             // [V]
  const float* keep;          // [N][H]
};

struct EmbedPlan {
  size_t off_key[2] = {}, off_pos[2] = {}, off_hist = 0, off_part = 0, total = 0;
};

// False for sizes that are not valid.
bool make_embed_plan(int64_t N, int64_t H, int64_t V, EmbedPlan* p);
// The plan's buffers in a workspace.
inline void carve_embed(const EmbedPlan& p, char* ws, EmbedGradArgs* a) {
  for (int i = 0; i < 2; ++i) {
    a->key[i] = reinterpret_cast<uint32_t*>(ws + p.off_key[i]);
    a->pos[i] = reinterpret_cast<uint32_t*>(ws + p.off_pos[i]);
  }
  a->hist = reinterpret_cast<uint32_t*>(ws + p.off_hist);
  a->part = reinterpret_cast<float*>(ws + p.off_part);
}

// ---- token log probabilities -------------------------------------------------------
// Tokens up to which a bf16 call streams W once through the few-token kernel
// instead of the 256 x 256 tiles (see kernels_logprobs.hip for both sides).
constexpr int64_t kFewTokens = 128;
// Vocabulary rows per part of the few-token kernel (one or two parts a workgroup) and of
// the float32 one (one).
constexpr int64_t kLpRows = 64;
// Vocabulary up to which the 64-row tiles are joined with alternatives: 32 of the
// join's 1024 threads hold at most 2048 tiles.
constexpr int64_t kLpMaxTopV = int64_t(64) * 1024 * kLpRows;
// Bytes of candidates (lists, or logits) per token chunk, and tokens per chunk. The
// few-token kernel has one chunk.
constexpr int64_t kLpListBytes = int64_t(1) << 30;
constexpr int64_t kLpMaxChunk = 8192;

// Candidates that a list of 128 vocabulary rows has room for, as many as the joins'
// registers take: for more than 8 alternatives it saves the tiles a search for exactly
// top_k.
inline int64_t lp_candidates(int top_k) {
  return top_k <= 1 ? top_k : top_k <= 8 ? 8 : top_k <= 16 ? 16 : 32;
}

struct LpPlan {
  Plan p;                     // sizes (H padded), the gather's blocks; its offsets are not used
  bool few = false;           // the few-token kernel
  bool tiles = false;         // the 256 x 256 tiles (neither: float32)
  bool gather = false;        // live tokens first (bf16 tiles with tokens given)
  int top_k = 0;
  // Partials: per part_rows vocabulary rows and token the max, sum and weighted
  // sum. Candidates, 256 x 256 tiles: per list_rows rows and token up to kc of the
  // largest logits; otherwise the largest logit per part and all logits.
  int64_t part_rows = 0, parts = 0, list_rows = 0, lists = 0, kc = 0;
  int64_t nc = 0, n_chunks = 0;   // tokens per chunk
  // Elements between parts / tokens, and between lists / candidates / tokens:
  // tokens adjacent for the tiles (a workgroup joins 32), otherwise parts adjacent
  // (a workgroup joins one token).
  int64_t sp = 0, st = 0, cl = 0, ck = 0, ct = 0;
  size_t off_sc = 0, off_nt = 0, off_tokloss = 0, off_idx = 0, off_yc = 0, off_bcnt = 0,
         off_ccnt = 0, off_h = 0, off_wp = 0, off_part = 0, off_pd = 0, off_zt = 0, off_tau = 0,
         off_cv = 0, off_ci = 0, off_first = 0, off_zmax = 0, off_z = 0, total = 0;
};

bool make_lp_plan(int64_t N, int64_t H, int64_t V, int dtype, int top_k, bool tokens, LpPlan* p);
// Tokens of the largest launch: the few-token kernel takes all of a call at once.
inline int64_t lp_launch_rows(const LpPlan& q, int64_t N) { return q.few || N < q.nc ? N : q.nc; }

// Vocabulary tiles of a chunk of nt tokens whose candidates are extracted first, to
// give the others a bound; 0: all at once. A sixteenth of them, at least one round of
// 256 workgroups, and only where that leaves most of the work for after.
inline int64_t lp_first_tiles(const LpPlan& q, int64_t nt) {
  if (q.kc == 0) return 0;
  const int64_t tt = (nt + kTileBF16 - 1) / kTileBF16, tv = q.parts;
  int64_t pre = (tv + 15) / 16 < 512 ? (tv + 15) / 16 : 512;
  if (pre * tt < 256) pre = (256 + tt - 1) / tt;
  return 2 * pre <= tv ? pre : 0;
}

// The plan of the backward: the head's, with more K segments of dH where dH has up to
// 16 tiles, each of which would otherwise run a long loop over the chunk's vocabulary
// beside the many short ones of dW. us of a training step with the head's segments (at
// most four) and with 128 / tiles: 3 tokens of 178 over 43742 (1 tile) 260 and 108, 500
// of 512 over 131072 (4) 815 and 407, 300 of 1024 over 32000 (8) 251 and 183, 1000 of
// 1024 over 32000 (16) 317 and 293; with 256 / tiles the last two take 197 and 355, and
// 32 tiles lose (300 of 4096 over 32000: 482 and 526). bf16 gradients always have the
// float32 sum of dH, to which what rounding G left is added last. False for invalid sizes.
inline bool make_lp_backward_plan(int64_t N, int64_t H, int64_t V, int dtype, int grad_dtype,
                                  Plan* p) {
  if (!make_plan(N, H, V, dtype, p, true, grad_dtype)) return false;
  if (p->dtype != kBF16 || p->g_parts != 1 || N <= 0) return true;
  auto more = [&](int64_t times) {                 // behind the head's own buffers
    const size_t at = p->total;
    p->total = (at + size_t(times) * size_t(N) * p->H * sizeof(float) + 255) & ~size_t(255);
    return at;
  };
  const int64_t tiles = p->n_tok_tiles * ((p->H + kTileBF16 - 1) / kTileBF16);
  int64_t segs = tiles > 16 ? 1 : 128 / tiles < 32 ? 128 / tiles : 32;
  if (segs > p->vchunk / 512) segs = p->vchunk / 512;
  if (segs > 1 && segs > p->dh_segs) {
    p->dh_kseg = ((p->vchunk + segs - 1) / segs + 63) / 64 * 64;
    p->dh_segs = (p->vchunk + p->dh_kseg - 1) / p->dh_kseg;
    p->off_dhpart = more(p->dh_segs);
  }
  if (!p->dh_kseg && !p->need_dh_acc) {
    p->need_dh_acc = true;
    p->off_dhacc = more(1);
  }
  return true;
}
// Bytes of the slots of the ids that are labels, whole 16-byte pieces, and of their
// float32 dW rows (bf16 gradients).
inline size_t lp_slot_bytes(int64_t V) { return (size_t(V) * sizeof(uint32_t) + 255) & ~size_t(255); }
inline size_t lp_keep_bytes(int64_t N, int64_t H) {
  return (size_t(N) * size_t(H) * sizeof(float) + 255) & ~size_t(255);
}
// Whether G comes from the few-token kernel (bf16 G; the gathered rows are aligned).
inline bool lp_few_backward(const Plan& p) {
  return p.dtype == kBF16 && p.g_parts == 1 && p.N <= kFewTokens;
}

// Segment of the float32 dH product's K (vocabulary rows of a chunk): its
// ceil(N / 64) x ceil(H / 64) tiles are split until about 256 workgroups run next to
// dW's, in segments of at least 128 rows (257 x 515 over 5003: 106 us a step with 1024,
// 101 with 256).
inline int64_t lp_f32_segment(const Plan& p) {
  const int64_t tiles = ((p.N + 63) / 64) * ((p.H + 63) / 64);
  int64_t segs = tiles > 0 ? 256 / tiles : 1;
  if (segs > p.vchunk / 128) segs = p.vchunk / 128;
  if (segs < 1) segs = 1;
  return ((p.vchunk + segs - 1) / segs + 31) / 32 * 32;
}
inline size_t lp_f32_part_bytes(const Plan& p) {
  const int64_t kseg = lp_f32_segment(p), segs = (p.vchunk + kseg - 1) / kseg;
  return segs > 1 ? size_t(segs) * size_t(p.N) * size_t(p.H) * sizeof(float) : 0;
}

struct LpArgs {
  const void* h;
  const void* W;
  const int64_t* tokens;      // may be null: no given tokens
  int64_t N, H, V, ignore_index;
  float softcap, temperature;
  int top_k;
  float* logp;
  float* entropy;
  float* lse;
  float* top_logp;
  int64_t* top_ids;
  int dtype;
  int32_t* status;
};

struct LpGradArgs {
  const float* lse;
  const float* entropy;       // null without grad_entropy
  const float* grad_logp;     // may be null
  const float* grad_entropy;  // may be null
  float temperature;
  // gathered order: the lse and the gradient's coefficients
  float* lse_g;
  float* c0;
  float* c1;
  float* ca;
  float* rest;                // what rounding the given token's G left (bf16 G)
};

}  // namespace flce

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>

#include "flce_internal.h"

namespace flce {

hipError_t launch_rms_norm(const NormArgs& a, const Launcher& L);
hipError_t launch_rms_norm_backward(const NormBwdArgs& a, const Launcher& L);
hipError_t launch_linear(const LinearArgs& a, const Launcher& L);
// Parts of a row whose maxima a forward of these arguments can leave (0: none); all but the
// last are equally long: 64 columns up to 32 rows, 128 from there.
int64_t linear_max_blocks(const LinearArgs& a);
hipError_t launch_linear_backward(const LinearPlan& p, const LinearBwdArgs& a, char* ws,
                                  const Launcher& L);
// maxima: room for a.blocks of them a row, formed where a.maxima has none; may be null.
hipError_t launch_sample(const SampleArgs& a, float* maxima, const Launcher& L);
hipError_t launch_dropout(const DropoutArgs& a, const Launcher& L);
hipError_t launch_embedding(const EmbedArgs& a, const Launcher& L);
hipError_t launch_embedding_backward(const EmbedGradArgs& a, const Launcher& L);
// The weighted form in two parts: the sort, which fills a.slot (and says which of the two
// lists it leaves), and the sums.
hipError_t launch_weighted_sort(const EmbedGradArgs& a, const Launcher& L, int* list);
hipError_t launch_weighted_sums(const EmbedGradArgs& a, int list, const Launcher& L);
hipError_t launch_logprobs(const LpPlan& q, const LpArgs& a, char* ws, const Launcher& L);
// The logit gradient of vocabulary chunk `chunk` (a.g) from the coefficients,
// and the kernel that forms those.
hipError_t launch_lp_coefficients(const Plan& p, const Args& a, const LpGradArgs& g,
                                  const Launcher& L);
hipError_t launch_lp_gradient(const Plan& p, const Args& a, const LpGradArgs& g, int64_t chunk,
                              const Launcher& L);
hipError_t launch_lp_f32_products(const Plan& p, const Args& a, int64_t chunk, const Launcher& L);
hipError_t launch_token_status(const int64_t* tokens, int64_t N, int64_t V, int64_t padding,
                               int32_t* status, const Launcher& L);

}  // namespace flce
#endif
