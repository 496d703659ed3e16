// The operators around the head's loss: the arguments of their launches and the
// host-side plans of their workspaces. Launches need HIP; the plans do not, so
// the checks build and run on a machine without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

#include "flce_plan.h"

namespace flce {

constexpr int kBF16 = 1;      // FLCE_BF16

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
};

// Workgroups of the norm's backward, each with a share of dw: four per CU.
constexpr int64_t kNormShares = 1024;
inline int64_t norm_shares(int64_t N) { return N < kNormShares ? N : kNormShares; }

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
