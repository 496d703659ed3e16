// Synchronous argument checks and workspace plans of the operators around the
// head's loss (no HIP calls).
#include "ops_plan.h"

#include <cmath>
#include <initializer_list>

#include "../../include/flce.h"

namespace flce {

static_assert(kBF16 == FLCE_BF16, "the header's type code");

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31, kMaxWidth = int64_t(1) << 24;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
// Workgroups of `threads` threads in one grid, which holds less than 2^32 threads.
constexpr int64_t max_groups(int64_t threads) { return ((int64_t(1) << 32) - 1) / threads; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

bool is_dtype(int d) { return d == FLCE_F32 || d == FLCE_BF16; }
size_t esize(int d) { return d == FLCE_BF16 ? 2 : 4; }

// A buffer of a call: [rows][cols] elements of es bytes, ld apart.
struct Buf {
  const void* p;
  int64_t rows, cols, ld;
  size_t es;
  bool none() const { return !p || rows <= 0 || cols <= 0; }
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + (size_t(rows - 1) * size_t(ld) + size_t(cols)) * es; }
};
Buf matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return Buf{p, rows, cols, ld, es};
}
Buf vec(const void* p, int64_t n, size_t es) { return Buf{p, 1, n, n, es}; }

bool overlap(const Buf& a, const Buf& b) {
  return !a.none() && !b.none() && a.begin() < b.end() && b.begin() < a.end();
}
bool same(const Buf& a, const Buf& b) {
  return a.p == b.p && a.ld == b.ld && a.es == b.es;
}
// Row strides: at least a row, and no size that leaves 64 bits.
bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 31); }
bool misaligned(const Buf& b) { return !b.none() && b.begin() % b.es != 0; }

// The outputs overlap neither each other nor an input.
bool clash(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf* a = outs.begin(); a != outs.end(); ++a) {
    for (const Buf* b = a + 1; b != outs.end(); ++b)
      if (overlap(*a, *b)) return true;
    for (const Buf& b : ins)
      if (overlap(*a, b)) return true;
  }
  return false;
}

// The float32 gradient's grids: tiles of 32 tokens along y, the products' tiles in one.
bool lp_f32_grids_ok(const Plan& p) {
  const int64_t ht = ceil_div(p.H, 64), segs = ceil_div(p.vchunk, lp_f32_segment(p));
  return ceil_div(p.ldg, 32) <= 65535 &&
         (ceil_div(p.N, 64) * segs + ceil_div(p.vchunk, 64)) * ht <= max_groups(256);
}

}  // namespace

bool make_embed_plan(int64_t N, int64_t H, int64_t V, EmbedPlan* p) {
  if (N < 0 || H <= 0 || V <= 0) return false;
  if (N > kMaxRows || H > kMaxWidth || V > kMaxRows) return false;
  EmbedPlan q;
  const int64_t windows = ceil_div(N, embed_window(N)), blocks = ceil_div(N, kSortBlock);
  const size_t list = align256(size_t(N) * sizeof(uint32_t));
  const int lists = N <= kSortChunk ? 1 : 2;
  size_t off = 0;
  for (int i = 0; i < lists; ++i) {
    q.off_key[i] = off; off += list;
    q.off_pos[i] = off; off += list;
  }
  if (N > kSortMerge) { q.off_hist = off; off = align256(off + size_t(256 * blocks) * 4); }
  if (windows > 1) { q.off_part = off; off = align256(off + size_t(2 * windows) * H * 4); }
  q.total = off > 0 ? off : 256;
  *p = q;
  return true;
}

bool make_lp_plan(int64_t N, int64_t H, int64_t V, int dtype, int top_k, bool tokens, LpPlan* out) {
  LpPlan q;
  if (top_k < 0 || top_k > FLCE_MAX_TOP) return false;
  if (!make_plan(N, H, V, dtype, &q.p, false, -1, 0)) return false;
  const bool bf16 = dtype == FLCE_BF16;
  q.top_k = top_k;
  q.few = bf16 && N <= kFewTokens && V <= kLpMaxTopV;
  q.tiles = bf16 && !q.few;
  q.gather = q.tiles && tokens;
  q.p.compact = q.gather;
  q.part_rows = q.tiles ? kTileBF16 : kLpRows;
  q.parts = ceil_div(V, q.part_rows);
  const int64_t step = q.tiles ? kTileBF16 : kLpRows;      // tokens per tile
  const int64_t nmax = ceil_div(N > 0 ? N : 1, step) * step;
  int64_t nc = nmax < kLpMaxChunk ? nmax : kLpMaxChunk;
  if (q.tiles) {
    q.list_rows = kTileBF16 / 2;
    q.lists = ceil_div(V, q.list_rows);
    q.kc = lp_candidates(top_k);
  }
  if (top_k > 0 && !q.few) {            // the few-token kernel takes all rows at once
    const int64_t per_token = q.tiles ? q.lists * q.kc * 5 : V * 4;
    const int64_t fit = kLpListBytes / per_token / step * step;
    if (nc > fit) nc = fit > step ? fit : step;
  }
  q.nc = nc;
  q.n_chunks = ceil_div(N, nc);
  if (q.tiles) {
    q.sp = nc; q.st = 1;
    q.ct = 1; q.ck = nc; q.cl = q.kc * nc;
  } else {
    q.sp = 1; q.st = q.parts;
  }
  size_t off = 0;
  auto take = [&](size_t bytes) { const size_t at = off; off = align256(off + bytes); return at; };
  q.off_sc = take(sizeof(Scalars));
  q.off_nt = take(sizeof(int64_t));
  if (N > 0) {
    if (q.gather) {
      q.p.n_gather_blocks = ceil_div(N, kGatherBlock);
      q.off_tokloss = take(size_t(N) * sizeof(double));
      q.off_idx = take(size_t(N) * sizeof(int32_t));
      q.off_yc = take(size_t(N) * sizeof(int64_t));
      q.off_bcnt = take(size_t(q.p.n_gather_blocks) * sizeof(int32_t));
      q.off_ccnt = take(size_t(2 * q.n_chunks) * sizeof(int64_t));
    }
    if (q.gather || (q.tiles && q.p.pad_h)) q.off_h = take(size_t(N) * q.p.H * 2);
    if (q.tiles && q.p.pad_h) q.off_wp = take(size_t(V) * q.p.H * 2);
    const int64_t rows = !q.tiles && N < nc ? N : nc;  // tokens of the largest chunk
    q.off_part = take(size_t(q.parts) * rows * 2 * sizeof(float));
    q.off_pd = take(size_t(q.parts) * rows * sizeof(float));
    q.off_zt = take(size_t(rows) * sizeof(float));
    if (top_k > 0 && !q.tiles) {
      q.off_zmax = take(size_t(q.parts) * rows * sizeof(float));
      q.off_z = take(size_t(V) * rows * sizeof(float));
    }
    if (top_k > 0 && q.tiles) {
      q.off_tau = take(size_t(nc) * sizeof(float));
      q.off_first = take(size_t(top_k) * nc * sizeof(uint64_t));
      q.off_cv = take(size_t(q.lists) * q.kc * nc * sizeof(float));
      q.off_ci = take(size_t(q.lists) * q.kc * nc);
    }
  }
  q.total = off;
  *out = q;
  return true;
}

}  // namespace flce

using namespace flce;

extern "C" {

int flce_rms_norm_check_args(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                             const void* weight, int64_t N, int64_t H, float eps,
                             float weight_offset, const void* y, int64_t ld_y, const void* s,
                             int64_t ld_s, const float* rstd, const void* stream, int dtype,
                             int weight_dtype) {
  (void)stream;
  if (N < 0 || H <= 0 || !is_dtype(dtype) || !is_dtype(weight_dtype)) return FLCE_ERR_ARG;
  if (N > kMaxGrid || H > kMaxWidth) return FLCE_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset)) return FLCE_ERR_ARG;
  if (!weight || (N > 0 && (!x || !y))) return FLCE_ERR_ARG;
  if ((residual != nullptr) != (s != nullptr) && N > 0) return FLCE_ERR_ARG;
  if (bad_ld(ld_x, H) || bad_ld(ld_y, H)) return FLCE_ERR_ARG;
  if (residual && (bad_ld(ld_res, H) || bad_ld(ld_s, H))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), ws = esize(weight_dtype);
  const Buf bx = matrix(x, N, H, ld_x, es), by = matrix(y, N, H, ld_y, es),
            br = matrix(residual, N, H, ld_res, es), bs = matrix(s, N, H, ld_s, es),
            bw = vec(weight, H, ws), bq = vec(rstd, N, 4);
  // in place: y may be x (then s may not), s may be the residual or x
  if (overlap(by, bx) && !same(by, bx)) return FLCE_ERR_ARG;
  if (overlap(bs, bx) && !same(bs, bx)) return FLCE_ERR_ARG;
  if (overlap(bs, br) && !same(bs, br)) return FLCE_ERR_ARG;
  if (overlap(by, br) || overlap(by, bs)) return FLCE_ERR_ARG;
  if (overlap(bw, by) || overlap(bw, bs)) return FLCE_ERR_ARG;
  if (clash({bq}, {bx, br, by, bs, bw})) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && weight_dtype != FLCE_F32) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bx, by, br, bs, bw, bq})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

size_t flce_rms_norm_backward_workspace_size(int64_t N, int64_t H) {
  if (N < 0 || H <= 0 || N > kMaxGrid || H > kMaxWidth) return 0;
  const size_t n = align256(size_t(norm_shares(N)) * size_t(H) * 4);
  return n ? n : 256;
}

int flce_rms_norm_backward_check_args(const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds,
                                      const void* s, int64_t ld_s, const void* weight,
                                      const float* rstd, int64_t N, int64_t H,
                                      float weight_offset, const void* dx, int64_t ld_dx,
                                      const void* dweight, int accumulate_dweight,
                                      const void* stream, int dtype, int weight_dtype,
                                      const void* workspace, size_t workspace_bytes) {
  (void)stream; (void)accumulate_dweight;
  if (N < 0 || H <= 0 || !is_dtype(dtype) || !is_dtype(weight_dtype)) return FLCE_ERR_ARG;
  if (N > kMaxGrid || H > kMaxWidth || !std::isfinite(weight_offset)) return FLCE_ERR_ARG;
  if (!weight || (N > 0 && (!dy || !s || !rstd || !dx))) return FLCE_ERR_ARG;
  if (bad_ld(ld_dy, H) || bad_ld(ld_s, H) || bad_ld(ld_dx, H)) return FLCE_ERR_ARG;
  if (ds && bad_ld(ld_ds, H)) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), ws = esize(weight_dtype);
  const Buf by = matrix(dy, N, H, ld_dy, es), bd = matrix(ds, N, H, ld_ds, es),
            bs = matrix(s, N, H, ld_s, es), bw = vec(weight, H, ws), bq = vec(rstd, N, 4),
            bx = matrix(dx, N, H, ld_dx, es), bdw = vec(dweight, H, ws),
            wk = vec(dweight ? workspace : nullptr, int64_t(workspace_bytes), 1);
  // in place: dx may be dy or ds
  if (overlap(bx, by) && !same(bx, by)) return FLCE_ERR_ARG;
  if (overlap(bx, bd) && !same(bx, bd)) return FLCE_ERR_ARG;
  if (clash({bx}, {bs, bw, bq, bdw, wk})) return FLCE_ERR_ARG;
  if (clash({bdw}, {by, bd, bs, bw, bq, wk})) return FLCE_ERR_ARG;
  if (clash({wk}, {by, bd, bs, bw, bq})) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && weight_dtype != FLCE_F32) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {by, bd, bs, bw, bq, bx, bdw})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (dweight) {
    if (!workspace || wk.begin() % 256 != 0) return FLCE_ERR_WORKSPACE;
    if (workspace_bytes < flce_rms_norm_backward_workspace_size(N, H)) return FLCE_ERR_WORKSPACE;
  }
  return FLCE_OK;
}

int flce_embedding_check_args(const int64_t* tokens, const void* W, int64_t N, int64_t H,
                              int64_t V, int64_t padding_index, float scale, const void* out,
                              int64_t ld_out, const void* stream, int dtype,
                              const int32_t* status) {
  (void)stream; (void)padding_index;
  if (N < 0 || H <= 0 || V <= 0 || !is_dtype(dtype) || !std::isfinite(scale)) return FLCE_ERR_ARG;
  EmbedPlan p;
  if (!make_embed_plan(N, H, V, &p) || bad_ld(ld_out, H)) return FLCE_ERR_ARG;
  if (!W || (N > 0 && (!tokens || !out))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype);
  const Buf bt = vec(tokens, N, 8), bw = matrix(W, V, H, H, es),
            bo = matrix(out, N, H, ld_out, es), bst = vec(status, 1, 4);
  if (clash({bo, bst}, {bt, bw})) return FLCE_ERR_ARG;
  if (ceil_div(N * ceil_div(H * int64_t(es), 2048), 4) > max_groups(256)) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bt, bw, bo, bst})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

size_t flce_embedding_backward_workspace_size(int64_t N, int64_t H, int64_t V) {
  EmbedPlan p;
  return make_embed_plan(N, H, V, &p) ? p.total : 0;
}

int flce_embedding_backward_check_args(const int64_t* tokens, const void* dout, int64_t ld_dout,
                                       int64_t N, int64_t H, int64_t V, int64_t padding_index,
                                       float scale, const void* dW, int accumulate_dW,
                                       const void* stream, int dtype, int grad_dtype,
                                       const void* workspace, size_t workspace_bytes,
                                       const int32_t* status) {
  (void)stream; (void)padding_index; (void)accumulate_dW;
  if (N < 0 || H <= 0 || V <= 0 || !is_dtype(dtype) || !is_dtype(grad_dtype)) return FLCE_ERR_ARG;
  EmbedPlan p;
  if (!std::isfinite(scale) || !make_embed_plan(N, H, V, &p) || bad_ld(ld_dout, H))
    return FLCE_ERR_ARG;
  if (!dW || (N > 0 && (!tokens || !dout))) return FLCE_ERR_ARG;
  const Buf bt = vec(tokens, N, 8), bd = matrix(dout, N, H, ld_dout, esize(dtype)),
            bw = matrix(dW, V, H, H, esize(grad_dtype)), bst = vec(status, 1, 4),
            wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({bw, bst, wk}, {bt, bd})) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && grad_dtype == FLCE_BF16) return FLCE_ERR_UNSUPPORTED;
  if (ceil_div(N, embed_window(N)) * ceil_div(H, 512) > max_groups(512) ||
      ceil_div(V * H * int64_t(esize(grad_dtype)), 65536) + ceil_div(N, kSortChunk) >
          max_groups(kSortChunk))
    return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bt, bd, bw, bst})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0 || workspace_bytes < p.total) return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

size_t flce_logprobs_workspace_size(int64_t N, int64_t H, int64_t V, int dtype, int top_k) {
  LpPlan a, b;
  if (!make_lp_plan(N, H, V, dtype, top_k, true, &a) ||
      !make_lp_plan(N, H, V, dtype, top_k, false, &b))
    return 0;
  return a.total > b.total ? a.total : b.total;
}

int flce_logprobs_check_args(const void* h, const void* W, const int64_t* tokens, int64_t N,
                             int64_t H, int64_t V, int64_t ignore_index, float softcap,
                             float temperature, int top_k, const float* logp,
                             const float* entropy, const float* lse, const float* top_logp,
                             const int64_t* top_ids, const void* stream, int dtype,
                             const void* workspace, size_t workspace_bytes,
                             const int32_t* status) {
  (void)ignore_index; (void)stream;
  if (!is_dtype(dtype)) return FLCE_ERR_ARG;
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return FLCE_ERR_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature))
    return FLCE_ERR_ARG;
  LpPlan p;
  if (!make_lp_plan(N, H, V, dtype, top_k, tokens != nullptr, &p)) return FLCE_ERR_ARG;
  if (!W || (N > 0 && !h)) return FLCE_ERR_ARG;
  if (N > 0 && ((tokens != nullptr) != (logp != nullptr))) return FLCE_ERR_ARG;
  if (N > 0 && top_k > 0 && (!top_logp || !top_ids)) return FLCE_ERR_ARG;
  if (top_k == 0 && (top_logp || top_ids)) return FLCE_ERR_ARG;
  const size_t es = esize(dtype);
  const Buf bh = matrix(h, N, H, H, es), bw = matrix(W, V, H, H, es), bt = vec(tokens, N, 8),
            bl = vec(logp, N, 4), be = vec(entropy, N, 4), bz = vec(lse, N, 4),
            bv = vec(top_logp, N * top_k, 4), bi = vec(top_ids, N * top_k, 8),
            bs = vec(status, 1, 4), wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({bl, be, bz, bv, bi, bs, wk}, {bh, bw, bt})) return FLCE_ERR_ARG;
  if (dtype == FLCE_BF16 && !bf16_shape_ok(N, p.p.H, V)) return FLCE_ERR_UNSUPPORTED;
  if (top_k > 0 && !p.tiles && V > kLpMaxTopV) return FLCE_ERR_UNSUPPORTED;
  if (dtype == FLCE_F32 && ceil_div(V, 64) > max_groups(256)) return FLCE_ERR_UNSUPPORTED;
  const uintptr_t mask = dtype == FLCE_BF16 ? 15u : 3u;
  if ((bw.begin() & mask) || (N > 0 && (bh.begin() & mask))) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bt, bl, be, bz, bv, bi, bs})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0) return FLCE_ERR_WORKSPACE;
  if (workspace_bytes < flce_logprobs_workspace_size(N, H, V, dtype, top_k))
    return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

size_t flce_logprobs_backward_workspace_size(int64_t N, int64_t H, int64_t V, int dtype,
                                             int grad_dtype) {
  Plan p;
  if (!make_lp_backward_plan(N, H, V, dtype, grad_dtype, &p)) return 0;
  // the head's backward, its dummy count, the token coefficients, and the partial
  // products of a split float32 dH, or what adds the part of the given tokens' G that
  // rounding to bf16 left: a sort, the slots and the float32 dW rows of those tokens
  size_t more = 0;
  if (dtype == FLCE_F32) more = align256(lp_f32_part_bytes(p));
  else if (grad_dtype == FLCE_BF16) {
    EmbedPlan e;
    if (!make_embed_plan(N, p.H, V, &e)) return 0;
    more = e.total + lp_slot_bytes(V) + lp_keep_bytes(N, p.H);
  }
  return p.total + 256 + 5 * align256(size_t(p.ld_part) * sizeof(float)) + more;
}

int flce_logprobs_backward_check_args(const void* h, const void* W, const int64_t* tokens,
                                      const float* lse, const float* entropy,
                                      const float* grad_logp, const float* grad_entropy,
                                      int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                                      float softcap, float temperature, const void* dH,
                                      const void* dW, int accumulate_dW, const void* stream,
                                      int dtype, int grad_dtype, const void* workspace,
                                      size_t workspace_bytes, const int32_t* status) {
  (void)ignore_index; (void)stream; (void)accumulate_dW;
  if (!is_dtype(dtype) || !is_dtype(grad_dtype)) return FLCE_ERR_ARG;
  if (!(softcap >= 0.f) || !std::isfinite(softcap)) return FLCE_ERR_ARG;
  if (!(temperature > 0.f) || !std::isfinite(temperature) || !std::isfinite(1.f / temperature))
    return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && grad_dtype == FLCE_BF16) return FLCE_ERR_UNSUPPORTED;
  Plan p;
  if (!make_plan(N, H, V, dtype, &p, true, grad_dtype)) return FLCE_ERR_ARG;
  if (!W || !dW || (N > 0 && (!h || !dH || !tokens || !lse))) return FLCE_ERR_ARG;
  if (N > 0 && !grad_logp && !grad_entropy) return FLCE_ERR_ARG;
  if (N > 0 && grad_entropy && !entropy) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), gs = esize(grad_dtype);
  const Buf bh = matrix(h, N, H, H, es), bw = matrix(W, V, H, H, es), bt = vec(tokens, N, 8),
            bz = vec(lse, N, 4), be = vec(entropy, N, 4), ga = vec(grad_logp, N, 4),
            gb = vec(grad_entropy, N, 4), dh = matrix(dH, N, H, H, gs),
            dw = matrix(dW, V, H, H, gs), bs = vec(status, 1, 4),
            wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({dh, dw, bs, wk}, {bh, bw, bt, bz, be, ga, gb})) return FLCE_ERR_ARG;
  if (dtype == FLCE_BF16 && !bf16_shape_ok(N, p.H, V)) return FLCE_ERR_UNSUPPORTED;
  if (dtype == FLCE_F32 && !lp_f32_grids_ok(p)) return FLCE_ERR_UNSUPPORTED;
  const uintptr_t mask = dtype == FLCE_BF16 ? 15u : 3u;
  if (((bw.begin() | dw.begin()) & mask) || (N > 0 && ((bh.begin() | dh.begin()) & mask)))
    return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bt, bz, be, ga, gb, bs})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0) return FLCE_ERR_WORKSPACE;
  if (workspace_bytes < flce_logprobs_backward_workspace_size(N, H, V, dtype, grad_dtype))
    return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

}  // extern "C"
