// Synchronous argument checks of dropout, alone and with the norm (no HIP calls).
#include <cmath>

#include "../../include/flce.h"
#include "check_util.h"
#include "ops_plan.h"

using namespace flce;

namespace {

bool bad_p(double p) { return !(p >= 0.0 && p < 1.0); }

// Workgroups of the dropout pass in one grid.
bool grid_ok(int64_t N, int64_t H) {
  const int64_t blocks = N * ceil_div(H, 8);
  const int64_t each = 256 * (blocks >= kDropMany ? kDropBlocks : 1);
  return ceil_div(blocks, each) <= max_groups(256);
}

}  // namespace

extern "C" {

int flce_dropout_check_args(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                            int64_t N, int64_t H, double p, uint64_t seed, uint64_t offset,
                            const int64_t* step, const void* out, int64_t ld_out,
                            const void* stream, int dtype) {
  (void)stream; (void)seed; (void)offset;
  if (N < 0 || H <= 0 || !is_dtype(dtype) || bad_p(p)) return FLCE_ERR_ARG;
  if (N > kMaxGrid || H > kMaxWidth) return FLCE_ERR_ARG;
  if (N > 0 && (!x || !out)) return FLCE_ERR_ARG;
  if (bad_ld(ld_x, H) || bad_ld(ld_out, H) || (residual && bad_ld(ld_res, H))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype);
  const Buf bx = matrix(x, N, H, ld_x, es), br = matrix(residual, N, H, ld_res, es),
            bo = matrix(out, N, H, ld_out, es), bs = vec(step, 1, 8);
  // in place: out may be x or the residual
  if (overlap(bo, bx) && !same(bo, bx)) return FLCE_ERR_ARG;
  if (overlap(bo, br) && !same(bo, br)) return FLCE_ERR_ARG;
  if (overlap(bo, bs)) return FLCE_ERR_ARG;
  if (!grid_ok(N, H)) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bx, br, bo, bs})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

int flce_dropout_norm_check_args(const void* x, int64_t ld_x, const void* residual,
                                 int64_t ld_res, const void* weight, int64_t N, int64_t H,
                                 float eps, float weight_offset, double p, uint64_t seed,
                                 uint64_t offset, const int64_t* step, const void* y,
                                 int64_t ld_y, const void* s, int64_t ld_s, const float* rstd,
                                 const void* stream, int dtype, int weight_dtype) {
  (void)stream; (void)seed; (void)offset;
  if (N < 0 || H <= 0 || !is_dtype(dtype) || !is_dtype(weight_dtype)) return FLCE_ERR_ARG;
  if (N > kMaxGrid || H > kMaxWidth || bad_p(p)) return FLCE_ERR_ARG;
  if (!(eps >= 0.f) || !std::isfinite(eps) || !std::isfinite(weight_offset)) return FLCE_ERR_ARG;
  if (!weight || (N > 0 && (!x || !y || !s))) return FLCE_ERR_ARG;
  if (bad_ld(ld_x, H) || bad_ld(ld_y, H) || bad_ld(ld_s, H)) return FLCE_ERR_ARG;
  if (residual && bad_ld(ld_res, H)) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), ws = esize(weight_dtype);
  const Buf bx = matrix(x, N, H, ld_x, es), by = matrix(y, N, H, ld_y, es),
            br = matrix(residual, N, H, ld_res, es), bs = matrix(s, N, H, ld_s, es),
            bw = vec(weight, H, ws), bq = vec(rstd, N, 4), bt = vec(step, 1, 8);
  // in place: y may be x (then s may not), s may be the residual or x
  if (overlap(by, bx) && !same(by, bx)) return FLCE_ERR_ARG;
  if (overlap(bs, bx) && !same(bs, bx)) return FLCE_ERR_ARG;
  if (overlap(bs, br) && !same(bs, br)) return FLCE_ERR_ARG;
  if (clash({by}, {br, bs, bw, bt}) || clash({bs}, {bw, bt})) return FLCE_ERR_ARG;
  if (clash({bq}, {bx, br, by, bs, bw, bt})) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && weight_dtype != FLCE_F32) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bx, by, br, bs, bw, bq, bt})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

int flce_dropout_norm_backward_check_args(
    const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds, const void* s, int64_t ld_s,
    const void* weight, const float* rstd, int64_t N, int64_t H, float weight_offset, double p,
    uint64_t seed, uint64_t offset, const int64_t* step, const void* dx, int64_t ld_dx,
    const void* dresidual, int64_t ld_dres, const void* dweight, int accumulate_dweight,
    const void* stream, int dtype, int weight_dtype, const void* workspace,
    size_t workspace_bytes) {
  (void)stream; (void)accumulate_dweight; (void)seed; (void)offset;
  if (N < 0 || H <= 0 || !is_dtype(dtype) || !is_dtype(weight_dtype)) return FLCE_ERR_ARG;
  if (N > kMaxGrid || H > kMaxWidth || !std::isfinite(weight_offset) || bad_p(p))
    return FLCE_ERR_ARG;
  if (!weight || (N > 0 && (!dy || !s || !rstd || !dx))) return FLCE_ERR_ARG;
  if (bad_ld(ld_dy, H) || bad_ld(ld_s, H) || bad_ld(ld_dx, H)) return FLCE_ERR_ARG;
  if ((ds && bad_ld(ld_ds, H)) || (dresidual && bad_ld(ld_dres, H))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), ws = esize(weight_dtype);
  const Buf by = matrix(dy, N, H, ld_dy, es), bd = matrix(ds, N, H, ld_ds, es),
            bs = matrix(s, N, H, ld_s, es), bw = vec(weight, H, ws), bq = vec(rstd, N, 4),
            bx = matrix(dx, N, H, ld_dx, es), br = matrix(dresidual, N, H, ld_dres, es),
            bdw = vec(dweight, H, ws), bt = vec(step, 1, 8),
            wk = vec(dweight ? workspace : nullptr, int64_t(workspace_bytes), 1);
  // in place: dx and dresidual may each be dy or ds
  for (const Buf* o : {&bx, &br})
    for (const Buf* i : {&by, &bd})
      if (overlap(*o, *i) && !same(*o, *i)) return FLCE_ERR_ARG;
  if (clash({bx, br}, {bs, bw, bq, bdw, bt, wk})) return FLCE_ERR_ARG;
  if (clash({bdw}, {by, bd, bs, bw, bq, bt, wk})) return FLCE_ERR_ARG;
  if (clash({wk}, {by, bd, bs, bw, bq, bt})) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && weight_dtype != FLCE_F32) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {by, bd, bs, bw, bq, bx, br, bdw, bt})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (dweight) {
    if (!workspace || wk.begin() % 256 != 0) return FLCE_ERR_WORKSPACE;
    if (workspace_bytes < flce_rms_norm_backward_workspace_size(N, H)) return FLCE_ERR_WORKSPACE;
  }
  return FLCE_OK;
}

}  // extern "C"
