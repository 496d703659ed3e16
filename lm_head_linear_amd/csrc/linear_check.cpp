// Synchronous argument checks and workspace plan of the linear transform (no HIP calls).
#include "../../include/flce.h"
#include "check_util.h"
#include "ops_plan.h"

namespace flce {

namespace {
// Half of the CUs' worth of tiles or more are left whole; others are cut until two workgroups
// stand on each CU, with eight stages at least to a segment. us of dx alone, tiles of 64 x 64,
// whole and cut:
//   bf16 over k 512 (one segment), over 2048: 4 tiles 14.1 11.1, 64 17.4 15.9, 120 21.0 19.4,
//     160 20.9 19.9, 256 22.6 24.0; over 8192: 4 37 15, 64 49 30, 120 56 43, 160 64 49, 256 74 68
//   float32 over 512: 4 15.9 13.0, 120 19.1 18.0, 160 20.2 25.0; over 2048: 4 47 15, 64 54 27,
//     120 54 36, 160 56 46, 256 66 65
// Cut for one, two or four workgroups a CU: bf16 96 tiles over 8192 42, 36 and 41; float32 over
// 2048 36, 32 and 33. At least 4, 8 or 16 stages: bf16 64 tiles over 512 10.7, 8.5 and 8.5,
// float32 14.6, 15.5 and 17.3.
LinearSplit split(int64_t tiles, int64_t K, int64_t stage) {
  LinearSplit s;
  const int64_t stages = ceil_div(K, stage);
  if (tiles <= 0 || tiles >= 128) return s;
  int64_t n = 512 / tiles;
  if (n > stages / 8) n = stages / 8;
  if (n < 2) return s;
  s.seg = ceil_div(stages, n) * stage;
  s.segs = ceil_div(K, s.seg);
  return s;
}

bool sizes_ok(int64_t N, int64_t I, int64_t O) {
  return N >= 0 && N <= kMaxGrid && I > 0 && I <= kMaxWidth && O > 0 && O <= kMaxWidth;
}
}  // namespace

bool make_linear_plan(int64_t N, int64_t I, int64_t O, int dtype, LinearPlan* out) {
  if (!sizes_ok(N, I, O) || !is_dtype(dtype)) return false;
  LinearPlan p;
  // 64 rows a workgroup where that leaves four of them for each CU, otherwise fewer (us of dz
  // and db for one, four and sixteen a CU: bf16 8192 x 1024 14.5, 12.8 and 16.9, 2048 x 1024
  // 7.7, 7.5 and 7.4, 8192 x 4096 43.7, 43.6 and 37.5; float32 8192 x 1024 18.8, 18.7 and 20.0)
  const int64_t groups = ceil_div(O * int64_t(esize(dtype)), 512);
  for (p.dz_rows = 64; p.dz_rows > 8 && groups * ceil_div(N, p.dz_rows) < 1024;) p.dz_rows /= 2;
  p.dz_parts = ceil_div(N, p.dz_rows);
  size_t off = 0;
  p.off_dz = off; off = align256(off + size_t(N) * O * esize(dtype));
  p.off_part = off; off = align256(off + size_t(p.dz_parts) * O * 4);
  const int64_t n128 = ceil_div(I, 128) * (ceil_div(N, 128) + ceil_div(O, 128));
  p.tile = linear_tile(n128, dtype);
  const int64_t stage = 128 / int64_t(esize(dtype)), cols = ceil_div(I, p.tile);
  p.dx = split(cols * ceil_div(N, p.tile), O, stage);
  p.dw = split(cols * ceil_div(O, p.tile), N, stage);
  p.off_dx = off; if (p.dx.segs > 1) off = align256(off + size_t(p.dx.segs) * N * I * 4);
  p.off_dw = off; if (p.dw.segs > 1) off = align256(off + size_t(p.dw.segs) * O * I * 4);
  p.total = off ? off : 256;
  *out = p;
  return true;
}

}  // namespace flce

using namespace flce;

namespace {

bool is_act(int a) { return a >= FLCE_ACT_NONE && a <= FLCE_ACT_SILU; }

// Tiles of 128 x 128 of a product in one grid of 256 threads each.
int64_t tiles(int64_t a, int64_t b) { return ceil_div(a, 128) * ceil_div(b, 128); }

}  // namespace

extern "C" {

int flce_linear_check_args(const void* x, int64_t ld_x, const void* weight, const void* bias,
                           const void* residual, int64_t ld_res, int64_t N, int64_t I, int64_t O,
                           int activation, const void* y, int64_t ld_y, const void* slope,
                           const void* stream, int dtype, int y_dtype) {
  (void)stream;
  if (!sizes_ok(N, I, O) || !is_dtype(dtype) || !is_dtype(y_dtype) || !is_act(activation))
    return FLCE_ERR_ARG;
  if (!weight || (N > 0 && (!x || !y))) return FLCE_ERR_ARG;
  if (bad_ld(ld_x, I) || bad_ld(ld_y, O) || (residual && bad_ld(ld_res, O))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype), ys = esize(y_dtype);
  const Buf bx = matrix(x, N, I, ld_x, es), bw = matrix(weight, O, I, I, es), bb = vec(bias, O, es),
            br = matrix(residual, N, O, ld_res, es), by = matrix(y, N, O, ld_y, ys),
            bs = matrix(slope, N, O, O, es);            // half or float: as wide as the rows
  // in place: y may be the residual
  if (overlap(by, br) && !same(by, br)) return FLCE_ERR_ARG;
  if (clash({by, bs}, {bx, bw, bb}) || overlap(bs, br)) return FLCE_ERR_ARG;
  if (dtype == FLCE_F32 && y_dtype != FLCE_F32) return FLCE_ERR_UNSUPPORTED;
  if (tiles(O, N) > max_groups(256) || ceil_div(O, 16) > max_groups(512)) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bx, bw, bb, br, by, bs})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  return FLCE_OK;
}

size_t flce_linear_backward_workspace_size(int64_t N, int64_t I, int64_t O, int dtype) {
  LinearPlan p;
  return make_linear_plan(N, I, O, dtype, &p) ? p.total : 0;
}

int flce_linear_backward_check_args(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                                    const void* weight, const void* slope, int64_t N, int64_t I,
                                    int64_t O, const void* dx, int64_t ld_dx,
                                    const void* dweight, const void* dbias, int accumulate,
                                    const void* stream, int dtype, const void* workspace,
                                    size_t workspace_bytes) {
  (void)stream; (void)accumulate;
  LinearPlan p;
  if (!make_linear_plan(N, I, O, dtype, &p)) return FLCE_ERR_ARG;
  if (N > 0 && (!dy || (dx && !weight) || (dweight && !x))) return FLCE_ERR_ARG;
  if (bad_ld(ld_dy, O) || (x && bad_ld(ld_x, I)) || (dx && bad_ld(ld_dx, I))) return FLCE_ERR_ARG;
  const size_t es = esize(dtype);
  const Buf bg = matrix(dy, N, O, ld_dy, es), bx = matrix(x, N, I, ld_x, es),
            bw = matrix(weight, O, I, I, es), bs = matrix(slope, N, O, O, es),
            bdx = matrix(dx, N, I, ld_dx, es), bdw = matrix(dweight, O, I, I, es),
            bdb = vec(dbias, O, es), wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({bdx, bdw, bdb, wk}, {bg, bx, bw, bs})) return FLCE_ERR_ARG;
  if (tiles(I, N) + 1024 + tiles(I, O) + ceil_div(O, 16) > max_groups(256) ||
      ceil_div(O, 128) * p.dz_parts > max_groups(256))
    return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bg, bx, bw, bs, bdx, bdw, bdb})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0 || workspace_bytes < p.total) return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

}  // extern "C"
