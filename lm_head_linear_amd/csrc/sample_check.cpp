// Synchronous argument checks and workspace plan of sampling (no HIP calls).
#include <cmath>

#include "../../include/flce.h"
#include "check_util.h"
#include "ops_plan.h"

namespace flce {

bool make_sample_plan(int64_t N, int64_t H, int64_t V, int dtype, SamplePlan* out) {
  if (N < 0 || N > kMaxGrid || H <= 0 || H > kMaxWidth || V <= 0 || V > kMaxWidth ||
      !is_dtype(dtype))
    return false;
  SamplePlan p;
  // rows of a pass: a workgroup of 1024 threads each
  int64_t fit = kSampleLogitBytes / (V * 4);
  if (fit > max_groups(1024)) fit = max_groups(1024);
  p.rows = N < fit ? N : fit;
  if (p.rows < 1) p.rows = 1;
  p.off_max = align256(size_t(p.rows) * V * 4);
  p.total = p.off_max + align256(size_t(p.rows < kFewTokens ? p.rows : kFewTokens) *
                                 ceil_div(V, 64) * 4);
  *out = p;
  return true;
}

}  // namespace flce

using namespace flce;

namespace {

// The settings, the uniform numbers and the outputs.
struct Common {
  float temperature;
  const float* temperatures;
  int32_t top_k;
  const int32_t* top_ks;
  float top_p;
  const float* top_ps;
  float min_p;
  const float* min_ps;
  float softcap;
};

bool settings_ok(const Common& c) {
  if (!(c.softcap >= 0.f) || !std::isfinite(c.softcap)) return false;
  if (!c.temperatures && (!(c.temperature >= 0.f) || !std::isfinite(c.temperature))) return false;
  if (!c.top_ks && c.top_k < 0) return false;
  if (!c.top_ps && !(c.top_p > 0.f && c.top_p <= 1.f)) return false;
  return c.min_ps || (c.min_p >= 0.f && c.min_p <= 1.f);
}

}  // namespace

extern "C" {

size_t flce_sample_logits_workspace_size(int64_t N, int64_t V, int dtype) {
  if (N < 0 || N > kMaxGrid || V <= 0 || V > kMaxWidth || !is_dtype(dtype)) return 0;
  const size_t n = align256(size_t(N) * sample_parts(N, V, dtype) * 4);
  return n ? n : 256;
}

int flce_sample_logits_check_args(const void* logits, int64_t ld_logits, int64_t N, int64_t V,
                                  const float* uniforms, float temperature,
                                  const float* temperatures, int32_t top_k,
                                  const int32_t* top_ks, float top_p, const float* top_ps,
                                  float min_p, const float* min_ps, float softcap,
                                  const int64_t* tokens, const float* logp, const void* stream,
                                  int dtype, const void* workspace, size_t workspace_bytes) {
  (void)stream;
  if (N < 0 || N > kMaxGrid || V <= 0 || V > kMaxWidth || !is_dtype(dtype)) return FLCE_ERR_ARG;
  if (N > 0 && (!logits || !uniforms || !tokens)) return FLCE_ERR_ARG;
  if (bad_ld(ld_logits, V)) return FLCE_ERR_ARG;
  if (!settings_ok({temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p, min_ps, softcap}))
    return FLCE_ERR_ARG;
  const Buf bz = matrix(logits, N, V, ld_logits, esize(dtype)), bu = vec(uniforms, N, 4),
            bt = vec(temperatures, N, 4), bk = vec(top_ks, N, 4), bp = vec(top_ps, N, 4),
            bm = vec(min_ps, N, 4), bo = vec(tokens, N, 8), bl = vec(logp, N, 4),
            wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({bo, bl, wk}, {bz, bu, bt, bk, bp, bm})) return FLCE_ERR_ARG;
  if (N > max_groups(1024)) return FLCE_ERR_UNSUPPORTED;
  for (const Buf& b : {bz, bu, bt, bk, bp, bm, bo, bl})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0 ||
      workspace_bytes < flce_sample_logits_workspace_size(N, V, dtype))
    return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

size_t flce_sample_workspace_size(int64_t N, int64_t H, int64_t V, int dtype) {
  SamplePlan p;
  return make_sample_plan(N, H, V, dtype, &p) ? p.total : 0;
}

int flce_sample_check_args(const void* h, const void* W, int64_t N, int64_t H, int64_t V,
                           const float* uniforms, float temperature, const float* temperatures,
                           int32_t top_k, const int32_t* top_ks, float top_p,
                           const float* top_ps, float min_p, const float* min_ps, float softcap,
                           const int64_t* tokens, const float* logp, const void* stream,
                           int dtype, const void* workspace, size_t workspace_bytes) {
  (void)stream;
  SamplePlan p;
  if (!make_sample_plan(N, H, V, dtype, &p)) return FLCE_ERR_ARG;
  if (!W || (N > 0 && (!h || !uniforms || !tokens))) return FLCE_ERR_ARG;
  if (!settings_ok({temperature, temperatures, top_k, top_ks, top_p, top_ps, min_p, min_ps, softcap}))
    return FLCE_ERR_ARG;
  const size_t es = esize(dtype);
  const Buf bh = matrix(h, N, H, H, es), bw = matrix(W, V, H, H, es), bu = vec(uniforms, N, 4),
            bt = vec(temperatures, N, 4), bk = vec(top_ks, N, 4), bp = vec(top_ps, N, 4),
            bm = vec(min_ps, N, 4), bo = vec(tokens, N, 8), bl = vec(logp, N, 4),
            wk = vec(workspace, int64_t(workspace_bytes), 1);
  if (clash({bo, bl, wk}, {bh, bw, bu, bt, bk, bp, bm})) return FLCE_ERR_ARG;
  for (const Buf& b : {bh, bw, bu, bt, bk, bp, bm, bo, bl})
    if (misaligned(b)) return FLCE_ERR_UNSUPPORTED;
  if (!workspace || wk.begin() % 256 != 0 || workspace_bytes < p.total) return FLCE_ERR_WORKSPACE;
  return FLCE_OK;
}

}  // extern "C"
