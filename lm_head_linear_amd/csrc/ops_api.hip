// C-ABI entry points of the operators around the head's loss: checks, workspace
// carving, launches.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/flce.h"
#include "api_util.h"
#include "flce_internal.h"
#include "ops_plan.h"

using flce::Launcher;
using flce::Range;

namespace {
int status_of(hipError_t e) { return e == hipSuccess ? FLCE_OK : FLCE_ERR_HIP; }
}  // namespace

extern "C" {

int flce_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                  const void* weight, int64_t N, int64_t H, float eps, float weight_offset,
                  void* y, int64_t ld_y, void* s, int64_t ld_s, float* rstd, void* stream,
                  int dtype, int weight_dtype) {
  const int st = flce_rms_norm_check_args(x, ld_x, residual, ld_res, weight, N, H, eps,
                                          weight_offset, y, ld_y, s, ld_s, rstd, stream, dtype,
                                          weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  Range r("flce_rms_norm");
  const flce::NormArgs a{x, ld_x, residual, ld_res, weight, N, H, eps, weight_offset,
                         y, ld_y, s, ld_s, rstd, dtype, weight_dtype};
  return status_of(flce::launch_rms_norm(a, flce::make_launcher(stream)));
}

int flce_rms_norm_backward(const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds,
                           const void* s, int64_t ld_s, const void* weight, const float* rstd,
                           int64_t N, int64_t H, float weight_offset, void* dx, int64_t ld_dx,
                           void* dweight, int accumulate_dweight, void* stream, int dtype,
                           int weight_dtype, void* workspace, size_t workspace_bytes) {
  const int st = flce_rms_norm_backward_check_args(
      dy, ld_dy, ds, ld_ds, s, ld_s, weight, rstd, N, H, weight_offset, dx, ld_dx, dweight,
      accumulate_dweight, stream, dtype, weight_dtype, workspace, workspace_bytes);
  if (st != FLCE_OK) return st;
  Range r("flce_rms_norm_backward");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0) {
    if (!dweight || accumulate_dweight) return FLCE_OK;
    return status_of(
        flce::launch_zero_bytes(dweight, size_t(H) * (weight_dtype == FLCE_BF16 ? 2 : 4), L));
  }
  const flce::NormBwdArgs a{dy, ld_dy, ds, ld_ds, s, ld_s, weight, rstd, N, H, weight_offset,
                            dx, ld_dx, dweight, accumulate_dweight ? 1 : 0, dtype, weight_dtype,
                            dweight ? static_cast<float*>(workspace) : nullptr};
  return status_of(flce::launch_rms_norm_backward(a, L));
}

int flce_embedding(const int64_t* tokens, const void* W, int64_t N, int64_t H, int64_t V,
                   int64_t padding_index, float scale, void* out, int64_t ld_out, void* stream,
                   int dtype, int32_t* status) {
  const int st = flce_embedding_check_args(tokens, W, N, H, V, padding_index, scale, out, ld_out,
                                           stream, dtype, status);
  if (st != FLCE_OK) return st;
  Range r("flce_embedding");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0)
    return status ? status_of(flce::launch_token_status(tokens, 0, V, padding_index, status, L))
                  : FLCE_OK;
  const flce::EmbedArgs a{tokens, W, N, H, V, padding_index, scale, out, ld_out, dtype, status};
  return status_of(flce::launch_embedding(a, L));
}

int flce_embedding_backward(const int64_t* tokens, const void* dout, int64_t ld_dout, int64_t N,
                            int64_t H, int64_t V, int64_t padding_index, float scale, void* dW,
                            int accumulate_dW, void* stream, int dtype, int grad_dtype,
                            void* workspace, size_t workspace_bytes, int32_t* status) {
  const int st = flce_embedding_backward_check_args(tokens, dout, ld_dout, N, H, V, padding_index,
                                                    scale, dW, accumulate_dW, stream, dtype,
                                                    grad_dtype, workspace, workspace_bytes, status);
  if (st != FLCE_OK) return st;
  Range r("flce_embedding_backward");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0) {
    hipError_t e = hipSuccess;
    if (!accumulate_dW)
      e = flce::launch_zero_bytes(dW, size_t(V) * H * (grad_dtype == FLCE_BF16 ? 2 : 4), L);
    if (e == hipSuccess && status)
      e = flce::launch_token_status(tokens, 0, V, padding_index, status, L);
    return status_of(e);
  }
  flce::EmbedPlan p;
  if (!flce::make_embed_plan(N, H, V, &p)) return FLCE_ERR_ARG;
  char* ws = static_cast<char*>(workspace);
  flce::EmbedGradArgs a{tokens, dout, ld_dout, N, H, V, padding_index, scale, dW,
                        accumulate_dW ? 1 : 0, dtype, grad_dtype, status, p.window, {}, {},
                        nullptr, nullptr};
  for (int i = 0; i < 2; ++i) {
    a.key[i] = reinterpret_cast<uint32_t*>(ws + p.off_key[i]);
    a.pos[i] = reinterpret_cast<uint32_t*>(ws + p.off_pos[i]);
  }
  a.hist = reinterpret_cast<uint32_t*>(ws + p.off_hist);
  a.part = reinterpret_cast<float*>(ws + p.off_part);
  return status_of(flce::launch_embedding_backward(a, L));
}

}  // extern "C"
