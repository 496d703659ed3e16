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

int flce_linear(const void* x, int64_t ld_x, const void* weight, const void* bias,
                const void* residual, int64_t ld_res, int64_t N, int64_t I, int64_t O,
                int activation, void* y, int64_t ld_y, void* slope, void* stream, int dtype,
                int y_dtype) {
  const int st = flce_linear_check_args(x, ld_x, weight, bias, residual, ld_res, N, I, O,
                                        activation, y, ld_y, slope, stream, dtype, y_dtype);
  if (st != FLCE_OK || N == 0) return st;
  Range r("flce_linear");
  const flce::LinearArgs a{x, ld_x, weight, bias, residual, ld_res, N, I, O, activation,
                           y, ld_y, slope, dtype, y_dtype};
  return status_of(flce::launch_linear(a, flce::make_launcher(stream)));
}

int flce_linear_backward(const void* dy, int64_t ld_dy, const void* x, int64_t ld_x,
                         const void* weight, const void* slope, int64_t N, int64_t I, int64_t O,
                         void* dx, int64_t ld_dx, void* dweight, void* dbias, int accumulate,
                         void* stream, int dtype, void* workspace, size_t workspace_bytes) {
  const int st = flce_linear_backward_check_args(dy, ld_dy, x, ld_x, weight, slope, N, I, O, dx,
                                                 ld_dx, dweight, dbias, accumulate, stream, dtype,
                                                 workspace, workspace_bytes);
  if (st != FLCE_OK) return st;
  Range r("flce_linear_backward");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0) {
    const size_t es = dtype == FLCE_BF16 ? 2 : 4;
    hipError_t e = hipSuccess;
    if (dweight && !accumulate) e = flce::launch_zero_bytes(dweight, size_t(O) * I * es, L);
    if (e == hipSuccess && dbias && !accumulate) e = flce::launch_zero_bytes(dbias, size_t(O) * es, L);
    return status_of(e);
  }
  flce::LinearPlan p;
  if (!flce::make_linear_plan(N, I, O, dtype, &p)) return FLCE_ERR_ARG;
  const flce::LinearBwdArgs a{dy, ld_dy, x, ld_x, weight, slope, N, I, O, dx, ld_dx, dweight,
                              dbias, accumulate ? 1 : 0, dtype};
  return status_of(flce::launch_linear_backward(p, a, static_cast<char*>(workspace), L));
}

int flce_sample_logits(const void* logits, int64_t ld_logits, int64_t N, int64_t V,
                       const float* uniforms, float temperature, const float* temperatures,
                       int32_t top_k, const int32_t* top_ks, float top_p, const float* top_ps,
                       float min_p, const float* min_ps, float softcap, int64_t* tokens,
                       float* logp, void* stream, int dtype, void* workspace,
                       size_t workspace_bytes) {
  const int st = flce_sample_logits_check_args(logits, ld_logits, N, V, uniforms, temperature,
                                               temperatures, top_k, top_ks, top_p, top_ps, min_p,
                                               min_ps, softcap, tokens, logp, stream, dtype,
                                               workspace, workspace_bytes);
  if (st != FLCE_OK || N == 0) return st;
  Range r("flce_sample_logits");
  flce::SampleArgs a{logits, ld_logits, N, V, uniforms, {temperatures, temperature},
                           {top_ps, top_p}, {min_ps, min_p}, {top_ks, top_k}, softcap, tokens,
                           logp, dtype, flce::sample_weight_bits(V)};
  float* maxima = nullptr;
  if (top_ks || top_k > 0 || temperatures || temperature == 0.f) {
    a.blocks = flce::sample_parts(N, V, dtype);
    a.block = dtype == FLCE_BF16 ? 128 : 64;
    if (a.blocks) maxima = static_cast<float*>(workspace);
  }
  return status_of(flce::launch_sample(a, maxima, flce::make_launcher(stream)));
}

int flce_sample(const void* h, const void* W, int64_t N, int64_t H, int64_t V,
                const float* uniforms, float temperature, const float* temperatures,
                int32_t top_k, const int32_t* top_ks, float top_p, const float* top_ps,
                float min_p, const float* min_ps, float softcap, int64_t* tokens, float* logp,
                void* stream, int dtype, void* workspace, size_t workspace_bytes) {
  const int st = flce_sample_check_args(h, W, N, H, V, uniforms, temperature, temperatures, top_k,
                                        top_ks, top_p, top_ps, min_p, min_ps, softcap, tokens,
                                        logp, stream, dtype, workspace, workspace_bytes);
  if (st != FLCE_OK || N == 0) return st;
  Range range("flce_sample");
  const Launcher L = flce::make_launcher(stream);
  flce::SamplePlan p;
  if (!flce::make_sample_plan(N, H, V, dtype, &p)) return FLCE_ERR_ARG;
  const size_t es = dtype == FLCE_BF16 ? 2 : 4;
  auto from = [](auto* v, int64_t r) { return v ? v + r : v; };
  for (int64_t r = 0; r < N; r += p.rows) {
    const int64_t n = N - r < p.rows ? N - r : p.rows;
    flce::LinearArgs z{static_cast<const char*>(h) + size_t(r) * H * es, H, W, nullptr,
                             nullptr, V, n, H, V, FLCE_ACT_NONE, workspace, V, nullptr, dtype,
                             FLCE_F32};
    const int64_t blocks = flce::linear_max_blocks(z);
    if (blocks) z.maxima = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.off_max);
    hipError_t e = flce::launch_linear(z, L);
    if (e != hipSuccess) return status_of(e);
    const flce::SampleArgs a{workspace, V, n, V, uniforms + r, {from(temperatures, r), temperature},
                             {from(top_ps, r), top_p}, {from(min_ps, r), min_p},
                             {from(top_ks, r), top_k}, softcap, tokens + r, from(logp, r), FLCE_F32,
                             flce::sample_weight_bits(V), z.maxima, blocks,
                             blocks == (V + 63) / 64 ? 64 : 128};
    e = flce::launch_sample(a, nullptr, L);
    if (e != hipSuccess) return status_of(e);
  }
  return FLCE_OK;
}

int flce_dropout(const void* x, int64_t ld_x, const void* residual, int64_t ld_res, int64_t N,
                 int64_t H, double p, uint64_t seed, uint64_t offset, const int64_t* step,
                 void* out, int64_t ld_out, void* stream, int dtype) {
  const int st = flce_dropout_check_args(x, ld_x, residual, ld_res, N, H, p, seed, offset, step,
                                         out, ld_out, stream, dtype);
  if (st != FLCE_OK || N == 0) return st;
  Range r("flce_dropout");
  const flce::DropoutArgs a{x, ld_x, residual, ld_res, N, H,
                            flce::make_drop(p, seed, offset, step), out, ld_out, dtype};
  return status_of(flce::launch_dropout(a, flce::make_launcher(stream)));
}

int flce_dropout_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                      const void* weight, int64_t N, int64_t H, float eps, float weight_offset,
                      double p, uint64_t seed, uint64_t offset, const int64_t* step, void* y,
                      int64_t ld_y, void* s, int64_t ld_s, float* rstd, void* stream, int dtype,
                      int weight_dtype) {
  const int st = flce_dropout_norm_check_args(x, ld_x, residual, ld_res, weight, N, H, eps,
                                              weight_offset, p, seed, offset, step, y, ld_y, s,
                                              ld_s, rstd, stream, dtype, weight_dtype);
  if (st != FLCE_OK || N == 0) return st;
  Range r("flce_dropout_norm");
  const flce::DropSpec drop = flce::make_drop(p, seed, offset, step);
  const flce::NormArgs a{x, ld_x, residual, ld_res, weight, N, H, eps, weight_offset,
                         y, ld_y, s, ld_s, rstd, dtype, weight_dtype, &drop};
  return status_of(flce::launch_rms_norm(a, flce::make_launcher(stream)));
}

int flce_dropout_norm_backward(const void* dy, int64_t ld_dy, const void* ds, int64_t ld_ds,
                               const void* s, int64_t ld_s, const void* weight, const float* rstd,
                               int64_t N, int64_t H, float weight_offset, double p, uint64_t seed,
                               uint64_t offset, const int64_t* step, void* dx, int64_t ld_dx,
                               void* dresidual, int64_t ld_dres, void* dweight,
                               int accumulate_dweight, void* stream, int dtype, int weight_dtype,
                               void* workspace, size_t workspace_bytes) {
  const int st = flce_dropout_norm_backward_check_args(
      dy, ld_dy, ds, ld_ds, s, ld_s, weight, rstd, N, H, weight_offset, p, seed, offset, step, dx,
      ld_dx, dresidual, ld_dres, dweight, accumulate_dweight, stream, dtype, weight_dtype,
      workspace, workspace_bytes);
  if (st != FLCE_OK) return st;
  Range r("flce_dropout_norm_backward");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0) {
    if (!dweight || accumulate_dweight) return FLCE_OK;
    return status_of(
        flce::launch_zero_bytes(dweight, size_t(H) * (weight_dtype == FLCE_BF16 ? 2 : 4), L));
  }
  const flce::DropSpec drop = flce::make_drop(p, seed, offset, step);
  const flce::NormBwdArgs a{dy, ld_dy, ds, ld_ds, s, ld_s, weight, rstd, N, H, weight_offset,
                            dx, ld_dx, dweight, accumulate_dweight ? 1 : 0, dtype, weight_dtype,
                            dweight ? static_cast<float*>(workspace) : nullptr, &drop, dresidual,
                            ld_dres};
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
                        accumulate_dW ? 1 : 0, dtype, grad_dtype, status, {}, {},
                        nullptr, nullptr, nullptr};
  flce::carve_embed(p, ws, &a);
  return status_of(flce::launch_embedding_backward(a, L));
}

int flce_logprobs(const void* h, const void* W, const int64_t* tokens, int64_t N, int64_t H,
                  int64_t V, int64_t ignore_index, float softcap, float temperature, int top_k,
                  float* logp, float* entropy, float* lse, float* top_logp, int64_t* top_ids,
                  void* stream, int dtype, void* workspace, size_t workspace_bytes,
                  int32_t* status) {
  const int st = flce_logprobs_check_args(h, W, tokens, N, H, V, ignore_index, softcap,
                                          temperature, top_k, logp, entropy, lse, top_logp,
                                          top_ids, stream, dtype, workspace, workspace_bytes,
                                          status);
  if (st != FLCE_OK) return st;
  Range r("flce_logprobs");
  const Launcher L = flce::make_launcher(stream);
  if (N == 0)
    return status ? status_of(flce::launch_token_status(nullptr, 0, V, ignore_index, status, L))
                  : FLCE_OK;
  flce::LpPlan q;
  if (!flce::make_lp_plan(N, H, V, dtype, top_k, tokens != nullptr, &q)) return FLCE_ERR_ARG;
  const flce::LpArgs a{h, W, tokens, N, H, V, ignore_index, softcap, temperature, top_k,
                       logp, entropy, lse, top_logp, top_ids, dtype, status};
  return status_of(flce::launch_logprobs(q, a, static_cast<char*>(workspace), L));
}

int flce_logprobs_backward(const void* h, const void* W, const int64_t* tokens, const float* lse,
                           const float* entropy, const float* grad_logp,
                           const float* grad_entropy, int64_t N, int64_t H, int64_t V,
                           int64_t ignore_index, float softcap, float temperature, void* dH,
                           void* dW, int accumulate_dW, void* stream, int dtype, int grad_dtype,
                           void* workspace, size_t workspace_bytes, int32_t* status) {
  const int st = flce_logprobs_backward_check_args(
      h, W, tokens, lse, entropy, grad_logp, grad_entropy, N, H, V, ignore_index, softcap,
      temperature, dH, dW, accumulate_dW, stream, dtype, grad_dtype, workspace, workspace_bytes,
      status);
  if (st != FLCE_OK) return st;
  Range r("flce_logprobs_backward");
  const Launcher L = flce::make_launcher(stream);
  flce::Plan p;
  if (!flce::make_lp_backward_plan(N, H, V, dtype, grad_dtype, &p)) return FLCE_ERR_ARG;
  hipError_t e = hipSuccess;
  if (N == 0) {
    if (!accumulate_dW) e = flce::launch_zero_bytes(dW, size_t(V) * H * p.grad_elem, L);
    if (e == hipSuccess && status)
      e = flce::launch_token_status(nullptr, 0, V, ignore_index, status, L);
    return status_of(e);
  }
  char* ws = static_cast<char*>(workspace);
  char* own = ws + p.total;                         // behind the head's own workspace
  const size_t arr = (size_t(p.ld_part) * sizeof(float) + 255) & ~size_t(255);
  flce::Args a{};
  a.h = h; a.W = W; a.labels = tokens;
  a.N = N; a.H = H; a.V = V;
  a.ignore_index = ignore_index; a.softcap = softcap;
  a.num_tokens = reinterpret_cast<int64_t*>(own);
  a.dH = dH; a.dW = dW;
  a.mb_scale = 1.f; a.accumulate_dW = accumulate_dW ? 1 : 0;
  a.status = status;
  a.sc = reinterpret_cast<flce::Scalars*>(ws + p.off_scalars);
  a.tok_loss = reinterpret_cast<double*>(ws + p.off_tokloss);
  a.g = ws + p.off_g;
  a.dh_acc = p.need_dh_acc ? reinterpret_cast<float*>(ws + p.off_dhacc) : nullptr;
  a.dh_part = p.dh_kseg ? reinterpret_cast<float*>(ws + p.off_dhpart) : nullptr;
  if (p.compact) {
    a.idx = reinterpret_cast<int32_t*>(ws + p.off_idx);
    a.yc = reinterpret_cast<int64_t*>(ws + p.off_yc);
    a.bcnt = reinterpret_cast<int32_t*>(ws + p.off_bcnt);
    a.hc = ws + p.off_hc;
  }
  own += 256;
  const flce::LpGradArgs g{lse, entropy, grad_logp, grad_entropy, temperature,
                           reinterpret_cast<float*>(own), reinterpret_cast<float*>(own + arr),
                           reinterpret_cast<float*>(own + 2 * arr),
                           reinterpret_cast<float*>(own + 3 * arr),
                           reinterpret_cast<float*>(own + 4 * arr)};
  own += 5 * arr;
  if (dtype == FLCE_F32) a.dh_part = reinterpret_cast<float*>(own);
  // bf16 gradients: what rounding the given tokens' G leaves is added to their dH rows and,
  // (what was left) h over the gathered rows, to the float32 dW rows of those tokens
  const bool rest = dtype == FLCE_BF16 && grad_dtype == FLCE_BF16;
  flce::EmbedGradArgs left{};
  int list = 0;
  if (rest) {
    flce::EmbedPlan ep;
    if (!flce::make_embed_plan(N, p.H, V, &ep)) return FLCE_ERR_ARG;
    flce::carve_embed(ep, own, &left);
    left.slot = reinterpret_cast<uint32_t*>(own + ep.total);
    a.dw_keep = reinterpret_cast<float*>(own + ep.total + flce::lp_slot_bytes(V));
    a.dw_slot = left.slot;
    a.rest = g.rest;
  }
  {
    Range s("flce.setup");
    e = flce::pad_inputs(p, a, ws, true, L);
    if (e == hipSuccess && p.compact) e = flce::launch_scan_gather(p, a, false, L);
    if (e == hipSuccess && !p.compact && status)
      e = flce::launch_token_status(tokens, N, V, ignore_index, status, L);
    if (e == hipSuccess) e = flce::launch_lp_coefficients(p, a, g, L);
    if (rest) {
      left.tokens = a.yc; left.dout = a.hc; left.ld_dout = p.H;
      left.N = N; left.H = p.H; left.V = V; left.padding = ignore_index;
      left.scale = 1.f; left.dW = a.dW; left.accumulate = 1;
      left.dtype = dtype; left.grad_dtype = grad_dtype;
      left.weight = g.rest; left.keep = a.dw_keep;
      if (e == hipSuccess) e = flce::launch_weighted_sort(left, L, &list);
    }
  }
  for (int64_t c = 0; e == hipSuccess && c < p.n_chunks; ++c) {
    Range s("flce.backward_chunk");
    e = flce::launch_lp_gradient(p, a, g, c, L);
    if (e == hipSuccess)
      e = dtype == FLCE_BF16 ? flce::bf16_chunk_products(p, a, c, L)
                             : flce::launch_lp_f32_products(p, a, c, L);
  }
  if (e == hipSuccess && rest) {
    Range s("flce.rounding_rest");
    e = flce::launch_weighted_sums(left, list, L);
  }
  if (e == hipSuccess) e = flce::crop_outputs(p, ws, dH, dW, L);
  return status_of(e);
}

}  // extern "C"
