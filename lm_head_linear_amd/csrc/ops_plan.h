// The operators around the head's loss: the arguments of their launches and the
// host-side plans of their workspaces. Launches need HIP; the plans do not, so
// the checks build and run on a machine without a GPU.
#pragma once

#include <cstddef>
#include <cstdint>

namespace flce {

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
// Tokens that one workgroup sorts in LDS, and tokens per workgroup beyond that.
constexpr int64_t kSortLocal = 16384;
constexpr int64_t kSortBlock = 8192;

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
  int64_t window;             // sorted tokens per wave of the sums
  uint32_t* key[2];           // sorted keys and the tokens' positions, twice
  uint32_t* pos[2];
  uint32_t* hist;             // [256][blocks] digit counts (N > kSortLocal)
  float* part;                // [windows][2][H] partial rows
};

struct EmbedPlan {
  int64_t window = 0;
  size_t off_key[2] = {}, off_pos[2] = {}, off_hist = 0, off_part = 0, total = 0;
};

// False for sizes that are not valid.
bool make_embed_plan(int64_t N, int64_t H, int64_t V, EmbedPlan* p);

}  // namespace flce

#if defined(__HIPCC__)
#include <hip/hip_runtime.h>

#include "flce_internal.h"

namespace flce {

hipError_t launch_rms_norm(const NormArgs& a, const Launcher& L);
hipError_t launch_rms_norm_backward(const NormBwdArgs& a, const Launcher& L);
hipError_t launch_embedding(const EmbedArgs& a, const Launcher& L);
hipError_t launch_embedding_backward(const EmbedGradArgs& a, const Launcher& L);
hipError_t launch_token_status(const int64_t* tokens, int64_t N, int64_t V, int64_t padding,
                               int32_t* status, const Launcher& L);

}  // namespace flce
#endif
