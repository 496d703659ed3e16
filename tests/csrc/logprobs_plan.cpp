// The log probabilities' workspace (ops_plan.h) against what their launches write, for
// sizes on both sides of every rule: a launch of the rows it is given must stay within
// each buffer, and the buffers within the total and apart.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <utility>
#include <vector>

#include "../../include/flce.h"
#include "../../lm_head_linear_amd/csrc/ops_plan.h"

using namespace flce;

static int bad = 0;

static void check(int64_t N, int64_t H, int64_t V, int dtype, int top_k, bool tokens) {
  LpPlan q;
  if (!make_lp_plan(N, H, V, dtype, top_k, tokens, &q)) return;
  const int64_t rows = lp_launch_rows(q, N);       // of the largest launch
  std::vector<std::pair<size_t, size_t>> used;     // begin, end in bytes
  auto add = [&](size_t off, int64_t n, size_t es) { used.push_back({off, off + size_t(n) * es}); };
  if (q.tiles) {
    // partials [part][token], candidates [list][candidate][token], keys and tau
    add(q.off_part, (q.parts - 1) * q.sp + (rows - 1) * q.st + 1, 8);
    add(q.off_pd, (q.parts - 1) * q.sp + (rows - 1) * q.st + 1, 4);
    add(q.off_zt, rows, 4);
    if (top_k > 0) {
      const int64_t last = (q.lists - 1) * q.cl + (q.kc - 1) * q.ck + (rows - 1) * q.ct + 1;
      add(q.off_cv, std::max(last, rows * q.lists * q.kc), 4);   // or a token's together
      add(q.off_ci, std::max(last, rows * q.lists * q.kc), 1);
      add(q.off_tau, rows, 4);
      add(q.off_first, (top_k - 1) * q.nc + rows, 8);
    }
  } else {
    // a token's parts together; all logits and each part's largest with alternatives
    add(q.off_part, (rows - 1) * q.st + (q.parts - 1) * q.sp + 1, 8);
    add(q.off_pd, (rows - 1) * q.st + (q.parts - 1) * q.sp + 1, 4);
    add(q.off_zt, rows, 4);
    if (top_k > 0) {
      add(q.off_zmax, (rows - 1) * q.st + (q.parts - 1) * q.sp + 1, 4);
      add(q.off_z, rows * V, 4);
    }
  }
  std::sort(used.begin(), used.end());
  size_t end = 0;
  for (auto& u : used) {
    if (u.first < end || u.second > q.total) {
      std::printf("FAIL N=%lld H=%lld V=%lld dtype=%d top_k=%d: bytes %zu to %zu behind %zu of %zu\n",
                  (long long)N, (long long)H, (long long)V, dtype, top_k, u.first, u.second, end,
                  q.total);
      ++bad;
      return;
    }
    end = u.second;
  }
  if (!q.few && (q.n_chunks - 1) * q.nc >= N) { std::printf("FAIL chunks\n"); ++bad; }
  if (q.n_chunks * q.nc < N) { std::printf("FAIL chunks end early\n"); ++bad; }
}

int main() {
  for (int64_t N : {1, 63, 64, 65, 100, 127, 128, 129, 255, 257, 1000, 8191, 8192, 8193, 20000})
    for (int64_t V : {1, 64, 255, 257, 1000, 32000, 131072, 262144, 2097152, 2097153, 3000000,
                      4194304, 4194305, 6000001})
      for (int64_t H : {1, 8, 133})
        for (int dtype : {FLCE_F32, FLCE_BF16})
          for (int k : {0, 1, 3, 8, 9, 17, 32})
            for (bool tokens : {false, true}) check(N, H, V, dtype, k, tokens);
  if (bad == 0) std::printf("all launches within their workspace\n");
  return bad != 0;
}
