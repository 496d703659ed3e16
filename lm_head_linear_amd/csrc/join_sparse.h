// The top_k largest of a token's keys, found by a group of threads through a list that
// may be too short for all of them. Shared verbatim by the HIP kernel and by the host
// program of the CPU tests, which runs the threads of a group one at a time in other
// orders than a GPU does: nothing here may depend on who comes first between two
// barriers.
#pragma once

#include <cstdint>

#include "../../include/flce.h"
#include "gemm_index.h"

namespace flce {

constexpr int kSparseG = 32;                       // threads a token
constexpr int kSparseKeys = 512;                   // keys that its list holds

template <int JT>
struct SparseKeys {                                // JT tokens, in LDS
  uint64_t list[JT][kSparseKeys];
  uint64_t best[JT][kSparseG + 1], won[JT][FLCE_MAX_TOP + 1], bound[JT], floor_key[JT];
  int count[JT], kept[JT];
};

// Passes that a token of at most `keys` keys needs. A pass whose list overflows holds
// kSparseKeys distinct keys from the floor up, and raises the floor to their K-th largest:
// the kSparseKeys - K smaller ones of them are not seen again, and the K largest of all
// are, because K keys of the list reach the new floor.
FLCE_HD int64_t sparse_passes(int64_t keys, int K) { return 1 + keys / (kSparseKeys - K); }

// Thread g of token tk: feed(push) hands over its share of the token's keys, the same in
// every pass, distinct and none 0. In the end won[tk][0 .. K - 1] holds the K largest in
// order, 0 behind the last; a barrier comes before the return. Of the keys in the list
// those from a bound up are kept, the K-th largest of the threads' largest, and each
// counts the larger ones. Env: sync() and any(bool) are barriers of the workgroup, add(int*)
// counts up and gives what was there.
template <int JT, class Env, class Feed>
FLCE_HD void sparse_top(SparseKeys<JT>& st, int tk, int g, int K, int64_t keys, const Env& env,
                        const Feed& feed) {
  constexpr int G = kSparseG, CAP = kSparseKeys;
  if (g == 0) st.floor_key[tk] = 1;
  for (int64_t left = sparse_passes(keys, K); left > 0; --left) {
    if (g == 0) { st.count[tk] = 0; st.kept[tk] = 0; st.bound[tk] = 1; }
    st.won[tk][g] = 0;
    env.sync();
    const uint64_t least = st.floor_key[tk];
    feed([&](uint64_t key) {
      if (key < least) return;
      const int at = env.add(&st.count[tk]);       // any order: the keys are ranked
      if (at < CAP) st.list[tk][at] = key;
    });
    env.sync();
    const int n = st.count[tk] < CAP ? st.count[tk] : CAP;
    uint64_t mine = 0;
    for (int i = g; i < n; i += G) mine = st.list[tk][i] > mine ? st.list[tk][i] : mine;
    st.best[tk][g] = mine;
    env.sync();
    int above = 0;
    for (int i = 0; i < G; ++i) above += st.best[tk][i] > mine ? 1 : 0;
    if (mine != 0 && above == K - 1) st.bound[tk] = mine;
    env.sync();
    const uint64_t from = st.bound[tk];
    uint64_t hold[CAP / G];                        // this thread's keys from the bound up
#pragma unroll
    for (int u = 0; u < CAP / G; ++u) {
      const int i = u * G + g;
      hold[u] = i < n && st.list[tk][i] >= from ? st.list[tk][i] : 0;
    }
    env.sync();
#pragma unroll
    for (int u = 0; u < CAP / G; ++u)
      if (hold[u] != 0) st.list[tk][env.add(&st.kept[tk])] = hold[u];
    env.sync();
    const int m = st.kept[tk];
    for (int i = g; i < m; i += G) {
      const uint64_t k = st.list[tk][i];
      int larger = 0;
      for (int o = 0; o < m && larger < K; ++o) larger += st.list[tk][o] > k ? 1 : 0;
      if (larger < K) st.won[tk][larger] = k;
    }
    const bool over = st.count[tk] > CAP;
    if (!env.any(over)) break;                     // the same in all threads
    if (g == 0 && over) st.floor_key[tk] = st.won[tk][K - 1];
    env.sync();                                    // won is read: the next pass clears it
  }
}

}  // namespace flce
