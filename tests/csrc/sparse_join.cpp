// The selection of the join over bounded tiles (join_sparse.h) on the host: the threads
// of one token run one at a time from barrier to barrier, in an order chosen for each
// phase. The outcome may not depend on the order, and the passes stay within the bound
// that the header states.
#include <algorithm>
#include <condition_variable>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <random>
#include <thread>
#include <vector>

#include "../../lm_head_linear_amd/csrc/join_sparse.h"

using namespace flce;

enum Order { kRising, kFalling, kShuffled };

// One thread at a time has the turn; at a barrier it goes to the next of the phase's
// order, and from the last to the first of the next phase.
struct Barrier {
  std::mutex m;
  std::condition_variable cv;
  std::vector<int> order;
  int at = 0;
  bool any = false, result = false;
  Order kind;
  std::mt19937 rng{7};
  explicit Barrier(Order k) : order(kSparseG), kind(k) {
    for (int i = 0; i < kSparseG; ++i) order[i] = k == kFalling ? kSparseG - 1 - i : i;
    shuffle();
  }
  void shuffle() {
    if (kind == kShuffled) std::shuffle(order.begin(), order.end(), rng);
  }
  void start(int g) {
    std::unique_lock<std::mutex> l(m);
    cv.wait(l, [&] { return at < kSparseG && order[at] == g; });
  }
  long phase = 0;
  void next(int g, bool x) {
    std::unique_lock<std::mutex> l(m);
    any = any || x;
    const long mine = phase;
    if (++at == kSparseG) {
      at = 0;
      result = any;
      any = false;
      ++phase;
      shuffle();
    }
    cv.notify_all();
    cv.wait(l, [&] { return phase > mine && order[at] == g; });
  }
  void done() {
    std::unique_lock<std::mutex> l(m);
    if (++at == kSparseG) at = 0;
    cv.notify_all();
  }
};

struct Env {
  Barrier* b;
  int g;
  void sync() const { b->next(g, false); }
  bool any(bool x) const {
    b->next(g, x);
    return b->result;
  }
  int add(int* p) const { return (*p)++; }
};

static int run(const std::vector<uint64_t>& keys, int K, Order kind, const char* what) {
  static SparseKeys<1> st;
  Barrier bar(kind);
  const int64_t bound = sparse_passes(int64_t(keys.size()), K);
  std::vector<std::thread> threads;
  for (int g = 0; g < kSparseG; ++g)
    threads.emplace_back([&, g] {
      bar.start(g);
      int64_t passes = 0;
      sparse_top(st, 0, g, K, int64_t(keys.size()), Env{&bar, g}, [&](auto push) {
        if (++passes > bound && g == 0) {
          std::printf("FAIL %s K=%d order=%d: more than %lld passes\n", what, K, int(kind),
                      (long long)bound);
          std::fflush(stdout);
          std::_Exit(1);
        }
        for (size_t i = g; i < keys.size(); i += kSparseG) push(keys[i]);
      });
      bar.done();
    });
  for (auto& t : threads) t.join();
  std::vector<uint64_t> want(keys);
  std::sort(want.rbegin(), want.rend());
  want.resize(K, 0);
  for (int k = 0; k < K; ++k)
    if (st.won[0][k] != want[k]) {
      std::printf("FAIL %s K=%d order=%d: place %d\n", what, K, int(kind), k);
      return 1;
    }
  return 0;
}

int main() {
  int bad = 0;
  std::mt19937_64 rng(3);
  for (int n : {0, 1, 31, 512, 513, 1050, 8500}) {
    std::vector<uint64_t> rising(n), falling(n), mixed(n);
    for (int i = 0; i < n; ++i) {
      rising[i] = uint64_t(i + 1) << 32;
      falling[i] = uint64_t(n - i) << 32;
      mixed[i] = (rng() | 1) & ~uint64_t(0xffff);
      mixed[i] |= uint64_t(i + 1);                 // distinct
    }
    for (int K : {1, 5, 9, 20, 32})
      for (Order o : {kRising, kFalling, kShuffled}) {
        bad += run(rising, K, o, "rising");
        bad += run(falling, K, o, "falling");
        bad += run(mixed, K, o, "mixed");
      }
  }
  if (bad == 0) std::printf("the same alternatives in every order\n");
  return bad != 0;
}
