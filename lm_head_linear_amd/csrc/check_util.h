// What the operators' synchronous argument checks share: sizes, buffers and their
// overlaps (no HIP calls).
#pragma once

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "../../include/flce.h"

namespace flce {
namespace {

constexpr int64_t kMaxRows = int64_t(1) << 31, kMaxWidth = int64_t(1) << 24;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
// Workgroups of `threads` threads in one grid, which holds less than 2^32 threads.
constexpr int64_t max_groups(int64_t threads) { return ((int64_t(1) << 32) - 1) / threads; }

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool is_dtype(int d) { return d == FLCE_F32 || d == FLCE_BF16; }
inline size_t esize(int d) { return d == FLCE_BF16 ? 2 : 4; }

// A buffer of a call: [rows][cols] elements of es bytes, ld apart.
struct Buf {
  const void* p;
  int64_t rows, cols, ld;
  size_t es;
  bool none() const { return !p || rows <= 0 || cols <= 0; }
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + (size_t(rows - 1) * size_t(ld) + size_t(cols)) * es; }
};
inline Buf matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  return Buf{p, rows, cols, ld, es};
}
inline Buf vec(const void* p, int64_t n, size_t es) { return Buf{p, 1, n, n, es}; }

inline bool overlap(const Buf& a, const Buf& b) {
  return !a.none() && !b.none() && a.begin() < b.end() && b.begin() < a.end();
}
inline bool same(const Buf& a, const Buf& b) {
  return a.p == b.p && a.ld == b.ld && a.es == b.es;
}
// Row strides: at least a row, and no size that leaves 64 bits.
inline bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld > (int64_t(1) << 31); }
inline bool misaligned(const Buf& b) { return !b.none() && b.begin() % b.es != 0; }

// The outputs overlap neither each other nor an input.
inline bool clash(std::initializer_list<Buf> outs, std::initializer_list<Buf> ins) {
  for (const Buf* a = outs.begin(); a != outs.end(); ++a) {
    for (const Buf* b = a + 1; b != outs.end(); ++b)
      if (overlap(*a, *b)) return true;
    for (const Buf& b : ins)
      if (overlap(*a, b)) return true;
  }
  return false;
}

}  // namespace
}  // namespace flce
