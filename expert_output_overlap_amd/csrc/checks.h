// Host-side argument checks that the C ABI's operators share.
#pragma once

#include <stdint.h>

#include "../../include/moe_overlap.h"

namespace {

inline int64_t elem(int dtype) { return dtype == MOE_BF16 ? 2 : 4; }

inline bool is_dtype(int t) { return t == MOE_BF16 || t == MOE_F32; }

inline bool off(const void* p, uintptr_t align) { return (uintptr_t)p % align != 0; }

struct Span {  // n bytes, or rows of `row` bytes every `stride` bytes in them
  const void* p;
  int64_t n, row = 0, stride = 0;
};

// Bytes of two buffers in common.  Rows of one stride may lie between each other's, as two slices of one wider tensor do
inline bool meet(const Span& a, const Span& b) {
  const uintptr_t p = (uintptr_t)a.p, q = (uintptr_t)b.p;
  if (!p || !q || a.n <= 0 || b.n <= 0 || p >= q + (uintptr_t)b.n || q >= p + (uintptr_t)a.n) return false;
  if (a.stride == 0 || a.stride != b.stride) return true;
  const int64_t s = a.stride, to = (int64_t)((p < q ? q - p : p - q) % (uintptr_t)s);  // from the lower one's row on
  const Span &low = p < q ? a : b, &high = p < q ? b : a;
  return to < low.row || to + high.row > s;
}

// Whether an output overlaps an input or another output; same(o, i): a pair that may be the same buffer
template <int O, int I, class F>
inline bool overlaps(const Span (&out)[O], const Span (&in)[I], F same) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (meet(out[o], in[i]) && !(out[o].p == in[i].p && same(o, i))) return true;
    for (int q = 0; q < o; ++q)
      if (meet(out[o], out[q])) return true;
  }
  return false;
}

}  // namespace
