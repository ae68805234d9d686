// args.h -- checks of the C ABI's arguments, shared by the entry points of the
// segmented products, the router and the 4-bit products. Internal to
// libgemm_f32.so.
#pragma once

#include <cstdint>

#include "../../include/segment_gemm_f32.h"
#include "segments.h"

namespace gemm {

constexpr int64_t kMaxPitch = 0x7fffffffLL;     // pitches and banks < 2^31
constexpr int64_t kMaxSpan = int64_t{1} << 44;  // elements one stack may span

struct Range {
  uintptr_t lo = 0, hi = 0;
};

inline bool overlap(const Range &a, const Range &b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool dim_ok(int64_t x) { return x >= 0 && x <= GEMM_F32_MAX_SEGMENT_SIZE; }

// A stack of matrices the call may touch: its pitch and stride, and (unless it
// is empty) its pointer. `disjoint`: a result, whose matrices must not share
// elements.
inline bool stack_ok(const SegMatrix &m, int elem, bool disjoint, Range *range) {
  if (m.ld < (m.cols > 1 ? m.cols : 1) || m.ld > kMaxPitch || m.stride < 0) return false;
  const int64_t one = matrix_extent(m.rows, m.cols, m.ld);
  if (one == 0 || m.count == 0) return true;
  if (one > kMaxSpan || (m.count > 1 && m.stride > kMaxSpan / (m.count - 1))) return false;
  const int64_t span = (m.count - 1) * m.stride + one;
  if (span > kMaxSpan) return false;
  if (disjoint && m.count > 1 && m.stride < one) return false;
  const uintptr_t p = reinterpret_cast<uintptr_t>(m.p);
  if (p == 0 || p % static_cast<uintptr_t>(elem) != 0) return false;
  range->lo = p;
  range->hi = p + static_cast<uintptr_t>(span) * elem;
  return true;
}

// `count` values of `elem` bytes at p (null allowed where optional).
inline bool array_ok(const void *p, int64_t count, int elem, bool optional, Range *range) {
  if (p == nullptr) return optional || count == 0;
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (a % static_cast<uintptr_t>(elem) != 0) return false;
  range->lo = a;
  range->hi = a + static_cast<uintptr_t>(count) * elem;
  return true;
}

}  // namespace gemm
