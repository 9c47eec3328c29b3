// The memory of one operand of a call, and whether two operands share a byte.
// Operands are rows of contiguous bytes, one or two strides apart, and may lie
// between one another's rows (the q, k and v of a fused projection), so the ends of
// their ranges do not decide.  Host only.
#pragma once

#include <algorithm>
#include <cstdint>

namespace w2v {

struct Extent {
  uintptr_t at = 0, end = 0;              // first byte, past the last one
  int64_t width = 0;                      // bytes of a row
  int64_t stride[2] = {0, 0}, n[2] = {1, 1};
};

// n0 rows stride0 bytes apart, n1 times at stride1; false if they pass 2^60 bytes,
// which no memory does.  (Strides are not negative; that of a single entry says nothing.)
inline bool make_extent(const void* p, int64_t width, int64_t stride0, int64_t n0, int64_t stride1, int64_t n1,
                        Extent* e) {
  *e = Extent();
  e->at = e->end = reinterpret_cast<uintptr_t>(p);
  if (width <= 0 || n0 <= 0 || n1 <= 0) return true;  // empty
  const __int128 bytes = static_cast<__int128>(stride0) * (n0 - 1) + static_cast<__int128>(stride1) * (n1 - 1) + width;
  if (bytes > (static_cast<__int128>(1) << 60) || e->at + static_cast<uintptr_t>(bytes) < e->at) return false;
  e->end = e->at + static_cast<uintptr_t>(bytes);
  e->width = width;
  e->stride[0] = stride0; e->n[0] = n0;
  e->stride[1] = stride1; e->n[1] = n1;
  return true;
}

// One stride between rows of two operands, and how often it may be taken.
struct ExtentAxis {
  int64_t stride, lo, hi;
};

inline int64_t floor_div(int64_t a, int64_t b) { return a / b - (a % b < 0); }  // b > 0

// Whether some lo <= c_k <= hi bring distance + sum_k c_k stride_k into [from, to];
// axes from the longest stride down.  Of each axis only those c are tried that the
// rest can still make good: one or two where strides are nested.
inline bool distance_reached(const ExtentAxis* axis, int axes, int64_t distance, int64_t from, int64_t to) {
  if (axes == 0) return from <= distance && distance <= to;
  int64_t low = 0, high = 0;  // of the other axes' sum
  for (int k = 1; k < axes; ++k) {
    low += axis[k].lo * axis[k].stride;
    high += axis[k].hi * axis[k].stride;
  }
  const int64_t first = std::max(axis->lo, -floor_div(distance + high - from, axis->stride));
  const int64_t last = std::min(axis->hi, floor_div(to - distance - low, axis->stride));
  if (axes == 1) return first <= last;
  for (int64_t c = first; c <= last; ++c)
    if (distance_reached(axis + 1, axes - 1, distance + c * axis->stride, from, to)) return true;
  return false;
}

// Whether a and b share a byte.  Rows at A and B do if -b.width < B - A < a.width.
inline bool overlap(const Extent& a, const Extent& b) {
  if (a.width == 0 || b.width == 0 || a.at >= b.end || b.at >= a.end) return false;
  ExtentAxis axis[4];
  int axes = 0;
  auto add = [&](int64_t stride, int64_t lo, int64_t hi) {
    if (lo == hi) return;
    for (int k = 0; k < axes; ++k) {
      if (axis[k].stride == stride) {
        axis[k].lo += lo;
        axis[k].hi += hi;
        return;
      }
    }
    axis[axes++] = {stride, lo, hi};
  };
  for (int k = 0; k < 2; ++k) {
    add(a.stride[k], 1 - a.n[k], 0);
    add(b.stride[k], 0, b.n[k] - 1);
  }
  std::sort(axis, axis + axes, [](const ExtentAxis& x, const ExtentAxis& y) { return x.stride > y.stride; });
  return distance_reached(axis, axes, static_cast<int64_t>(b.at - a.at), 1 - b.width, a.width - 1);
}

// Whether one of the extents written shares a byte with another one of them or with
// one that is read.
inline bool writes_overlap(const Extent* writes, int n_writes, const Extent* reads, int n_reads) {
  for (int i = 0; i < n_writes; ++i) {
    for (int k = i + 1; k < n_writes; ++k)
      if (overlap(writes[i], writes[k])) return true;
    for (int k = 0; k < n_reads; ++k)
      if (overlap(writes[i], reads[k])) return true;
  }
  return false;
}

}  // namespace w2v
