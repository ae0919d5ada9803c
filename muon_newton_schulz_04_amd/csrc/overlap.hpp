// Whether tensors of a list share memory: host-side checks of the clip and the
// stack plans. Plain C++.
#pragma once

#include <algorithm>
#include <cstdint>
#include <vector>

namespace muon {
namespace tensor_overlap {

// A tensor's place in memory: rows of `width` bytes, `stride` bytes apart
// (one row: stride 0), from the first byte to behind the last.
struct Interval {
  uintptr_t lo, hi;
  uintptr_t width, stride;
  bool write;
};

// Whether a written span meets another one (sorted by lo).
inline bool spans_meet(const Interval* beg, const Interval* end) {
  uintptr_t max_hi_any = 0, max_hi_w = 0;
  for (const Interval* x = beg; x < end; ++x) {
    if (x->lo < max_hi_w || (x->write && x->lo < max_hi_any)) return true;
    max_hi_any = std::max(max_hi_any, x->hi);
    if (x->write) max_hi_w = std::max(max_hi_w, x->hi);
  }
  return false;
}

// The same for tensors whose spans run into each other (sorted by lo), when
// they are column slices of one matrix: all rows one stride apart, so every
// byte of a tensor lies in its columns [c, c + width) modulo the stride, and
// tensors in separate groups of columns share none. True also where that
// cannot be told (other strides, columns across the end of the stride).
inline bool slices_meet(const Interval* beg, const Interval* end) {
  uintptr_t stride = 0;
  for (const Interval* x = beg; x < end; ++x) {
    if (x->stride != 0 && stride != 0 && x->stride != stride) return true;
    stride = std::max(stride, x->stride);
  }
  if (stride == 0) return true;
  auto column = [=](const Interval& x) { return (x.lo - beg->lo) % stride; };
  std::vector<Interval> by_column(beg, end);
  for (const Interval& x : by_column)
    if (x.width > stride - column(x)) return true;
  std::stable_sort(by_column.begin(), by_column.end(),
                   [&](const Interval& x, const Interval& y) { return column(x) < column(y); });
  for (size_t i = 0, j; i < by_column.size(); i = j) {
    uintptr_t right = 0;
    for (j = i; j < by_column.size() && (j == i || column(by_column[j]) < right); ++j)
      right = std::max(right, column(by_column[j]) + by_column[j].width);
    std::sort(by_column.begin() + i, by_column.begin() + j,
              [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
    if (spans_meet(by_column.data() + i, by_column.data() + j)) return true;
  }
  return false;
}

// Whether a written tensor may share a byte with another one of the list.
inline bool overlaps(std::vector<Interval>& iv) {
  std::sort(iv.begin(), iv.end(), [](const Interval& x, const Interval& y) { return x.lo < y.lo; });
  const Interval* const p = iv.data();
  for (size_t i = 0, j; i < iv.size(); i = j) {  // runs of spans that meet
    uintptr_t hi = 0;
    for (j = i; j < iv.size() && (j == i || iv[j].lo < hi); ++j) hi = std::max(hi, iv[j].hi);
    if (spans_meet(p + i, p + j) && slices_meet(p + i, p + j)) return true;
  }
  return false;
}

}  // namespace tensor_overlap
}  // namespace muon
