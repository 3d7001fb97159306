// Whether the memory that a call writes meets what else it writes or reads:
// sets of rows that lie along up to three axes, checked on the host before
// anything is launched.  The answer is exact (interleaved sets, as the keys and
// values of one cache, are told apart), not a comparison of address ranges.
#pragma once

#include <stdint.h>

namespace rvq {

// Rows of `row` bytes at base + sum of index * stride (bytes) over three axes.
struct RowSet {
  const void *base;
  int64_t row;
  struct Axis {
    int64_t count, stride;
  } axis[3];
};
inline RowSet row_set(const void *base, int64_t row, int64_t count, int64_t stride) {
  return {base, row, {{count, stride}, {1, 0}, {1, 0}}};
}

enum class Overlap { kNone, kSome, kUnknown };

// Whether integers k_i in [low_i, high_i] exist with -a < start + sum k_i * stride_i < b
// (`other`: not all of them 0).  Axes are taken from the longest stride to the
// shortest, each k only as far as the axes after it can still reach the goal:
// for nested layouts that is one or two values an axis.
class ReachSearch {
 public:
  using Wide = __int128;
  void add(int64_t low, int64_t high, int64_t stride) {
    if (low == 0 && high == 0) return;
    int at = n_++;
    const Wide size = stride < 0 ? -(Wide)stride : (Wide)stride;
    if (stride < 0) {  // k -> -k
      const int64_t l = low;
      low = -high, high = -l;
    }
    for (; at > 0 && axis_[at - 1].stride < size; --at) axis_[at] = axis_[at - 1];
    axis_[at] = {low, high, size};
  }
  Overlap find(Wide start, int64_t a, int64_t b, bool other) {
    rest_[n_].low = rest_[n_].high = 0;
    for (int i = n_; i-- > 0;) {
      rest_[i].low = rest_[i + 1].low + axis_[i].low * axis_[i].stride;
      rest_[i].high = rest_[i + 1].high + axis_[i].high * axis_[i].stride;
    }
    a_ = a, b_ = b, steps_ = 0;
    return walk(0, start, other);
  }

 private:
  struct Axis {
    Wide low, high, stride;
  } axis_[6];
  struct {
    Wide low, high;
  } rest_[7];
  Wide a_, b_;
  int n_ = 0, steps_ = 0;
  static constexpr int kMaxSteps = 1 << 18;  // some milliseconds; a layout that takes more is not taken

  static Wide floor_div(Wide x, Wide y) { return x >= 0 ? x / y : -((-x + y - 1) / y); }
  Overlap walk(int i, Wide at, bool other) {
    if (at + rest_[i].high <= -a_ || at + rest_[i].low >= b_) return Overlap::kNone;
    if (i == n_) return other ? Overlap::kNone : Overlap::kSome;
    const Axis &x = axis_[i];
    if (x.stride == 0) return walk(i + 1, at, false);  // low < high: some k is not 0
    if (at + x.stride + rest_[i + 1].low >= b_ && at - x.stride + rest_[i + 1].high <= -a_) return walk(i + 1, at, other);
    // -a < at + k * stride + [rest.low, rest.high] < b
    Wide k = floor_div(-a_ - at - rest_[i + 1].high, x.stride) + 1;
    Wide last = -floor_div(-(b_ - at - rest_[i + 1].low), x.stride) - 1;
    k = k < x.low ? x.low : k;
    last = last > x.high ? x.high : last;
    for (; k <= last; ++k) {
      if (++steps_ > kMaxSteps) return Overlap::kUnknown;
      const Overlap o = walk(i + 1, at + k * x.stride, other && k == 0);
      if (o != Overlap::kNone) return o;
    }
    return Overlap::kNone;
  }
};

// Whether two rows of one set overlap.  (Usual sets, each axis longer than all
// within it, need no search; nor, below, do sets with nothing between their
// first and last bytes in common.)
inline Overlap overlaps_itself(const RowSet &s) {
  ReachSearch::Wide extent = s.row;
  bool nested = true;
  for (int i = 3; i-- > 0;) {
    if (s.axis[i].count == 1) continue;
    nested = nested && s.axis[i].stride >= extent;
    extent += (ReachSearch::Wide)(s.axis[i].count - 1) * s.axis[i].stride;
  }
  if (nested) return Overlap::kNone;
  ReachSearch r;
  for (const auto &x : s.axis) r.add(-(x.count - 1), x.count - 1, x.stride);
  return r.find(0, s.row, s.row, true);
}

// The first byte of a set and the one after its last.
struct Span {
  ReachSearch::Wide first, end;
};
inline Span span(const RowSet &s) {
  const ReachSearch::Wide at = reinterpret_cast<uintptr_t>(s.base);
  Span r = {at, at + s.row};
  for (const auto &x : s.axis) {
    const ReachSearch::Wide reach = (ReachSearch::Wide)(x.count - 1) * x.stride;
    (reach < 0 ? r.first : r.end) += reach;
  }
  return r;
}

// Whether a row of s and one of t overlap.
inline Overlap overlap(const RowSet &s, const RowSet &t) {
  const Span a = span(s), b = span(t);
  if (a.end <= b.first || b.end <= a.first) return Overlap::kNone;
  ReachSearch r;
  for (int i = 0; i < 3; ++i) {
    const auto &x = s.axis[i], &y = t.axis[i];
    if (x.count > 1 && y.count > 1 && x.stride == y.stride) {  // only the difference of the two indexes counts
      r.add(-(y.count - 1), x.count - 1, x.stride);
    } else {
      r.add(0, x.count - 1, x.stride);
      r.add(-(y.count - 1), 0, y.stride);
    }
  }
  const ReachSearch::Wide start =
      (ReachSearch::Wide)reinterpret_cast<uintptr_t>(s.base) - (ReachSearch::Wide)reinterpret_cast<uintptr_t>(t.base);
  return r.find(start, s.row, t.row, false);
}

// Whether rows that are written may lie where rows of the same number and size
// are read (strides in bytes): they are the same ones, or meet none of them.
inline bool rows_apart(const void *out, int64_t out_stride, const void *in, int64_t in_stride, int64_t rows, int64_t row) {
  if (out == in && (rows <= 1 || out_stride == in_stride)) return true;
  return overlap(row_set(out, row, rows, out_stride), row_set(in, row, rows, in_stride)) == Overlap::kNone;
}

}  // namespace rvq
