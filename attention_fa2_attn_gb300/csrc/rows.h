// rows.h -- whether strided operands share a byte (host arithmetic only).
//
// An operand is rows of `bytes` dense bytes, one for each (batch, head, position), at strides
// of their own. Two rows meet where their starts are less than a row apart, so two operands do
// where  at_b - at_a + sum over the dimensions of both of stride * index  comes within a row
// of 0: a search over the indexes, largest stride first, that leaves a branch as soon as what
// the smaller strides reach cannot bring the sum there. Dimensions of equal strides count as
// one. For layouts whose dimensions nest (all that a projection has) two or three indexes
// of a dimension are left.
#pragma once

#include <stdint.h>

namespace fa {

struct Rows {
  const void* at;
  long long stride[3];  // bytes; that of a dimension of one is not read
  long long size[3];
  long long bytes;  // of a row
};

// `n` dense bytes.
inline Rows dense_rows(const void* at, long long n) { return Rows{at, {0, 0, 0}, {1, 1, 1}, n}; }

class RowsSearch {
 public:
  // Rows of bytes_a at sum 0 against rows of bytes_b at the sum.
  RowsSearch(long long bytes_a, long long bytes_b) : a_(bytes_a), b_(bytes_b) {}

  // stride * index, index in [lo, hi]
  void term(long long stride, long long lo, long long hi) {
    if (stride == 0 || lo == hi) {
      base_ += stride * lo;
      return;
    }
    if (stride < 0) {
      const long long l = lo;
      stride = -stride;
      lo = -hi;
      hi = -l;
    }
    int i = 0;
    while (i < n_ && t_[i].stride > stride) ++i;
    if (i < n_ && t_[i].stride == stride) {
      t_[i].lo += lo;
      t_[i].hi += hi;
      return;
    }
    for (int k = n_++; k > i; --k) t_[k] = t_[k - 1];
    t_[i] = {stride, lo, hi, 0, 0};
  }

  // Whether some sum from `start` on meets; false too where the search is given up.
  bool meets(long long start) {
    long long lo = 0, hi = 0;
    for (int i = n_ - 1; i >= 0; --i) {
      t_[i].rest_lo = lo;
      t_[i].rest_hi = hi;
      lo += t_[i].stride * t_[i].lo;
      hi += t_[i].stride * t_[i].hi;
    }
    left_ = 4000;  // some 20 us: where dimensions do not nest, any number of indexes may be in reach
    return from(0, start + base_);
  }

 private:
  struct Term {
    long long stride, lo, hi, rest_lo, rest_hi;
  };
  static long long floor_div(long long x, long long y) { return x / y - (x % y < 0 ? 1 : 0); }

  bool from(int i, long long x) {
    if (i == n_) return x < a_ && x + b_ > 0;
    const Term& t = t_[i];
    // x + stride * index + rest < a_ and > -b_ for some rest
    long long lo = floor_div(-b_ - t.rest_hi - x, t.stride) + 1, hi = -floor_div(-(a_ - t.rest_lo - x), t.stride) - 1;
    if (lo < t.lo) lo = t.lo;
    if (hi > t.hi) hi = t.hi;
    for (long long k = lo; k <= hi; ++k) {
      if (--left_ < 0) return false;
      if (from(i + 1, x + t.stride * k)) return true;
    }
    return false;
  }

  Term t_[6];
  int n_ = 0, left_ = 0;
  long long a_, b_, base_ = 0;
};

// The bytes that an operand spans, from its start.
struct Span {
  long long lo, hi;
};
inline Span span_of(const Rows& a) {
  Span s = {0, a.bytes};
  for (int i = 0; i < 3; ++i)
    if (a.size[i] > 1) (a.stride[i] < 0 ? s.lo : s.hi) += a.stride[i] * (a.size[i] - 1);
  return s;
}

// Whether two operands share a byte (a null pointer: no).
inline bool rows_meet(const Rows& a, const Rows& b) {
  if (!a.at || !b.at) return false;
  const long long apart = static_cast<long long>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at));
  const Span sa = span_of(a), sb = span_of(b);
  if (apart + sb.lo >= sa.hi || apart + sb.hi <= sa.lo) return false;  // nearly always
  RowsSearch s(a.bytes, b.bytes);
  for (int i = 0; i < 3; ++i) {
    if (a.size[i] > 1) s.term(a.stride[i], 1 - a.size[i], 0);
    if (b.size[i] > 1) s.term(b.stride[i], 0, b.size[i] - 1);
  }
  return s.meets(apart);
}

// Whether two rows of one operand share a byte.
inline bool rows_meet_themselves(const Rows& a) {
  // no, where each dimension steps over all of those before it, the smallest stride first
  long long reach = a.bytes, done = 0;
  int left = 0;
  for (int i = 0; i < 3; ++i) left += a.size[i] > 1;
  for (bool nested = true; nested;) {
    if (left == 0) return false;
    int k = -1;
    for (int i = 0; i < 3; ++i)
      if (a.size[i] > 1 && a.stride[i] > done && (k < 0 || a.stride[i] < a.stride[k])) k = i;
    nested = k >= 0 && a.stride[k] >= reach;
    if (nested) {
      done = a.stride[k];
      reach += a.stride[k] * (a.size[k] - 1);
      --left;
    }
  }
  for (int lead = 0; lead < 3; ++lead) {  // the first dimension in which two rows differ
    if (a.size[lead] < 2) continue;
    RowsSearch s(a.bytes, a.bytes);
    s.term(a.stride[lead], 1, a.size[lead] - 1);
    for (int i = lead + 1; i < 3; ++i)
      if (a.size[i] > 1) s.term(a.stride[i], 1 - a.size[i], a.size[i] - 1);
    if (s.meets(0)) return true;
  }
  return false;
}

}  // namespace fa
