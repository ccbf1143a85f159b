// Whether two strided tensors share a byte (host only, no CUDA).
//
// Ranges of addresses tell tensors of their own apart.  Views of one allocation
// (queries and keys out of one projection, the two pools of a layer) lie between
// one another's rows; for those the question is whether
//   -(bytes of b's row) < a - b + sum_i c_i s_i < bytes of a's row
// has a solution in whole numbers c_i within the axes' sizes.  Equal strides of the
// two are one number.  From the largest stride down, only those c are followed
// whose rest can still reach the interval: one or two, where each stride steps over
// the smaller ones.  Views for which that does not hold and which take more than
// kMostSteps count as sharing.
#pragma once

#include <stdint.h>

namespace sca {

struct Rows {
  const void* base;
  int64_t bytes;              // of a row, contiguous
  int64_t stride[3], n[3];    // in bytes, >= 0; sizes, >= 1
};

namespace disjoint {

using Wide = __int128;        // sizes times strides pass 64 bits
constexpr int kMostSteps = 4096;

struct Search {
  Wide s[6], lo[6], hi[6], low, high;   // strides, what their numbers may be, the open interval
  int count, steps;

  // some sum of axis i and on, added to x, lies in the interval
  bool reaches(int i, Wide x) {
    if (++steps > kMostSteps) return true;
    if (i == count) return x > low && x < high;
    Wide least = 0, most = 0;           // of the axes behind i
    for (int j = i + 1; j < count; ++j) {
      least += lo[j] * s[j];
      most += hi[j] * s[j];
    }
    // x + c s + most > low and x + c s + least < high
    auto floor_div = [](Wide u, Wide v) { return u >= 0 ? u / v : -((-u + v - 1) / v); };
    Wide from = floor_div(low - x - most, s[i]) + 1, to = -floor_div(-(high - x - least), s[i]) - 1;
    from = from > lo[i] ? from : lo[i];
    to = to < hi[i] ? to : hi[i];
    for (Wide c = from; c <= to; ++c)
      if (reaches(i + 1, x + c * s[i])) return true;
    return false;
  }
};

}  // namespace disjoint

inline bool share_bytes(const Rows& a, const Rows& b) {
  using disjoint::Wide;
  const Wide a0 = reinterpret_cast<uintptr_t>(a.base), b0 = reinterpret_cast<uintptr_t>(b.base);
  Wide ea = a.bytes, eb = b.bytes;
  for (int i = 0; i < 3; ++i) {
    ea += static_cast<Wide>(a.n[i] - 1) * a.stride[i];
    eb += static_cast<Wide>(b.n[i] - 1) * b.stride[i];
  }
  if (a0 + ea <= b0 || b0 + eb <= a0) return false;
  disjoint::Search q = {};
  q.low = -static_cast<Wide>(a.bytes);
  q.high = b.bytes;
  auto add = [&](Wide s, Wide lo, Wide hi) {
    if (s == 0 || lo == hi) return;
    int i = 0;
    while (i < q.count && q.s[i] > s) ++i;
    if (i == q.count || q.s[i] != s) {
      for (int j = q.count++; j > i; --j) {
        q.s[j] = q.s[j - 1];
        q.lo[j] = q.lo[j - 1];
        q.hi[j] = q.hi[j - 1];
      }
      q.s[i] = s;
      q.lo[i] = q.hi[i] = 0;
    }
    q.lo[i] += lo;
    q.hi[i] += hi;
  };
  for (int i = 0; i < 3; ++i) {
    add(a.stride[i], 0, a.n[i] - 1);
    add(b.stride[i], 1 - b.n[i], 0);
  }
  return q.reaches(0, a0 - b0);
}

}  // namespace sca
