// Whether two strided tensors share memory.  Views of one buffer (queries and keys of a projection) interleave: their address
// ranges overlap where no element does.
#pragma once

#include <stdint.h>

namespace fa {

// Pieces of `bytes` contiguous bytes, at p + sum of stride[i] * (0 .. n[i] - 1).  Strides in bytes, not negative.
struct Pieces {
  const void* p;
  long long bytes;
  long long n[3], stride[3];
};

namespace overlap {

// Terms stride * k, lo <= k <= hi, of the distance from a piece of `a` to one of `b`.
struct Terms {
  int count = 0, left = 4096;   // steps of the search
  long long stride[6], lo[6], hi[6];
  void add(long long s, long long from, long long to) {
    if (s == 0 || from == to) return;
    int i = 0;
    while (i < count && stride[i] > s) ++i;
    if (i < count && stride[i] == s) {   // the same stride in both
      lo[i] += from;
      hi[i] += to;
      return;
    }
    for (int j = count++; j > i; --j) stride[j] = stride[j - 1], lo[j] = lo[j - 1], hi[j] = hi[j - 1];
    stride[i] = s, lo[i] = from, hi[i] = to;
  }
};

inline long long floor_div(long long a, long long b) { return a / b - (a % b < 0 ? 1 : 0); }

// Whether the terms from i on bring `at` into [from, to].
inline bool reaches(Terms& t, int i, long long at, long long from, long long to) {
  if (i == t.count) return at >= from && at <= to;
  if (--t.left < 0) return true;
  long long rest_lo = 0, rest_hi = 0;
  for (int j = i + 1; j < t.count; ++j) rest_lo += t.stride[j] * t.lo[j], rest_hi += t.stride[j] * t.hi[j];
  long long k = -floor_div(-(from - at - rest_hi), t.stride[i]), last = floor_div(to - at - rest_lo, t.stride[i]);
  if (k < t.lo[i]) k = t.lo[i];
  if (last > t.hi[i]) last = t.hi[i];
  for (; k <= last; ++k)
    if (reaches(t, i + 1, at + k * t.stride[i], from, to)) return true;
  return false;
}

}  // namespace overlap

// Exact.  The terms of the distance between two pieces, the longest stride first: where strides are nested, as those of views
// of one buffer, each leaves one or two values to try.  Where they are so unlike that 4096 steps do not settle it: true.
inline bool pieces_overlap(const Pieces& a, const Pieces& b) {
  long long span[2] = {a.bytes, b.bytes};
  for (int i = 0; i < 3; ++i) span[0] += a.stride[i] * (a.n[i] - 1), span[1] += b.stride[i] * (b.n[i] - 1);
  const long long d = (long long)(reinterpret_cast<intptr_t>(b.p) - reinterpret_cast<intptr_t>(a.p));
  if (d >= span[0] || -d >= span[1]) return false;
  overlap::Terms t;
  for (int i = 0; i < 3; ++i) {
    t.add(b.stride[i], 0, b.n[i] - 1);
    t.add(a.stride[i], -(a.n[i] - 1), 0);
  }
  return overlap::reaches(t, 0, d, -(b.bytes - 1), a.bytes - 1);
}

}  // namespace fa
