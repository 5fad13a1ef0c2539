// Where the tensors of a call lie, and whether two of them share memory (host only).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace sparge {

// Where a tensor's bytes lie: runs of `run` bytes, one of each head of each token,
// at three strides (in elements of `size` bytes).
struct Layout {
  int64_t at, n[3], step[3], run;
  int64_t span;  // from the first byte to the last; -1: more than there can be
};
constexpr int64_t kMaxSpan = int64_t(1) << 56;
inline Layout layout_of(const void* p, const int64_t (&n)[3], const int64_t (&stride)[3], int64_t run,
                        int64_t size) {
  Layout l = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(p)), {n[0], n[1], n[2]}, {}, run, 0};
  l.span = l.run;
  for (int k = 0; k < 3; ++k) {
    if (l.n[k] == 1) continue;
    if (l.span < 0 || stride[k] > kMaxSpan / size / l.n[k]) {
      l.span = -1;
      continue;
    }
    l.step[k] = stride[k] * size;
    l.span += l.step[k] * (l.n[k] - 1);
  }
  return l;
}

// Whether two runs, `delta` bytes apart and further by any of the dimensions'
// multiples of their steps, can share a byte: -before < delta + sum < after.  The
// largest step comes first, so where dimensions nest, which they do in views of
// a tensor, a few multiples of each are in question.  `other` is false as long as
// the two are the same run of one tensor.  More than `left` trials: taken as yes.
struct Dimension {
  int64_t step, lo, hi;  // multiples from lo to hi, 0 among them
};
inline bool runs_meet(const Dimension* d, int n, int64_t delta, int64_t before, int64_t after,
                      bool other, int& left) {
  if (--left < 0) return true;
  if (n == 0) return other && delta > -before && delta < after;
  if (d->step == 0)  // a run that repeats meets itself
    return runs_meet(d + 1, n - 1, delta, before, after, other || d->hi > 0, left);
  int64_t lo = 0, hi = 0;  // what the smaller steps can add
  for (int j = 1; j < n; ++j) lo += d[j].step * d[j].lo, hi += d[j].step * d[j].hi;
  // (Division rounds towards 0: one multiple to spare.  Of a tensor and itself one
  // order of each pair is enough.)
  const int64_t first = std::max(other ? d->lo : 0, (-before - delta - hi) / d->step - 1);
  const int64_t last = std::min(d->hi, (after - delta - lo) / d->step + 1);
  for (int64_t c = first; c <= last; ++c)
    if (runs_meet(d + 1, n - 1, delta + c * d->step, before, after, other || c != 0, left))
      return true;
  return false;
}
constexpr int kTrials = 1 << 16;
inline bool larger_step(const Dimension& a, const Dimension& b) { return a.step > b.step; }

inline bool meets_itself(const Layout& a) {
  if (a.span < 0) return true;
  Dimension d[3];
  for (int k = 0; k < 3; ++k) d[k] = {a.step[k], 1 - a.n[k], a.n[k] - 1};
  std::sort(d, d + 3, larger_step);
  // Each step clears all that the smaller ones reach: the usual case.
  int64_t reach = a.run;
  bool nested = true;
  for (int k = 2; k >= 0; --k) {
    if (d[k].hi > 0) nested = nested && d[k].step >= reach;
    reach += d[k].step * d[k].hi;
  }
  int left = kTrials;
  return !nested && runs_meet(d, 3, 0, a.run, a.run, false, left);
}

inline bool meet(const Layout& a, const Layout& b) {
  if (a.span < 0 || b.span < 0) return true;
  const int64_t delta = b.at - a.at;
  if (delta >= a.span || -delta >= b.span) return false;
  Dimension d[6];
  int n = 0;
  for (int k = 0; k < 3; ++k)
    if (a.n[k] > 1) d[n++] = {a.step[k], 1 - a.n[k], 0};
  for (int k = 0; k < 3; ++k) {
    if (b.n[k] == 1) continue;
    Dimension* same = std::find_if(d, d + n, [&](const Dimension& o) {
      return o.step == b.step[k] && o.hi == 0;
    });
    if (same == d + n) d[n++] = {b.step[k], 0, 0};
    same->hi = b.n[k] - 1;
  }
  std::sort(d, d + n, larger_step);
  int left = kTrials;
  return runs_meet(d, n, delta, b.run, a.run, true, left);
}

// Written where it is read, by the thread that read it.
inline bool same_place(const Layout& a, const Layout& b) {
  bool same = a.at == b.at && a.run == b.run;
  for (int k = 0; k < 3; ++k) same = same && a.n[k] == b.n[k] && a.step[k] == b.step[k];
  return same;
}

}  // namespace sparge
