// Strided views of memory: whether one steps on itself, and whether two share
// a byte. Host only.
#pragma once

#include <stdint.h>

namespace attn {

struct View {   // element strides of batch, head, token
  long long b, h, t;
};

// Rows of `width` bytes at `base`, `n` times `step` bytes apart per dimension.
struct Rows {
  uintptr_t base;
  long long width, step[3], n[3];
};

inline Rows rows_of(const void* p, const View& s, int B, int H, int T, long long width, long long es) {
  return Rows{reinterpret_cast<uintptr_t>(p), width * es, {s.b * es, s.h * es, s.t * es}, {B, H, T}};
}

// Whether some x within [lo, hi] per dimension, not all 0 where `other`, has
//   low < delta + sum of step * x < high.
// The dimensions are tried from the largest step down, each only where what
// lies below can still reach the interval: one or two values where the steps
// are nested as in slices of one tensor. A search that grows beyond that is
// given up, with "yes".
class RowSearch {
 public:
  void add(long long step, long long lo, long long hi) {
    if (step == 0 || lo == hi) return;   // (lo == hi: both 0)
    for (int i = 0; i < n_; ++i)
      if (step_[i] == step) {
        lo_[i] += lo, hi_[i] += hi;
        return;
      }
    int i = n_++;
    for (; i > 0 && step_[i - 1] < step; --i) step_[i] = step_[i - 1], lo_[i] = lo_[i - 1], hi_[i] = hi_[i - 1];
    step_[i] = step, lo_[i] = lo, hi_[i] = hi;
  }
  bool run(long long delta, long long low, long long high, bool other) {
    low_ = low, high_ = high, budget_ = 1 << 14;
    least_[n_] = most_[n_] = 0;
    for (int i = n_ - 1; i >= 0; --i) {
      least_[i] = least_[i + 1] + step_[i] * lo_[i];
      most_[i] = most_[i + 1] + step_[i] * hi_[i];
    }
    return from(0, delta, other);
  }

 private:
  static long long floor_div(long long a, long long b) { return a / b - (a % b < 0); }   // b > 0
  bool from(int i, long long at, bool zero) {
    if (--budget_ < 0) return true;
    if (i == n_) return !zero && low_ < at && at < high_;
    const long long s = step_[i];
    const long long first = -floor_div(at + most_[i + 1] - low_ - 1, s), last = floor_div(high_ - 1 - at - least_[i + 1], s);
    for (long long x = first > lo_[i] ? first : lo_[i]; x <= last && x <= hi_[i]; ++x)
      if (from(i + 1, at + s * x, zero && x == 0)) return true;
    return false;
  }
  int n_ = 0, budget_ = 0;
  long long step_[6], lo_[6], hi_[6], least_[7], most_[7], low_ = 0, high_ = 0;
};

// Whether no two rows of the view share a byte.
inline bool distinct(const Rows& r) {
  RowSearch s;
  for (int i = 0; i < 3; ++i) {
    if (r.n[i] > 1 && r.step[i] == 0) return false;
    for (int j = 0; j < i; ++j)   // (one step up here and one down there; add() takes equal steps as one dimension)
      if (r.n[i] > 1 && r.n[j] > 1 && r.step[i] == r.step[j]) return false;
    s.add(r.step[i], 1 - r.n[i], r.n[i] - 1);
  }
  return !s.run(0, -r.width, r.width, true);
}

// Whether no row of one shares a byte with a row of the other.
inline bool apart(const Rows& a, const Rows& b) {
  RowSearch s;
  for (int i = 0; i < 3; ++i) {
    s.add(b.step[i], 0, b.n[i] - 1);
    s.add(a.step[i], 1 - a.n[i], 0);
  }
  return !s.run(static_cast<long long>(b.base) - static_cast<long long>(a.base), -b.width, a.width, false);
}

}  // namespace attn
