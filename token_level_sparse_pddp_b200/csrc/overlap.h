// Whether tensors of a call share memory (host).
#pragma once

#include <cstdint>

namespace tlsp {

// A tensor's bytes: `run` of them at `at` plus each combination of its axes' steps.
struct Span {
  struct Axis {
    int64_t n;
    __int128 step;
  };
  __int128 at;
  int64_t run;
  int axes = 0;
  Axis axis[3];  // longer than 1, steps >= 0, longest first

  Span(const void* ptr, int64_t run_bytes) : at((__int128)(uintptr_t)ptr), run(run_bytes) {}
  Span& with(int64_t n, __int128 step) {
    if (n < 2) {
      if (n < 1) run = 0;  // no bytes
      return *this;
    }
    if (step < 0) {
      at += (n - 1) * step;
      step = -step;
    }
    int i = axes++;
    for (; i > 0 && axis[i - 1].step < step; --i) axis[i] = axis[i - 1];
    axis[i] = {n, step};
    return *this;
  }
  // Bytes from the first to behind the last, of the axes from `from` on.
  __int128 reach(int from) const {
    __int128 b = run;
    for (int i = from; i < axes; ++i) b += (axis[i].n - 1) * axis[i].step;
    return b;
  }
  // No two of its elements share memory (each axis steps over all that lies within it).
  bool distinct() const {
    for (int i = 0; i < axes; ++i)
      if (axis[i].step < reach(i + 1)) return false;
    return true;
  }
};

namespace detail {

inline __int128 floor_div(__int128 a, __int128 b) { return a / b - (a % b != 0 && (a < 0)); }

// Axes from ia of `a` against those from ib of `b`, which starts `delta` bytes behind `a`.
inline bool apart(const Span& a, int ia, const Span& b, int ib, __int128 delta, int& left) {
  if (delta >= a.reach(ia) || -delta >= b.reach(ib)) return true;
  if (--left < 0) return false;
  const bool in_a = ia < a.axes, in_b = ib < b.axes;
  if (!in_a && !in_b) return false;
  const __int128 sa = in_a ? a.axis[ia].step : -1, sb = in_b ? b.axis[ib].step : -1;
  const __int128 step = sa > sb ? sa : sb;
  // With equal steps only the difference of the two indices counts.
  const int na = sa == step ? 1 : 0, nb = sb == step ? 1 : 0;
  const __int128 wa = a.reach(ia + na), wb = b.reach(ib + nb);
  __int128 first = na ? -(__int128)(a.axis[ia].n - 1) : 0, last = nb ? b.axis[ib].n - 1 : 0;
  if (step == 0) {
    first = last = 0;
  } else {  // differences k at which the two windows touch: -wb < delta + k step < wa
    const __int128 lo = floor_div(-wb - delta, step) + 1, hi = floor_div(wa - delta - 1, step);
    first = first > lo ? first : lo;
    last = last < hi ? last : hi;
  }
  for (__int128 k = first; k <= last; ++k)
    if (!apart(a, ia + na, b, ib + nb, delta + k * step, left)) return false;
  return true;
}

}  // namespace detail

// Whether two tensors are known to have no byte in common. Exact for slices of one wider
// tensor (equal steps) and for tensors one behind the other; what takes more than a few
// dozen comparisons counts as shared.
inline bool apart(const Span& a, const Span& b) {
  if (a.run == 0 || b.run == 0) return true;
  int left = 64;
  return detail::apart(a, 0, b, 0, b.at - a.at, left);
}

}  // namespace tlsp
