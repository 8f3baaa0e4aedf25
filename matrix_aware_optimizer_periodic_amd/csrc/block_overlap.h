// Whether strided tensors have a value in one place, exactly, so that a call can
// refuse outputs that another workgroup still reads while slices of one packed
// buffer, whose addresses interleave, pass.  Host only.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace muon {

// Values ptr + sum_i x_i stride_i, 0 <= x_i < count_i (strides of 0 or more).
struct Places {
  const void* ptr;
  int64_t stride[4], count[4];
};

// step x, low <= x <= high, step above 0.
struct PlaceTerm {
  __int128 step, low, high;
};

// Whether x_i exist with sum_i step_i x_i = target, the largest step first: only
// an x that leaves no more than the others can make up is followed, one or two
// for each step of dimensions that lie within each other.  Layouts that take more
// than `turns` of them count as meeting.
inline bool reaches(const PlaceTerm* t, int n, __int128 target, int& turns) {
  if (n == 0) return target == 0;
  __int128 low = 0, high = 0;
  for (int i = 1; i < n; ++i) {
    low += t[i].step * t[i].low;
    high += t[i].step * t[i].high;
  }
  auto down = [](__int128 a, __int128 b) { return a / b - (a % b != 0 && a < 0 ? 1 : 0); };
  const __int128 first = std::max(t[0].low, -down(high - target, t[0].step)), last = std::min(t[0].high, down(target - low, t[0].step));
  for (__int128 x = first; x <= last; ++x) {
    if (--turns < 0) return true;
    if (reaches(t + 1, n - 1, target - t[0].step * x, turns)) return true;
  }
  return false;
}

constexpr int kPlaceTurns = 4096;

inline int sort_terms(PlaceTerm* t, int n) {
  std::sort(t, t + n, [](const PlaceTerm& a, const PlaceTerm& b) { return a.step > b.step; });
  return n;
}

// From the first value to the last, in values.
inline __int128 span_of(const Places& p) {
  __int128 s = 0;
  for (int i = 0; i < 4; ++i) s += __int128(p.stride[i]) * (p.count[i] - 1);
  return s;
}

// Whether a and b share a value of `size` bytes (both pointers multiples of it).
inline bool places_meet(const Places& a, const Places& b, int64_t size) {
  for (int i = 0; i < 4; ++i)
    if (a.count[i] < 1 || b.count[i] < 1) return false;
  // (the usual case: all that a call compares takes 0.08 us, where what follows took 0.5)
  const __int128 apart = __int128(reinterpret_cast<uintptr_t>(b.ptr)) - __int128(reinterpret_cast<uintptr_t>(a.ptr));
  if (apart > span_of(a) * size || -apart > span_of(b) * size) return false;
  PlaceTerm t[8];
  int n = 0;
  auto add = [&](int64_t stride, int64_t low, int64_t high) {
    if (stride == 0 || (low == 0 && high == 0)) return;
    for (int i = 0; i < n; ++i)
      if (t[i].step == stride) {
        t[i].low += low;
        t[i].high += high;
        return;
      }
    t[n++] = PlaceTerm{stride, low, high};
  };
  for (int i = 0; i < 4; ++i) {
    add(a.stride[i], 0, a.count[i] - 1);
    add(b.stride[i], 1 - b.count[i], 0);
  }
  int turns = kPlaceTurns;
  return reaches(t, sort_terms(t, n), apart / size, turns);
}

// Whether two values of a are in one place.
inline bool places_repeat(const Places& a) {
  for (int64_t count : a.count)
    if (count < 1) return false;
  // Every step past all that the next ones reach: the usual case.
  __int128 below = 0;
  bool nested = true;
  for (int i = 3; i >= 0; --i) {
    if (a.count[i] == 1) continue;
    nested = nested && a.stride[i] > below;
    below += __int128(a.stride[i]) * (a.count[i] - 1);
  }
  if (nested) return false;
  PlaceTerm t[4];
  int n = 0;
  for (int i = 0; i < 4; ++i) {
    if (a.count[i] == 1) continue;
    if (a.stride[i] == 0) return true;
    t[n++] = PlaceTerm{a.stride[i], 1 - a.count[i], a.count[i] - 1};
  }
  sort_terms(t, n);
  // two values differ first in dimension i, by x of 1 or more there
  int turns = kPlaceTurns;
  for (int i = 0; i < n; ++i) {
    PlaceTerm from = t[i];
    from.low = 1;
    std::swap(t[i], from);
    if (reaches(t + i, n - i, 0, turns)) return true;
    std::swap(t[i], from);
  }
  return false;
}

// Whether a and b are the same values, each in its place (the stride of a
// dimension of one says nothing).
inline bool same_places(const Places& a, const Places& b) {
  if (a.ptr != b.ptr) return false;
  for (int i = 0; i < 4; ++i)
    if (a.count[i] != b.count[i] || (a.count[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return true;
}

}  // namespace muon
