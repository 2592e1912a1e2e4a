// vr_places.h -- whether two strided arguments share a byte (host).
//
// An argument is rows of `width` bytes at `at` + sum of i_k stride_k, 0 <= i_k < n_k. Two rows of
// a and b, D bytes apart, share one where -a.width < D < b.width; D is the difference of the
// addresses and a multiple d_k of each axis's stride, where -(b.n_k - 1) <= d_k <= a.n_k - 1. From
// the largest stride on only those multiples are tried from which the smaller ones can still get
// there: one or two, where each axis steps over the ones inside. Of axes that run into one
// another there are more, and the arguments count as sharing.
#pragma once

#include <stdint.h>

namespace vrop {

struct Places {
  static constexpr int kAxes = 3;
  uintptr_t at = 0, end = 0;
  int64_t width = 0;  // 0: nothing
  int axes = 0;
  int64_t n[kAxes], stride[kAxes];

  Places() = default;
  Places(const void* p, uint64_t bytes) : at((uintptr_t)p), end(at + bytes), width(p ? (int64_t)bytes : 0) {}
  // Of one element, or without a step, it adds nothing.
  void axis(uint64_t count, uint64_t step) {
    if (count <= 1 || !step) return;
    n[axes] = (int64_t)count, stride[axes++] = (int64_t)step;
    end += (count - 1) * step;
  }
};

struct PlaceSteps {
  int axes = 0;
  int64_t stride[2 * Places::kAxes], least[2 * Places::kAxes], most[2 * Places::kAxes];
  int64_t low[2 * Places::kAxes + 1], high[2 * Places::kAxes + 1];  // the sums of the axes from one on

  // Whether a sum of the axes from k on brings `at` into [from, to].
  bool reach(int k, int64_t at, int64_t from, int64_t to) const {
    if (at + high[k] < from || at + low[k] > to) return false;
    if (k == axes) return true;
    const int64_t s = stride[k], a = from - at - high[k + 1], b = to - at - low[k + 1];
    int64_t first = a / s + (a % s > 0), last = b / s - (b % s < 0);
    if (first < least[k]) first = least[k];
    if (last > most[k]) last = most[k];
    if (last - first >= 4) return true;
    for (int64_t d = first; d <= last; ++d)
      if (reach(k + 1, at + d * s, from, to)) return true;
    return false;
  }
};

inline bool overlap(const Places& a, const Places& b) {
  if (!a.width || !b.width || a.at >= b.end || b.at >= a.end) return false;
  PlaceSteps s;
  for (int side = 0; side < 2; ++side) {
    const Places& p = side ? b : a;
    for (int i = 0; i < p.axes; ++i) {
      int k = 0;  // axes of one stride are one, larger strides first
      while (k < s.axes && s.stride[k] > p.stride[i]) ++k;
      if (k == s.axes || s.stride[k] != p.stride[i]) {
        for (int j = s.axes++; j > k; --j) s.stride[j] = s.stride[j - 1], s.least[j] = s.least[j - 1], s.most[j] = s.most[j - 1];
        s.stride[k] = p.stride[i];
        s.least[k] = s.most[k] = 0;
      }
      if (side) s.least[k] -= p.n[i] - 1;
      else s.most[k] += p.n[i] - 1;
    }
  }
  s.low[s.axes] = s.high[s.axes] = 0;
  for (int k = s.axes - 1; k >= 0; --k) {
    s.low[k] = s.low[k + 1] + s.least[k] * s.stride[k];
    s.high[k] = s.high[k + 1] + s.most[k] * s.stride[k];
  }
  return s.reach(0, (int64_t)(a.at - b.at), 1 - a.width, b.width - 1);
}

// Whether one of the outputs shares a byte with an input or another output.
inline bool anyOverlap(const Places* outs, int nOuts, const Places* ins, int nIns) {
  for (int i = 0; i < nOuts; ++i) {
    for (int j = 0; j < nIns; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

}  // namespace vrop
