// places_replay.cc -- overlaps of strided arguments against sets of bytes, on random small ones.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>
#include <random>
#include <vector>

#include "vr_places.h"

using vrop::Places;

constexpr int kSpace = 4096;

static std::vector<char> bytesOf(const Places& p) {
  std::vector<char> set(kSpace, 0);
  int64_t n[3] = {1, 1, 1}, s[3] = {0, 0, 0};
  for (int i = 0; i < p.axes; ++i) n[i] = p.n[i], s[i] = p.stride[i];
  for (int64_t i = 0; i < n[0]; ++i)
    for (int64_t j = 0; j < n[1]; ++j)
      for (int64_t k = 0; k < n[2]; ++k)
        for (int64_t b = 0; b < p.width; ++b) set.at(p.at + i * s[0] + j * s[1] + k * s[2] + b) = 1;
  return set;
}

// Whether each axis steps over the ones inside.
static bool nested(const Places& p) {
  std::vector<std::pair<int64_t, int64_t>> axes;
  for (int i = 0; i < p.axes; ++i) axes.push_back({p.stride[i], p.n[i]});
  std::sort(axes.begin(), axes.end());
  int64_t inner = p.width;
  for (auto& a : axes) {
    if (a.first < inner) return false;
    inner += (a.second - 1) * a.first;
  }
  return true;
}

int main(int argc, char** argv) {
  std::mt19937 rng(7);
  const auto in = [&](int low, int high) { return low + (int)(rng() % (unsigned)(high - low + 1)); };
  const int rounds = argc > 1 ? atoi(argv[1]) : 200000;
  int shared = 0, apart = 0, inside = 0, careful = 0;
  for (int round = 0; round < rounds; ++round) {
    // batches of tokens of heads, one kind next to the other, some tokens left out, in any order
    const int width = in(1, 4), gap = in(0, 1) ? 0 : in(0, 4), heads = in(1, 3), tokens = in(1, 4);
    int64_t stride[3];  // of heads, tokens, batches
    stride[0] = width + gap;
    stride[1] = stride[0] * (heads * 2 + in(0, 2)) + in(0, 2);
    stride[2] = stride[1] * (tokens + in(0, 1)) + in(0, 3);
    const bool same = in(0, 3) != 0;
    Places p[2];
    for (int side = 0; side < 2; ++side) {
      int64_t st[3] = {stride[0], stride[1], stride[2]};
      if (side && !same)
        for (auto& x : st) x = in(0, 40);
      p[side] = Places((const void*)(uintptr_t)in(1, 160), in(0, 20) ? (side ? in(1, width + gap) : width) : 0);
      p[side].axis(in(1, 3), st[2]);
      p[side].axis(in(0, 3) ? tokens : 1, st[1]);
      p[side].axis(in(1, heads), st[0]);
    }
    const std::vector<char> a = bytesOf(p[0]), b = bytesOf(p[1]);
    bool truth = false;
    for (int i = 0; i < kSpace; ++i) truth = truth || (a[i] && b[i]);
    const bool said = overlap(p[0], p[1]);
    if (said != overlap(p[1], p[0]) || (truth && !said) || (!truth && said && same && nested(p[0]) && nested(p[1]))) {
      fprintf(stderr, "round %d: said %d, is %d\n", round, said, truth);
      return 1;
    }
    shared += truth;
    apart += !truth;
    careful += said && !truth;
    const auto span = [](const std::vector<char>& s) {
      const auto first = std::find(s.begin(), s.end(), 1);
      const auto last = std::find(s.rbegin(), s.rend(), 1);
      return std::make_pair((int)(first - s.begin()), kSpace - (int)(last - s.rbegin()));
    };
    const auto x = span(a), y = span(b);
    inside += !said && x.first < y.second && y.first < x.second;
  }
  // far apart in their steps: sums of more than 32 bits
  const uint64_t far = 1ull << 40;
  for (int64_t d = -5; d <= 5; ++d) {
    Places a((const void*)(far + 64), 4), b((const void*)(far + 64 + 3 * far + 2 * (1 << 20) + d), 3);
    a.axis(4, far), a.axis(3, 1 << 20);
    if (overlap(a, b) != (d > -3 && d < 4)) return fprintf(stderr, "far %d\n", (int)d), 1;
  }
  printf("ok: %d share, %d do not, %d of them within one another's span, %d refused all the same\n", shared, apart, inside,
         careful);
  return 0;
}
