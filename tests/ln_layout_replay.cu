// ln_layout_replay.cu -- replays the layouts of the layer norm kernels (the plans
// and the places of threads that the kernels use, from vr_ln_plan.cuh and
// vr_ln_rows.cuh) on the host for random sizes, strides and addresses, and checks:
//  * every row belongs to one group, and the threads of a warp that share shuffles,
//    or of a group that share barriers, go as many rounds;
//  * every column of a row is one thread's, whole packs lie inside the row and on
//    16-byte boundaries, in the first and the last row of a group;
//  * blocks, registers, named barriers, the buffers of the rows' sums, the rows' ring
//    and the joining of a block's sums stay inside what is launched;
//  * the workspace holds the sums that a backward pass leaves, whatever number of
//    clusters the GPU takes at a time.
// Exit status 0 when every check holds; prints the first failure otherwise.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "vr_ln_plan.cuh"

using namespace vrln;

namespace {

uint64_t state = 0x9E3779B97F4A7C15ull;
uint64_t next() {  // splitmix64
  uint64_t z = (state += 0x9E3779B97F4A7C15ull);
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}
uint64_t pick(uint64_t lo, uint64_t hi) { return lo + next() % (hi - lo + 1); }

struct Case {
  uint64_t rows, cols, stride, base;
  bool ragged;
  int es;
};

#define CHECK(what)                                                                            \
  if (!(what)) {                                                                               \
    fprintf(stderr, "%s\n  rows %llu cols %llu stride %llu base %llu size %d: %d threads of a row, " \
            "%d groups, %d blocks, step %u, grid %u\n", #what, (unsigned long long)c.rows,       \
            (unsigned long long)c.cols, (unsigned long long)c.stride, (unsigned long long)c.base, \
            c.es, l.tpr, l.groups, l.ctas, l.step, grid);                                       \
    exit(1);                                                                                   \
  }

// One launch of `grid` blocks: SUMS values of a row are added up at a time.
template <typename T, int E, int MODE>
void places(const Case& c, const Layout& l, unsigned grid, int regs, int sums, bool together) {
  constexpr int V = kV<T>, P = E / V;
  const int threads = l.tpr * l.groups, warps = threads / 32, cols = (int)c.cols;
  CHECK(threads % 32 == 0 && threads <= 1024 && threads * regs <= 65536);
  CHECK(grid >= 1 && grid % l.ctas == 0 && l.ctas <= 8 && (!together || grid <= 16));
  CHECK(MODE != IN_BLOCK || (l.groups <= 15 && l.tpr % 32 == 0 && warps <= kMaxWarps));
  CHECK(MODE != IN_WARP || (32 % l.tpr == 0 && l.tpr >= sums));
  CHECK(MODE != IN_CLUSTER || (l.groups == 1 && l.tpr / 32 * l.ctas <= 8 * 16 && l.ctas * sums <= 32));
  CHECK(!c.ragged || grid / l.ctas * l.groups >= c.rows || l.step * c.stride * c.es % 16 == 0);
  std::vector<uint8_t> seen(c.rows, 0);
  const unsigned check0 = (unsigned)pick(0, grid / l.ctas - 1);
  for (unsigned b = 0; b < grid / l.ctas; ++b) {
    for (int g = 0; g < l.groups; ++g) {
      const Place<T, MODE, P> at(l, c.rows, cols, b * l.ctas, g * l.tpr, 0);
      CHECK(at.group == g && at.rounds >= at.n);
      for (int i = 0; i < at.n; ++i) {
        const uint64_t row = at.row + (uint64_t)i * l.step;
        CHECK(row < c.rows && !seen[row]);
        seen[row] = 1;
      }
      if (b != check0 && b != 0 && b != grid / l.ctas - 1) continue;
      if (!at.n) continue;
      // the columns of this group's rows, and the rounds of its threads
      std::vector<uint8_t> owned(cols, 0);
      for (int rank = 0; rank < l.ctas; ++rank)
        for (int t = 0; t < l.tpr; ++t) {
          const int thread = g * l.tpr + t;
          const Place<T, MODE, P> me(l, c.rows, cols, b * l.ctas + rank, thread, rank);
          const Place<T, MODE, P> lead(l, c.rows, cols, b * l.ctas + rank, thread & ~31, rank);
          CHECK(me.row == at.row && me.n == at.n && me.rounds == lead.rounds);
          CHECK(MODE == IN_WARP || me.rounds == at.n);
          for (int i = 0; i < P; ++i) {
            if (!me.used(i)) continue;
            const int col = me.column(i);
            CHECK(col >= 0 && col + V <= cols);
            CHECK(col == me.column(0) + i * (MODE == IN_WARP ? me.stripe : 32) * V);
            for (int k = 0; k < V; ++k) ++owned[col + k];
            const uint64_t last = me.row + (uint64_t)(me.n - 1) * l.step;
            CHECK((c.base + (me.row * c.stride + col) * c.es) % 16 == 0);
            CHECK((c.base + (last * c.stride + col) * c.es) % 16 == 0);
          }
          if (me.edge >= 0) {
            CHECK(c.ragged && me.edge < cols);
            ++owned[me.edge];
          }
        }
      for (int i = 0; i < cols; ++i) CHECK(owned[i] == 1);
    }
  }
  for (uint64_t i = 0; i < c.rows; ++i) CHECK(seen[i]);
}

template <typename T, int E>
void launchOf(const Case& c, int mode, Layout l, unsigned grid, int regs, int sums, bool together = false) {
  l.offset = (int)(c.base & 15);
  l.skew = (int)((c.stride * c.es) & 15);
  if (mode == IN_WARP) places<T, E, IN_WARP>(c, l, grid, regs, sums, together);
  if (mode == IN_BLOCK) places<T, E, IN_BLOCK>(c, l, grid, regs, sums, together);
  if (mode == IN_CLUSTER) places<T, E, IN_CLUSTER>(c, l, grid, regs, sums, together);
}

int nForward = 0, nBackward = 0, nTogether = 0, nPlain = 0;

template <typename T, int E, int ROWS, int STAGES, int REGS>
void forward(const Case& c, int blockThreads, int maxThreads) {
  constexpr int V = kV<T>;
  Layout l;
  int mode;
  unsigned grid = 0;
  if (!layoutFor(c.cols, V, E / V, blockThreads, maxThreads, c.ragged, &l, &mode)) return;
  const int threads = l.tpr * l.groups;
  const size_t smem = (size_t)STAGES * ROWS * E * sizeof(T) * threads;
  CHECK(smem <= kMostShared);
  uint64_t most = mostAtOnce(l, residentWarps(REGS, smem, threads));
  CHECK(most >= 1);
  if (mode == IN_CLUSTER) most = pick(1, most);
  grid = gridFor(c.rows, &l, V, most, c.ragged, ROWS);
  launchOf<T, E>(c, mode, l, grid, REGS, ROWS);
  ++nForward;
}

template <typename T, int E, int ROWS, int STAGES>
void backward(const Case& c, BwdPlan p, int regs) {
  const Layout& l = p.l;
  unsigned grid = p.grid;
  const uint64_t held = mostSplits<T>(c.rows, c.cols);
  const size_t ring = (size_t)(p.threads / 32) * STAGES * ROWS * 2 * (E / kV<T>) * 32 * 16;
  CHECK(p.threads == l.tpr * l.groups && ring <= p.smem && p.smem <= kMostShared && p.rowsAtOnce == ROWS);
  if (p.mode == IN_CLUSTER) {
    grid = p.grid = gridFor(c.rows, &p.l, kV<T>, pick(1, p.most), c.ragged, ROWS);
  } else {
    // a group's sums of dw, then of db, every eighth word left out; group after group
    auto slot = [](uint64_t col) { return col + (col >> 3); };
    const uint64_t half = slot(c.cols + 7);
    CHECK(slot(c.cols - 1) < half);
    CHECK(((l.groups - 1) * 2 * half + half + slot(c.cols - 1) + 1) * sizeof(float) <= p.smem);
  }
  CHECK(grid / l.ctas <= held);
  launchOf<T, E>(c, p.mode, p.l, grid, regs, 2 * ROWS);
  ++nBackward;
  if (planTogether<T>(c.rows, c.cols, c.ragged, &p)) {
    launchOf<T, E>(c, p.mode, p.l, p.grid, regs, 2 * ROWS, true);
    ++nTogether;
  }
}

template <typename T>
void all(Case c) {
  // the forward pass's shapes
  forward<T, 16, 2, 2, 128>(c, 256, 512);
  forward<T, 16, 2, 2, 128>(c, 256, 256);
  forward<T, 16, 2, 2, 128>(c, 256, 64);
  forward<T, 32, 2, 2, 168>(c, 128, 384);
  forward<T, 32, 1, 3, 128>(c, 256, 512);
  if (sizeof(T) == 2) forward<T, 16, 4, 2, 168>(c, 128, 128);
  BwdPlan p;
  const int shape = planBackward<T>(c.rows, c.cols, c.ragged, &p);
  if (shape == WIDE) backward<T, 32, kWideRows<T>, 2>(c, p, 168);
  else if (shape == ONE_WARP) backward<T, 32, 2, 2>(c, p, 168);
  else if (shape == ONE_ROW) backward<T, 16, 1, 3>(c, p, 128);
  else if (shape == TWO_ROWS) backward<T, 16, 2, 2>(c, p, 128);
  else ++nPlain;
  const Layout l = {};
  const unsigned grid = 0;
  CHECK((uint64_t)splitsFor(c.rows, c.cols) <= mostSplits<T>(c.rows, c.cols));
}

}  // namespace

int main(int argc, char** argv) {
  const int trials = argc > 1 ? atoi(argv[1]) : 500;
  const uint64_t borders[] = {4,    8,    9,    63,   64,   65,    72,    128,   256,   264,   511,  512,
                              513,  640,  768,  776,  960,  961,   1016,  1024,  1025,  2047,  2055, 2056,
                              2064, 4088, 4095, 4096, 4103, 4104,  8184,  8191,  8192,  8199,  8200, 8201,
                              8208, 9000, 12288, 12289, 16376, 16384, 16385, 16391, 24576, 24584, 32769,
                              49152, 49160, 65536, 65537, 98304, 98312};
  for (int t = 0; t < trials; ++t) {
    Case c;
    c.es = t % 2 ? 4 : 2;
    const uint64_t wide = pick(0, 9);
    c.cols = wide < 3 ? borders[pick(0, sizeof(borders) / 8 - 1)] + pick(0, 2) : wide < 6 ? pick(1, 300)
             : wide < 9 ? pick(1, 9000) : pick(9000, 140000);
    const uint64_t tall = pick(0, 3);
    c.rows = tall == 0 ? pick(1, 40) : tall == 1 ? pick(1, 700) : pick(1, c.cols > 10000 ? 2000 : 20000);
    c.stride = c.cols + (pick(0, 1) ? 0 : pick(0, 1) ? 16 * pick(0, 3) / c.es : pick(0, 40));
    c.base = 4096 + (pick(0, 1) ? 0 : pick(0, 16 / c.es - 1) * c.es);
    const int V = 16 / c.es;
    c.ragged = c.base % 16 || c.stride * c.es % 16 || c.cols % V;
    if (c.es == 2) all<__half>(c);
    else all<float>(c);
  }
  if (trials >= 500 && (!nForward || !nBackward || !nTogether || !nPlain)) {
    fprintf(stderr, "a kind of launch was not reached\n");
    return 1;
  }
  printf("ok: %d forward, %d backward, %d of them one cluster's, %d plain\n", nForward, nBackward, nTogether,
         nPlain);
  return 0;
}
