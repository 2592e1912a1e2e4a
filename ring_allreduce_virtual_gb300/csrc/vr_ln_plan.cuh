// vr_ln_plan.cuh -- how a layer norm backward pass is laid out: which kernel, what
// grid and shared memory, and how many sums of dw and db it leaves (host).
#pragma once

#include "vr_ln_rows.cuh"

namespace vrln {

// Splits of the rows where dw and db are summed in a kernel of their own.
inline int splitsFor(uint64_t rows, uint64_t cols) {
  const uint64_t tiles = (cols + 31) / 32;
  uint64_t s = (uint64_t)kSMs * 8 / tiles + 1;
  const uint64_t most = (rows + 63) / 64;
  s = s < most ? s : most;
  return s ? (int)s : 1;
}

// Two matrices whose rows lie alike modulo 16 bytes.
inline bool alike(const void* p, uint64_t pStride, const void* q, uint64_t qStride, int es) {
  return (((uintptr_t)p - (uintptr_t)q) & 15) == 0 && (((pStride - qStride) * es) & 15) == 0;
}

// How a backward pass is laid out, and the sums of dw and db that it leaves.
// The shapes were chosen by measuring on a GB300 (dy and x read and dx written
// once, of the measured copy peak). 16 elements of 2 rows a thread, the blocks
// as large as one for each SM can be, leave the fewest sums to join (8192 bf16
// 0.95, 4096 bf16 0.93, 1024 bf16 0.90). Whole packs of 257 to 768 16-bit
// elements are one warp's at 32 elements a lane, which saves the barriers (768
// 0.84 against 0.78, 640 0.71 against 0.65; 896 0.84 against 0.87). float32 rows
// take 256 threads of the first (4096 0.95), as the ring of 512 would not fit, and
// beyond 4096 one row at a time (8192 0.92 against 0.84 with two in clusters). Rows
// too wide for that are 384 threads' with 32 elements of each row, up to 12288
// (12288 bf16 0.87 against 0.55 in clusters, 10240 float32 0.87 against 0.60).
// Then they are clusters', which wait for their slowest block at every row: of
// these blocks where they are fewer than of the first kinds (24576 bf16 0.75
// against 0.57, 49152 0.70 against 0.48, float32 0.88 and 0.84 against 0.64 and
// 0.53), else of those (16384 bf16 0.72, float32 0.80; 32768 bf16 0.66, 65536 0.53).
struct BwdPlan {
  Layout l;
  int mode, threads, rowsAtOnce;
  uint64_t most;
  unsigned grid;
  size_t smem;
};
template <typename T, int E, int ROWS, int STAGES, int REGS>
bool planShape(uint64_t rows, uint64_t cols, bool ragged, int blockThreads, int maxThreads,
               BwdPlan* p) {
  constexpr int V = kV<T>;
  if (!layoutFor(cols, V, E / V, blockThreads, maxThreads, ragged, &p->l, &p->mode)) return false;
  p->threads = p->l.tpr * p->l.groups;
  const size_t ring = (size_t)STAGES * ROWS * E * sizeof(T) * 2 * p->threads;
  // The groups' sums take the ring's place at the end, of every column.
  const size_t join = p->mode == IN_CLUSTER
                          ? 0
                          : (size_t)p->l.groups * 2 * ((cols + 7) * 9 / 8 + 1) * sizeof(float);
  p->smem = ring > join ? ring : join;
  p->rowsAtOnce = ROWS;
  p->most = mostAtOnce(p->l, residentWarps(REGS, p->smem, p->threads));
  p->grid = gridFor(rows, &p->l, V, p->most, ragged, ROWS);
  return p->smem <= kMostShared;
}
constexpr unsigned kTogether = 16;
enum { NO_PLAN = 0, TWO_ROWS = 1, ONE_ROW = 2, WIDE = 3, ONE_WARP = 4 };
template <typename T>
constexpr int kWideRows = sizeof(T) == 2 ? 2 : 1;
template <typename T>
int planBackward(uint64_t rows, uint64_t cols, bool ragged, BwdPlan* p) {
  if (rows >= kMostRows) return NO_PLAN;
  if (cols > 8192 + 8 &&
      planShape<T, 32, kWideRows<T>, 2, 168>(rows, cols, ragged, 384, 384, p)) {
    const int ctas = p->l.ctas;
    Layout l;  // of the shapes below
    int mode;
    if (ctas == 1 || !layoutFor(cols, kV<T>, 16 / kV<T>, 512, 512, ragged, &l, &mode) || ctas < l.ctas)
      return WIDE;
  }
  if constexpr (sizeof(T) == 2) {
    if (!ragged && cols > 256 && cols <= 768 &&
        planShape<T, 32, 2, 2, 168>(rows, cols, ragged, 384, 32, p))
      return ONE_WARP;
    return planShape<T, 16, 2, 2, 128>(rows, cols, ragged, 512, 512, p) ? TWO_ROWS : NO_PLAN;
  }
  if (cols > 4096 && planShape<T, 16, 1, 3, 128>(rows, cols, ragged, 512, 512, p)) return ONE_ROW;
  return planShape<T, 16, 2, 2, 128>(rows, cols, ragged, 256, 256, p) ? TWO_ROWS : NO_PLAN;
}

// Small calls: one cluster, each group of it up to 8 rows, and nothing left to
// join. The launch that it saves is 3 us of the host's time, against up to 2
// on the GPU (64 x 64 float32 3.7 us against 4.5, 256 x 1024 bf16 6.6 against
// 6.4, 200 x 1280 float32 9.5 against 7.4; 1000 x 1024 bf16 12.2 against 6.9).
template <typename T>
bool planTogether(uint64_t rows, uint64_t cols, bool ragged, BwdPlan* p) {
  const uint64_t groups = (uint64_t)p->l.groups;
  if (p->mode == IN_CLUSTER || rows > groups * kTogether * 8 || rows * cols > 1u << 18) return false;
  unsigned blocks = 1;
  while (blocks < kTogether && blocks * groups * 2 < rows) blocks *= 2;
  if (ragged && blocks * groups % kV<T>) blocks = kTogether;
  p->grid = blocks;
  p->l.step = (uint32_t)(blocks * groups);
  return true;
}

// The most sums that any layout of these sizes leaves.
template <typename T>
uint64_t mostSplits(uint64_t rows, uint64_t cols) {
  uint64_t most = splitsFor(rows, cols);
  for (const bool ragged : {false, true}) {
    BwdPlan p;
    if (rows && planBackward<T>(rows, cols, ragged, &p) != NO_PLAN && p.grid / p.l.ctas > most)
      most = p.grid / p.l.ctas;
  }
  return most;
}

}  // namespace vrln
