// vr_layernorm.cu -- layer norm over the last axis, forward and backward.
//
//   m = sum(x) / C, v = sum((x - m)^2) / C, r = 1 / sqrt(v + eps)
//   y = (x - m) r w + b
//   u = (x - m) r, g = dy w
//   dx = r (g - sum(g) / C - u sum(g u) / C)
//   dw = sum over rows of dy u,  db = sum over rows of dy
//
// Everything is computed in 32 bits and rounded once to the tensors' type; the
// variance is the mean of squared distances from the mean, never a difference
// of two large sums. All of it is bound by memory traffic (8 to 14 flop for 4
// to 12 bytes).
#include "vr_ln_plan.cuh"

namespace {

using namespace vrop;
using namespace vrln;

struct FwdArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  uint64_t rows, cols, xStride, yStride;
  float eps;
  Layout l;
};

struct BwdArgs {
  const void* dy;
  const void* x;
  const void* w;
  const float* mean;
  const float* rstd;
  void* dx;
  void* dw;
  void* db;
  uint64_t rows, cols, dyStride, xStride, dxStride;
  float* partials;  // [splits][2][cols]: sums of dy u and of dy over a split's rows
  int splits;
  bool together;  // the grid is one cluster, which joins its sums itself
  Layout l;
};

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// Rows of any width, stride and alignment: a block for each row, three walks
// over it.
template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) vrLnForwardAny(const __grid_constant__ FwdArgs a) {
  __shared__ float buf[2][kRowWarps];
  begin_kernel();
  const W* w = static_cast<const W*>(a.w);
  const W* b = static_cast<const W*>(a.b);
  const float c = 1.f / (float)a.cols;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.xStride;
    T* y = static_cast<T*>(a.y) + row * a.yStride;
    float s = 0.f, q = 0.f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kRowThreads) s += to_f32(x[i]);
    const float m = block_sum<kRowWarps>(s, buf[0]) * c;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
      const float d = to_f32(x[i]) - m;
      q = fmaf(d, d, q);
    }
    const float r = rsqrtf(block_sum<kRowWarps>(q, buf[1]) * c + a.eps);
    for (uint64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
      float u = (to_f32(x[i]) - m) * r;
      if (w) u *= to_f32(w[i]);
      if (b) u += to_f32(b[i]);
      y[i] = from_f32<T>(u);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
    }
  }
}

// ROWS rows of a group in registers, E elements of each in a thread, and STAGES -
// 1 times as many on their way: read once, written once.
template <typename T, typename W, int E, int ROWS, int STAGES, int MODE, bool RAGGED, int REGS>
__global__ void __maxnreg__(REGS) vrLnForwardRows(const __grid_constant__ FwdArgs a) {
  constexpr int V = kV<T>, P = E / V;
  extern __shared__ uint4 ring[];  // [warps][STAGES][ROWS][P][32]
  __shared__ RowSum<MODE, ROWS> sum;
  begin_kernel();
  const int cols = (int)a.cols;
  const Place<T, MODE, P> at(a.l, a.rows, cols);
  int turn = 0;
  if constexpr (MODE == IN_CLUSTER) cluster_sync();  // the others' buffers are there
  const T* xp = static_cast<const T*>(a.x) + at.row * a.xStride;
  T* yp = static_cast<T*>(a.y) + at.row * a.yStride;
  const uint64_t xStep = a.l.step * a.xStride, yStep = a.l.step * a.yStride;
  bool used[P];
#pragma unroll
  for (int i = 0; i < P; ++i) used[i] = at.used(i);
  uint4* const mine = ring + (threadIdx.x >> 5) * (STAGES * ROWS * P * 32) + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (!used[i])
      for (int k = 0; k < STAGES * ROWS; ++k) mine[(k * P + i) * 32] = make_uint4(0, 0, 0, 0);
  T ahead[ROWS];  // the next rows' elements outside the packs
  const uint32_t ringAt = (uint32_t)__cvta_generic_to_shared(mine);
  auto fetch = [&](int left, const T* p, int stage) {
    const uint32_t to = ringAt + stage * (ROWS * P * 512);
    each<ROWS>([&](auto kk) {
      constexpr int k = decltype(kk)::value;
      if (k < left) {
        const T* q = p + k * xStep;
        each<P>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          if (!used[i]) return;
          if constexpr (MODE == IN_WARP) copy16<(k * P + i) * 512, 0>(to, q + i * at.stripe * V);
          else copy16<(k * P + i) * 512, i * 512>(to, q);
        });
      }
    });
    copies_commit();
  };
  // Only the first warps of a row hold elements outside the packs.
  const bool edges = RAGGED && __any_sync(~0u, at.edge >= 0);
  auto fetchEdge = [&](int left, const T* p) {
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        ahead[k] = at.edge >= 0 && k < left ? p[k * xStep + at.edge] : from_f32<T>(0.f);
    }
  };
  const T* xf = xp + at.column(0);  // the rows to fetch next
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    fetch(at.n - i * ROWS, xf, i);
    xf += ROWS * xStep;
  }
  fetchEdge(at.n, xp);
  Params<T, W> w[P], b[P];
  float we = 1.f, be = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    w[i].load(static_cast<const W*>(a.w), at.column(i), used[i], 1.f);
    b[i].load(static_cast<const W*>(a.b), at.column(i), used[i], 0.f);
  }
  if (RAGGED && at.edge >= 0) {
    if (a.w) we = to_f32(static_cast<const W*>(a.w)[at.edge]);
    if (a.b) be = to_f32(static_cast<const W*>(a.b)[at.edge]);
  }
  const float c = 1.f / (float)cols;
  uint64_t row = at.row;
  int left = at.n, stage = 0;
  T* yo = yp + at.column(0);
  for (int round = 0; round < at.rounds; round += ROWS) {
    const int back = stage == 0 ? STAGES - 1 : stage - 1;
    fetch(left - (STAGES - 1) * ROWS, xf, back);
    xf += ROWS * xStep;
    copies_wait<STAGES - 1>();
    F2 x[ROWS][P][V / 2];
    float e[ROWS], s[ROWS];
    const uint4* from = mine + stage * (ROWS * P * 32);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      F2 s2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        unpack<T>(from[(k * P + i) * 32], x[k][i]);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) s2 = s2 + x[k][i][j];
      }
      s[k] = both(s2);
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        e[k] = to_f32(ahead[k]);
        s[k] += e[k];
      }
    }
    xp += ROWS * xStep;
    fetchEdge(left - ROWS, xp);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    sum(s, a.l, at.group, turn);
    float m[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      m[k] = s[k] * c;
      const F2 minus = f2(-m[k]);
      F2 q2 = f2(0.f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) x[k][i][j] = x[k][i][j] + minus;
        if (used[i]) {
#pragma unroll
          for (int j = 0; j < V / 2; ++j) q2 = fma2(x[k][i][j], x[k][i][j], q2);
        }
      }
      s[k] = both(q2);
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        e[k] -= m[k];
        if (at.edge >= 0) s[k] = fmaf(e[k], e[k], s[k]);
      }
    }
    sum(s, a.l, at.group, turn);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      s[k] = rsqrtf(s[k] * c + a.eps);
      const F2 r2 = f2(s[k]);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        F2 g[V / 2], h[V / 2];
        w[i].get(g);
        b[i].get(h);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) x[k][i][j] = fma2(x[k][i][j] * r2, g[j], h[j]);
        if (used[i] && k < left)
          *reinterpret_cast<uint4*>(yo + k * yStep + i * (MODE == IN_WARP ? at.stripe : 32) * V) =
              pack<T>(x[k][i]);
      }
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (at.edge >= 0 && k < left)
          yp[k * yStep + at.edge] = from_f32<T>(fmaf(e[k] * s[k], we, be));
    }
    if (at.lane == 0) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (k < left) {
          if (a.mean) a.mean[row + (uint64_t)k * a.l.step] = m[k];
          if (a.rstd) a.rstd[row + (uint64_t)k * a.l.step] = s[k];
        }
    }
    left -= ROWS;
    row += (uint64_t)ROWS * a.l.step;
    yp += ROWS * yStep;
    yo += ROWS * yStep;
  }
}

// dx of rows of any width: a block for each row, two walks over it.
template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) vrLnBackwardAny(const __grid_constant__ BwdArgs a) {
  __shared__ float buf[4][kRowWarps];
  begin_kernel();
  const W* w = static_cast<const W*>(a.w);
  const float c = 1.f / (float)a.cols;
  int turn = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* dy = static_cast<const T*>(a.dy) + row * a.dyStride;
    const T* x = static_cast<const T*>(a.x) + row * a.xStride;
    T* dx = static_cast<T*>(a.dx) + row * a.dxStride;
    const float m = a.mean[row], r = a.rstd[row];
    float s = 0.f, p = 0.f;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
      float g = to_f32(dy[i]);
      if (w) g *= to_f32(w[i]);
      s += g;
      p = fmaf(g, (to_f32(x[i]) - m) * r, p);
    }
    s = block_sum<kRowWarps>(s, buf[turn]) * c;
    p = block_sum<kRowWarps>(p, buf[turn + 1]) * c;
    turn ^= 2;
    for (uint64_t i = threadIdx.x; i < a.cols; i += kRowThreads) {
      float g = to_f32(dy[i]);
      if (w) g *= to_f32(w[i]);
      const float u = (to_f32(x[i]) - m) * r;
      dx[i] = from_f32<T>(r * (g - s - u * p));
    }
  }
}

// dw and db, first step: a warp for each 32 columns and split of the rows.
constexpr int kColWarps = 8;
template <typename T>
__global__ void __launch_bounds__(32 * kColWarps) vrLnColumns(const __grid_constant__ BwdArgs a) {
  __shared__ float buf[2][kColWarps][32];
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t col = (uint64_t)blockIdx.x * 32 + lane;
  const uint64_t r0 = a.rows * blockIdx.y / a.splits, r1 = a.rows * (blockIdx.y + 1) / a.splits;
  float dw = 0.f, db = 0.f;
  if (col < a.cols) {
    for (uint64_t row = r0 + warp; row < r1; row += kColWarps) {
      const float g = to_f32(static_cast<const T*>(a.dy)[row * a.dyStride + col]);
      const float u =
          (to_f32(static_cast<const T*>(a.x)[row * a.xStride + col]) - a.mean[row]) * a.rstd[row];
      dw = fmaf(g, u, dw);
      db += g;
    }
  }
  buf[0][warp][lane] = dw;
  buf[1][warp][lane] = db;
  __syncthreads();
  if (warp < 2 && col < a.cols) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kColWarps; ++i) s += buf[warp][i][lane];
    a.partials[((uint64_t)blockIdx.y * 2 + warp) * a.cols + col] = s;
  }
}

// dw and db, second step: the splits' sums added up in a fixed order. A block
// takes 32 columns, a warp of it every 32nd split, so that few loads follow one
// another: the kernel is all latency.
constexpr int kJoinWarps = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kJoinWarps) vrLnJoin(const __grid_constant__ BwdArgs a) {
  __shared__ float buf[kJoinWarps][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t first = (uint64_t)blockIdx.x * 32;
  W* out = static_cast<W*>(blockIdx.y ? a.db : a.dw);
  begin_kernel();
  if (!out) return;
  float s = 0.f;
  if (first + lane < a.cols) {
    const float* p = a.partials + (uint64_t)blockIdx.y * a.cols + first + lane;
#pragma unroll 8
    for (int i = warp; i < a.splits; i += kJoinWarps) s += p[(uint64_t)i * 2 * a.cols];
  }
  buf[warp][lane] = s;
  __syncthreads();
  s = warp_sum(buf[lane][warp]);  // column `warp`
  if (lane == 0 && first + warp < a.cols) out[first + warp] = from_f32<W>(s);
}

// The backward pass of rows that are kept on chip: dy and x are read once, dx is
// written once, and the sums of dw and db over a group's rows stay in
// registers until its last row. Each group's ROWS rows lie in shared memory
// through both of their walks (s and p; then dx), STAGES - 1 times as many on
// their way.
template <typename T, typename W, int E, int ROWS, int STAGES, int MODE, bool RAGGED, int REGS>
__global__ void __maxnreg__(REGS) vrLnBackwardRows(const __grid_constant__ BwdArgs a) {
  constexpr int V = kV<T>, P = E / V;
  extern __shared__ uint4 ring[];  // [warps][STAGES][ROWS][dy, x][P][32]
  __shared__ RowSum<MODE, 2 * ROWS> sum;
  begin_kernel();
  const int cols = (int)a.cols;
  const Place<T, MODE, P> at(a.l, a.rows, cols);
  int turn = 0;
  if constexpr (MODE == IN_CLUSTER) cluster_sync();  // the others' buffers are there
  const T* gp = static_cast<const T*>(a.dy) + at.row * a.dyStride;
  const T* xp = static_cast<const T*>(a.x) + at.row * a.xStride;
  const uint64_t gStep = a.l.step * a.dyStride, xStep = a.l.step * a.xStride,
                 oStep = a.l.step * a.dxStride;
  const int apart = (MODE == IN_WARP ? at.stripe : 32) * V;  // elements between a thread's packs
  bool used[P];
#pragma unroll
  for (int i = 0; i < P; ++i) used[i] = at.used(i);
  constexpr int kSet = ROWS * 2 * P * 32;
  uint4* const mine = ring + (threadIdx.x >> 5) * (STAGES * kSet) + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (!used[i])
      for (int k = 0; k < STAGES * ROWS * 2; ++k) mine[(k * P + i) * 32] = make_uint4(0, 0, 0, 0);
  T aheadG[ROWS], aheadX[ROWS];    // the next rows' elements outside the packs
  float nextM[ROWS], nextR[ROWS];  // and their statistics
  const uint32_t ringAt = (uint32_t)__cvta_generic_to_shared(mine);
  auto fetch = [&](int left, const T* g, const T* x, int stage) {
    const uint32_t to = ringAt + stage * (kSet * 16);
    each<ROWS>([&](auto kk) {
      constexpr int k = decltype(kk)::value;
      if (k < left) {
        const T *gk = g + k * gStep, *xk = x + k * xStep;
        each<P>([&](auto ii) {
          constexpr int i = decltype(ii)::value;
          if (!used[i]) return;
          constexpr int at0 = (2 * k * P + i) * 512, at1 = at0 + P * 512;
          if constexpr (MODE == IN_WARP) {
            copy16<at0, 0>(to, gk + i * apart);
            copy16<at1, 0>(to, xk + i * apart);
          } else {
            copy16<at0, i * 512>(to, gk);
            copy16<at1, i * 512>(to, xk);
          }
        });
      }
    });
    copies_commit();
  };
  // Only the first warps of a row hold elements outside the packs.
  const bool edges = RAGGED && __any_sync(~0u, at.edge >= 0);
  const float *mp = a.mean + at.row, *rp = a.rstd + at.row;
  auto fetchRest = [&](int left, const T* g, const T* x) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      nextM[k] = nextR[k] = 0.f;
      if (k < left) {
        nextM[k] = mp[(uint64_t)k * a.l.step];
        nextR[k] = rp[(uint64_t)k * a.l.step];
      }
    }
    mp += (uint64_t)ROWS * a.l.step;
    rp += (uint64_t)ROWS * a.l.step;
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        aheadG[k] = aheadX[k] = from_f32<T>(0.f);
        if (at.edge >= 0 && k < left) {
          aheadG[k] = g[k * gStep + at.edge];
          aheadX[k] = x[k * xStep + at.edge];
        }
      }
    }
  };
  const T *gf = gp + at.column(0), *xf = xp + at.column(0);  // the rows to fetch next
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) {
    fetch(at.n - i * ROWS, gf, xf, i);
    gf += ROWS * gStep;
    xf += ROWS * xStep;
  }
  fetchRest(at.n, gp, xp);
  Params<T, W> w[P];
  float we = 1.f;
#pragma unroll
  for (int i = 0; i < P; ++i)
    w[i].load(static_cast<const W*>(a.w), at.column(i), used[i], 1.f);
  if (RAGGED && at.edge >= 0 && a.w) we = to_f32(static_cast<const W*>(a.w)[at.edge]);
  F2 dw[P][V / 2], db[P][V / 2];
  float dwe = 0.f, dbe = 0.f;
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) dw[i][j] = db[i][j] = f2(0.f);
  const float c = 1.f / (float)cols;
  int left = at.n, stage = 0;
  T* oo = static_cast<T*>(a.dx) + at.row * a.dxStride + at.column(0);
  const int edgeAt = at.edge - at.column(0);
  for (int round = 0; round < at.rounds; round += ROWS) {
    const int back = stage == 0 ? STAGES - 1 : stage - 1;
    fetch(left - (STAGES - 1) * ROWS, gf, xf, back);
    gf += ROWS * gStep;
    xf += ROWS * xStep;
    float m[ROWS], r[ROWS], ge[ROWS], de[ROWS], s[2 * ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      m[k] = nextM[k];
      r[k] = nextR[k];
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        ge[k] = to_f32(aheadG[k]);
        de[k] = to_f32(aheadX[k]) - m[k];
      }
    }
    gp += ROWS * gStep;
    xp += ROWS * xStep;
    fetchRest(left - ROWS, gp, xp);
    copies_wait<STAGES - 1>();
    const uint4* from = mine + stage * kSet;
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      F2 s2 = f2(0.f), p2 = f2(0.f);
      if (k < left) {
        const F2 minus = f2(-m[k]), r2 = f2(r[k]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          F2 g[V / 2], x[V / 2], ww[V / 2];
          unpack<T>(from[(2 * k * P + i) * 32], g);
          unpack<T>(from[((2 * k + 1) * P + i) * 32], x);
          w[i].get(ww);
#pragma unroll
          for (int j = 0; j < V / 2; ++j) {
            const F2 d = x[j] + minus;
            db[i][j] = db[i][j] + g[j];
            dw[i][j] = fma2(g[j] * r2, d, dw[i][j]);
            const F2 gw = g[j] * ww[j];
            s2 = s2 + gw;
            p2 = fma2(gw, d, p2);
          }
        }
      }
      s[2 * k] = both(s2);
      s[2 * k + 1] = both(p2);
    }
    if (edges) {
#pragma unroll
      for (int k = 0; k < ROWS; ++k)
        if (k < left) {
          dbe += ge[k];
          dwe = fmaf(ge[k] * r[k], de[k], dwe);
          ge[k] *= we;
          s[2 * k] += ge[k];
          s[2 * k + 1] = fmaf(ge[k], de[k], s[2 * k + 1]);
        }
    }
    if (a.dx) {
      sum(s, a.l, at.group, turn);
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        // dx = r (g - s - (x - m) r p), s and p the means of g and of g u. Never r^2, which
        // leaves the range of a float long before dx does.
        const float c0 = -(s[2 * k] * c), c1 = -(r[k] * (r[k] * (s[2 * k + 1] * c)));
        const F2 minus = f2(-m[k]), r2 = f2(r[k]), c02 = f2(c0), c12 = f2(c1);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (used[i] && k < left) {
            F2 g[V / 2], x[V / 2], ww[V / 2];
            unpack<T>(from[(2 * k * P + i) * 32], g);
            unpack<T>(from[((2 * k + 1) * P + i) * 32], x);
            w[i].get(ww);
#pragma unroll
            for (int j = 0; j < V / 2; ++j)
              x[j] = fma2(x[j] + minus, c12, fma2(g[j], ww[j], c02)) * r2;
            *reinterpret_cast<uint4*>(oo + k * oStep + i * apart) = pack<T>(x);
          }
        }
        if (edges && at.edge >= 0 && k < left)
          oo[k * oStep + edgeAt] = from_f32<T>(fmaf(de[k], c1, ge[k] + c0) * r[k]);
      }
    }
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    left -= ROWS;
    oo += ROWS * oStep;
  }
  if (!a.dw && !a.db) return;
  copies_wait<0>();
  // The groups' sums are added up in shared memory, in the groups' order, so
  // that a block leaves one; a cluster's blocks write their own columns. In
  // shared memory every eighth word is left out: a thread's columns lie
  // together, and the same one of all lanes would lie in four banks.
  auto slot = [](int col) { return MODE == IN_CLUSTER ? col : col + (col >> 3); };
  float* part = a.partials + (uint64_t)(blockIdx.x / a.l.ctas) * 2 * a.cols;
  const int half = slot(cols + 7);  // dw, then db
  if constexpr (MODE != IN_CLUSTER) {
    __syncthreads();
    part = reinterpret_cast<float*>(ring) + at.group * 2 * half;
  }
  float* const partB = part + (MODE == IN_CLUSTER ? cols : half);
#pragma unroll
  for (int i = 0; i < P; ++i)
    if (used[i]) {
#pragma unroll
      for (int j = 0; j < V / 2; ++j) {
        const int col = at.column(i) + 2 * j;
        split(dw[i][j], part[slot(col)], part[slot(col + 1)]);
        split(db[i][j], partB[slot(col)], partB[slot(col + 1)]);
      }
    }
  if (RAGGED && at.edge >= 0) {
    part[slot(at.edge)] = dwe;
    partB[slot(at.edge)] = dbe;
  }
  if constexpr (MODE != IN_CLUSTER) {
    __syncthreads();
    float* all = reinterpret_cast<float*>(ring);
    float* out = a.partials + (uint64_t)blockIdx.x * 2 * a.cols;
    for (int i = threadIdx.x; i < 2 * cols; i += blockDim.x) {
      const int at0 = i < cols ? slot(i) : half + slot(i - cols);
      float t = all[at0];
      for (int k = 1; k < a.l.groups; ++k) t += all[k * 2 * half + at0];
      if (a.together) all[at0] = t;
      else out[i] = t;
    }
    if (!a.together) return;
    cluster_sync();
    const int blocks = gridDim.x;
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < 2 * cols; i += blocks * blockDim.x) {
      const int at0 = i < cols ? slot(i) : half + slot(i - cols);
      float t = 0.f;
#pragma unroll 8
      for (int k = 0; k < blocks; ++k) t += load_remote(&all[at0], k);
      W* to = static_cast<W*>(i < cols ? a.dw : a.db);
      if (to) to[i < cols ? i : i - cols] = from_f32<W>(t);
    }
    cluster_sync();  // the others may still be reading this block's sums
  }
}

// ------------------------------------------------------------------ host
bool typesOk(vrDataType_t t, vrDataType_t w) {
  return (t == vrFloat16 || t == vrBfloat16 || t == vrFloat32) && (w == t || w == vrFloat32);
}

// f(T, W) for the element type and the parameters' type.
template <typename F>
vrResult_t dispatch(vrDataType_t t, vrDataType_t w, F f) {
  if (t == vrFloat32) return f(float{}, float{});
  if (t == vrFloat16) return w == t ? f(__half{}, __half{}) : f(__half{}, float{});
  return w == t ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, float{});
}

// One shape of the kernel for rows up to `maxThreads` threads wide (times 8 for a
// cluster's blocks). False if a row does not fit.
enum { NARROW = 1, BLOCK = 2, CLUSTER = 4, WHOLE = 8, CUT = 16 };  // what the shape is built for
template <typename T, typename W, int E, int ROWS, int STAGES, int REGS, int FOR>
bool forwardShape(FwdArgs& a, bool ragged, int blockThreads, int maxThreads, cudaStream_t st,
                  vrResult_t* result) {
  constexpr int V = kV<T>;
  int mode;
  if (!layoutFor(a.cols, V, E / V, blockThreads, maxThreads, ragged, &a.l, &mode)) return false;
  const void* k = nullptr;
  auto pick = [&](auto m, auto r) {
    constexpr int MODE = decltype(m)::value;
    constexpr bool RAGGED = decltype(r)::value;
    if constexpr ((FOR & (1 << MODE)) != 0 && (FOR & (RAGGED ? CUT : WHOLE)) != 0)
      if (mode == MODE && ragged == RAGGED)
        k = (const void*)&vrLnForwardRows<T, W, E, ROWS, STAGES, MODE, RAGGED, REGS>;
  };
  const auto each = [&](auto m) {
    pick(m, std::false_type{});
    pick(m, std::true_type{});
  };
  each(std::integral_constant<int, IN_WARP>{});
  each(std::integral_constant<int, IN_BLOCK>{});
  each(std::integral_constant<int, IN_CLUSTER>{});
  if (!k) return false;
  const int threads = a.l.tpr * a.l.groups;
  const size_t smem = (size_t)STAGES * ROWS * E * sizeof(T) * threads;
  if (!allowShared(k)) {
    *result = vrCudaError;
    return true;
  }
  uint64_t most = mostAtOnce(a.l, residentWarps(REGS, smem, threads));
  if (mode == IN_CLUSTER) most = clustersAtOnce(k, a.l, smem, most);
  const unsigned grid = gridFor(a.rows, &a.l, V, most, ragged, ROWS);
  *result = launch(k, dim3(grid), dim3(threads), smem, st, a, a.l.ctas);
  return true;
}

// Rows that are kept in registers: all but the widest. The shapes were chosen by
// measuring on a GB300 (x read and y written once, of the measured copy peak);
// what decides is how many warps an SM holds, how many share a row's sums, and
// that no register is spilled (the ends of ragged rows take a few more).
//  16 elements of 2 rows a thread: narrow rows (256 bf16 0.90, 1024 bf16 0.88),
//    float32 up to 4096 (3000 0.96; with 32 of one row 0.69), and ragged rows up
//    to 8192 (8191 bf16 0.69, 3001 float32 0.84; 0.55 and 0.52).
//  32 elements of 2 rows: whole packs of 16-bit rows over 256 (4096 bf16 0.92
//    against 0.88, 640 0.77 against 0.61, 6000 0.84 against 0.66 with one row),
//    and all rows up to 12288 beyond the above (12288 bf16 0.86 against 0.69,
//    10240 float32 0.90 against 0.66) -- but for 7 or 8 warps a row, of which an
//    SM holds one row only, and 64 whole threads of the first shape (1024 bf16
//    0.88 against 0.86).
//  16 elements of 4 rows: ragged 16-bit rows up to 2048, whose one-element loads
//    are latency (2051 bf16 0.77 against 0.68).
//  32 elements of one row: the rest (8192 bf16 0.91 against 0.80, 16384 0.81).
//  Clusters, whose barrier is paid twice for each set of rows: of 32 elements of
//    2 rows in blocks of 384 threads where these are as few as of 512 (24576 bf16
//    0.56 against 0.40, 49152 0.53 against 0.36, 24576 float32 0.70 against 0.48),
//    else of one row (32768 bf16 0.46 against 0.44, 65536 0.43 against 0.37), of
//    float32 the first shape (32768 0.63 against 0.57) up to 65536.
template <typename T, typename W>
bool forwardRows(FwdArgs& a, cudaStream_t st, vrResult_t* r) {
  constexpr bool half = sizeof(T) == 2;
  a.l.offset = (int)((uintptr_t)a.x & 15);
  a.l.skew = (int)((a.xStride * sizeof(T)) & 15);
  const bool ragged = a.l.offset || a.l.skew || a.cols % kV<T>;
  const uint64_t warps = (a.cols / 32 + 31) / 32;  // of a row, 32 elements a thread
  const bool oneRow = warps == 7 || warps == 8;
  const auto blocks = [&](uint64_t threads) {  // of a row, 32 elements a thread
    uint64_t n = 1;
    while (n <= 8 && n * threads * 32 < a.cols / kV<T> * kV<T>) n *= 2;
    return n;
  };
  const bool asFew = blocks(384) == blocks(512);
  if constexpr (half) {
    const bool full = a.cols > 960 && a.cols <= 1024;  // 64 threads of 16 elements
    if (!ragged && a.cols > 256 && !full && !oneRow && asFew &&
        forwardShape<T, W, 32, 2, 2, 168, NARROW | BLOCK | CLUSTER | WHOLE>(a, ragged, 128, 384, st,
                                                                            r))
      return true;
    if (ragged && forwardShape<T, W, 16, 4, 2, 168, NARROW | BLOCK | CUT>(a, ragged, 128, 128, st, r))
      return true;
    return (ragged ? forwardShape<T, W, 16, 2, 2, 128, BLOCK | CUT>(a, ragged, 256, 512, st, r) ||
                         (asFew && forwardShape<T, W, 32, 2, 2, 168, BLOCK | CLUSTER | CUT>(
                                       a, ragged, 128, 384, st, r))
                   : forwardShape<T, W, 16, 2, 2, 128, NARROW | BLOCK | WHOLE>(a, ragged, 256, 64,
                                                                               st, r)) ||
           forwardShape<T, W, 32, 1, 3, 128, BLOCK | CLUSTER | WHOLE | CUT>(a, ragged, 256, 512, st, r);
  } else {
    // Just under 128 threads of 32 elements (4096 0.92 against 0.86 with 16 of two
    // rows; 3500 0.80 against 0.89).
    const bool full = !ragged && a.cols > 3840 && a.cols <= 4096;
    return (!full && forwardShape<T, W, 16, 2, 2, 128, NARROW | BLOCK | WHOLE | CUT>(
                         a, ragged, 256, ragged ? 512 : 256, st, r)) ||
           (!full && asFew && forwardShape<T, W, 32, 2, 2, 168, BLOCK | CLUSTER | WHOLE | CUT>(
                                  a, ragged, 128, 384, st, r)) ||
           ((ragged || a.cols > 16384) &&
            forwardShape<T, W, 16, 2, 2, 128, CLUSTER | WHOLE | CUT>(a, ragged, 256, 512, st, r)) ||
           (!ragged &&
            forwardShape<T, W, 32, 1, 3, 128, BLOCK | CLUSTER | WHOLE>(a, ragged, 256, 512, st, r));
  }
}

template <typename T, typename W, int MODE>
const void* backwardKernel(bool ragged) {
  return ragged ? (const void*)&vrLnBackwardRows<T, W, 16, 2, 2, MODE, true, 128>
                : (const void*)&vrLnBackwardRows<T, W, 16, 2, 2, MODE, false, 128>;
}
// False if the rows do not fit.
template <typename T, typename W>
bool backwardRows(BwdArgs& a, cudaStream_t st, vrResult_t* r) {
  const int offset = (int)((uintptr_t)a.x & 15), skew = (int)((a.xStride * sizeof(T)) & 15);
  const bool ragged = offset || skew || a.cols % kV<T>;
  BwdPlan p;
  const int shape = planBackward<T>(a.rows, a.cols, ragged, &p);
  if (shape == NO_PLAN) return false;
  const void* k = nullptr;
  if (p.mode == IN_WARP) k = backwardKernel<T, W, IN_WARP>(ragged);
  if (p.mode == IN_BLOCK) k = backwardKernel<T, W, IN_BLOCK>(ragged);
  if constexpr (sizeof(T) == 2)
    if (p.mode == IN_CLUSTER) k = backwardKernel<T, W, IN_CLUSTER>(ragged);
  if constexpr (sizeof(T) == 4)
    if (shape == ONE_ROW) {
      if (p.mode == IN_BLOCK)
        k = ragged ? (const void*)&vrLnBackwardRows<T, W, 16, 1, 3, IN_BLOCK, true, 128>
                   : (const void*)&vrLnBackwardRows<T, W, 16, 1, 3, IN_BLOCK, false, 128>;
      else
        k = ragged ? (const void*)&vrLnBackwardRows<T, W, 16, 1, 3, IN_CLUSTER, true, 128>
                   : (const void*)&vrLnBackwardRows<T, W, 16, 1, 3, IN_CLUSTER, false, 128>;
    }
  if constexpr (sizeof(T) == 2)
    if (shape == ONE_WARP)
      k = (const void*)&vrLnBackwardRows<T, W, 32, 2, 2, IN_WARP, false, 168>;
  if (shape == WIDE) {
    if (p.mode == IN_BLOCK)
      k = ragged ? (const void*)&vrLnBackwardRows<T, W, 32, kWideRows<T>, 2, IN_BLOCK, true, 168>
                 : (const void*)&vrLnBackwardRows<T, W, 32, kWideRows<T>, 2, IN_BLOCK, false, 168>;
    else
      k = ragged ? (const void*)&vrLnBackwardRows<T, W, 32, kWideRows<T>, 2, IN_CLUSTER, true, 168>
                 : (const void*)&vrLnBackwardRows<T, W, 32, kWideRows<T>, 2, IN_CLUSTER, false, 168>;
  }
  if (!k) return false;
  if (!allowShared(k)) {
    *r = vrCudaError;
    return true;
  }
  if (p.mode == IN_CLUSTER)
    p.grid = gridFor(a.rows, &p.l, kV<T>, clustersAtOnce(k, p.l, p.smem, p.most), ragged, p.rowsAtOnce);
  a.l = p.l;
  a.l.offset = offset;
  a.l.skew = skew;
  a.splits = (int)(p.grid / p.l.ctas);
  if ((a.dw || a.db) && planTogether<T>(a.rows, a.cols, ragged, &p)) {
    a.together = true;
    a.l.step = p.l.step;
    if (!allowLargeClusters(k)) {
      *r = vrCudaError;
      return true;
    }
  }
  *r = launch(k, dim3(p.grid), dim3(p.threads), p.smem, st, a, a.together ? (int)p.grid : p.l.ctas);
  return true;
}

bool badMatrix(const void* p, uint64_t cols, uint64_t stride, int es) {
  return !p || misaligned(p, es) || stride < cols;
}

}  // namespace

extern "C" VR_API vrResult_t vrLayerNormForward(const void* x, const void* weight,
                                                const void* bias, void* y, float* mean,
                                                float* rstd, size_t rows, size_t cols,
                                                size_t xStride, size_t yStride, float eps,
                                                vrDataType_t dtype, vrDataType_t weightType,
                                                void* stream) {
  NvtxRange range("vrLayerNormForward");
  if (!typesOk(dtype, weightType) || cols < 1 || !(eps >= 0.f) || !(eps - eps == 0.f))
    return vrInvalidArgument;
  if (rows == 0) return vrSuccess;
  const int es = elemSizeOf(dtype), ws = elemSizeOf(weightType);
  if (badMatrix(x, cols, xStride, es) || badMatrix(y, cols, yStride, es) ||
      misaligned(weight, ws) || misaligned(bias, ws) || misaligned(mean, 4) || misaligned(rstd, 4))
    return vrInvalidArgument;
  const bool inPlace = x == y && xStride == yStride;
  const Bytes outs[] = {bytesOf(y, rows, cols, yStride, es), bytesOf(mean, rows * 4), bytesOf(rstd, rows * 4)};
  const Bytes ins[] = {bytesOf(inPlace ? nullptr : x, rows, cols, xStride, es), bytesOf(weight, cols * ws),
                       bytesOf(bias, cols * ws)};
  if (anyOverlap(outs, 3, ins, 3)) return vrInvalidArgument;
  FwdArgs a = {x, weight, bias, y, mean, rstd, rows, cols, xStride, yStride, eps, {}};
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    vrResult_t r;
    if (alike(x, xStride, y, yStride, es) && rows < kMostRows &&
        forwardRows<T, W>(a, (cudaStream_t)stream, &r))
      return r;
    const uint64_t most = (uint64_t)kSMs * 8;
    return launch((const void*)&vrLnForwardAny<T, W>, dim3((unsigned)(rows < most ? rows : most)),
                  dim3(kRowThreads), 0, (cudaStream_t)stream, a);
  });
}

extern "C" VR_API vrResult_t vrLayerNormBackwardWorkspace(size_t rows, size_t cols,
                                                          vrDataType_t dtype, size_t* bytes) {
  if (!typesOk(dtype, dtype) || cols < 1 || !bytes) return vrInvalidArgument;
  const uint64_t splits =
      dtype == vrFloat32 ? mostSplits<float>(rows, cols) : mostSplits<__half>(rows, cols);
  *bytes = (size_t)(splits * 2 * cols * sizeof(float));
  return vrSuccess;
}

extern "C" VR_API vrResult_t vrLayerNormBackward(
    const void* dy, const void* x, const void* weight, const float* mean, const float* rstd,
    void* dx, void* dweight, void* dbias, size_t rows, size_t cols, size_t dyStride,
    size_t xStride, size_t dxStride, vrDataType_t dtype, vrDataType_t weightType, void* workspace,
    size_t workspaceBytes, void* stream) {
  NvtxRange range("vrLayerNormBackward");
  if (!typesOk(dtype, weightType) || cols < 1) return vrInvalidArgument;
  const int es = elemSizeOf(dtype), ws = elemSizeOf(weightType);
  if (misaligned(dweight, ws) || misaligned(dbias, ws)) return vrInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  if (rows == 0) {  // sums over no rows
    if ((dweight && cudaMemsetAsync(dweight, 0, cols * ws, st) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, cols * ws, st) != cudaSuccess)) {
      cudaGetLastError();
      return vrCudaError;
    }
    return vrSuccess;
  }
  if (badMatrix(dy, cols, dyStride, es) || badMatrix(x, cols, xStride, es) ||
      misaligned(weight, ws) || !mean || !rstd || misaligned(mean, 4) || misaligned(rstd, 4) ||
      (dx && badMatrix(dx, cols, dxStride, es)))
    return vrInvalidArgument;
  const bool params = dweight || dbias;
  BwdArgs a = {dy, x, weight, mean, rstd, dx, dweight, dbias, rows, cols,
               dyStride, xStride, dxStride, (float*)workspace, splitsFor(rows, cols), false, {}};
  size_t need = 0;
  if (params && (vrLayerNormBackwardWorkspace(rows, cols, dtype, &need) != vrSuccess ||
                 !workspace || misaligned(workspace, 16) || workspaceBytes < need))
    return vrInvalidArgument;
  const Bytes outs[] = {bytesOf(dx, rows, cols, dxStride, es), bytesOf(dweight, cols * ws),
                        bytesOf(dbias, cols * ws), bytesOf(workspace, need)};
  const Bytes ins[] = {bytesOf(dy, rows, cols, dyStride, es), bytesOf(x, rows, cols, xStride, es),
                       bytesOf(weight, cols * ws), bytesOf(mean, rows * 4), bytesOf(rstd, rows * 4)};
  if (anyOverlap(outs, 4, ins, 5)) return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    vrResult_t r = vrSuccess;
    const bool same = alike(dy, dyStride, x, xStride, es) && (!dx || alike(dx, dxStride, x, xStride, es));
    if (!same || !backwardRows<T, W>(a, st, &r)) {
      const uint64_t most = (uint64_t)kSMs * 8;
      if (dx)
        r = launch((const void*)&vrLnBackwardAny<T, W>,
                   dim3((unsigned)(rows < most ? rows : most)), dim3(kRowThreads), 0, st, a);
      if (r == vrSuccess && params)
        r = launch((const void*)&vrLnColumns<T>, dim3((unsigned)((cols + 31) / 32), a.splits),
                   dim3(32 * kColWarps), 0, st, a);
    }
    if (r == vrSuccess && params && !a.together)
      r = launch((const void*)&vrLnJoin<W>, dim3((unsigned)((cols + 31) / 32), 2),
                 dim3(32 * kJoinWarps), 0, st, a);
    return r;
  });
}
