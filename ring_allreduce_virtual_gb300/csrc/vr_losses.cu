// vr_losses.cu -- log probabilities of target tokens under rows of logits, the losses of
// policies and of preferences made of them, and the gradients of the logits.
//
//   lse = log(sum(exp(x))), logp = x[target] - lse
//   dx[j] = c ([j = target] - exp(x[j] - lse)), c the derivative by logp
// Policy: with e = logp - old, a row's loss is
//   w (-min(exp(e) A, clip(exp(e), 1 - low, 1 + high) A) + kl (exp(ref - logp) - (ref - logp) - 1))
// Preference: with S the sum of logp over a sequence and h = beta ((S - ref) of the chosen
// one less the same of the rejected), a pair's loss is
//   (1 - smoothing) softplus(-h) + smoothing softplus(h)
//
// Rows are summed in 32 bits over their largest element; what follows for each row, where
// an error in the last place decides on which side of the clipping's border a row is, is
// done in pairs of floats. All of it is bound by memory traffic (two exponentials an element).
#include <float.h>
#include <math.h>

#include <cmath>

#include "vr_packs.cuh"

namespace {

using namespace vrop;

struct LossArgs {
  const void* x;
  void* dx;
  const int64_t* target;
  uint64_t rows, cols, stride, dStride;
  float *logp, *lse, *rest, *coef;  // coef: the derivative by logp
  // policies
  const float *old, *advantage, *weight, *ref;
  float2* rowLoss;  // a number and what its rounding lost
  float2 low, high, least, most;  // logs of the ratio's borders, the borders: sums of two floats
  float kl, scale;
  float* loss;
  // the gradient's kernel
  const float* dlogp;
  const float* gain;  // multiplies dlogp, or NULL
  uint64_t segments;  // blocks of a row
  bool alike;         // dx's rows lie as x's modulo 16 bytes
  // the kernel that keeps a row on chip
  int ctas;           // blocks of a row
  uint32_t part;      // packs of a block
  bool eager;         // rows are copied before it is known whether they count
  uint32_t c65536;    // 65536
  // preferences
  const float* refSums;
  const int64_t* starts;
  double* sums;
  float* seqLogp;
  uint64_t pairs;
  float beta, smoothing;
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The sum of exponentials of some elements less the largest of them, both so far. It
// starts at the lowest finite number, so that elements of -inf add 0 and not NaN; +inf and
// NaN make the sum NaN.
struct Online {
  float m = -FLT_MAX, s = 0.f;
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      s *= exp2_fast((m - to) * kLog2e);
      m = to;
    }
  }
  // The distance from the largest is taken before the product with log2(e): its rounding
  // then is small where the exponential is large.
  __device__ __forceinline__ void add(float x) {
    raise(x);
    s += exp2_fast((x - m) * kLog2e);
  }
  // U packs, whose largest element is found first, of 16-bit types two at a time.
  template <typename T, int U>
  __device__ __forceinline__ void add(const uint4 (&v)[U], uint32_t c65536) {
    constexpr int V = kV<T>, H = V / 2;
    F2 f[U][H];
    float top;
    if constexpr (sizeof(T) == 2) {
      using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
      T2 most[U * 4];
      memcpy(most, v, sizeof(most));
#pragma unroll
      for (int n = U * 2; n; n >>= 1)
#pragma unroll
        for (int i = 0; i < n; ++i) most[i] = __hmax2(most[i], most[i + n]);
      top = fmaxf(to_f32(most[0].x), to_f32(most[0].y));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) unpack<T>(v[u], c65536, f[u]);
    if constexpr (sizeof(T) == 4) {
      top = -INFINITY;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < H; ++i) {
          float p, q;
          split(f[u][i], p, q);
          top = fmaxf(top, fmaxf(p, q));
        }
    }
    raise(top);
    const F2 less = f2(-m), scale = f2(kLog2e);
    F2 sum = f2(0.f);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < H; ++i) {
        float p, q;
        split((f[u][i] + less) * scale, p, q);
        sum = sum + f2(exp2_fast(p), exp2_fast(q));
      }
    s += both(sum);
  }
  __device__ __forceinline__ void join(float m2, float s2) {
    const float to = fmaxf(m, m2);
    s = s * exp2_fast((m - to) * kLog2e) + s2 * exp2_fast((m2 - to) * kLog2e);
    m = to;
  }
};

// A pack of elements that add nothing.
template <typename T>
__device__ __forceinline__ uint4 nothing() {
  const uint32_t w = sizeof(T) == 4 ? 0xff800000u : std::is_same_v<T, __half> ? 0xfc00fc00u : 0xff80ff80u;
  return make_uint4(w, w, w, w);
}

// A number as the sum of two floats, and what is done with it: 48 bits at the price of a few
// instructions, where one of 64 bits takes the time of 16. `add` is Knuth's two-sum; of a sum
// that is not finite the second float says nothing.
struct Pair {
  float s = 0.f, e = 0.f;
  __device__ __forceinline__ void add(float v, float rest = 0.f) {
    const float t = __fadd_rn(s, v), p = __fadd_rn(t, -s);
    const float lost = __fadd_rn(__fadd_rn(s, -__fadd_rn(t, -p)), __fadd_rn(v, -p)) + rest;
    e = t - t == 0.f ? e + lost : 0.f;
    s = t;
  }
  __device__ __forceinline__ void times(float f) {
    const float p = __fmul_rn(s, f), lost = fmaf(s, f, -p);
    e = p - p == 0.f ? fmaf(e, f, lost) : 0.f;
    s = p;
  }
  __device__ __forceinline__ float value() const { return s + e; }
  __device__ __forceinline__ void warp() {
#pragma unroll
    for (int k = 16; k; k >>= 1) add(__shfl_xor_sync(~0u, s, k), __shfl_xor_sync(~0u, e, k));
  }
};

// log(s): k log(2), of which the first part is k times 16 bits and so exact, and the logarithm
// of a number between 3/4 and 3/2, whose error is 2^-25 at most.
__device__ __forceinline__ Pair log_of(float s) {
  Pair l;
  if (!(s > 0.f && s < FLT_MAX)) {
    l.s = logf(s);
    return l;
  }
  constexpr double kLog2 = 0.693147180559945309417;
  constexpr float kUpper = (float)((double)(int)(kLog2 * 65536.0) / 65536.0), kLower = (float)(kLog2 - (double)kUpper);
  int k;
  float f = frexpf(s, &k);  // in [1/2, 1)
  if (f < 0.75f) f *= 2.f, --k;
  l.s = (float)k * kUpper;
  l.add(logf(f), (float)k * kLower);
  return l;
}

enum { LOGP = 0, POLICY = 1 };

// What one thread loads of a row ahead of the row's sum.
struct RowIn {
  float at, old, advantage, weight, ref;  // at: the target's logit
  template <int KIND, typename T>
  __device__ __forceinline__ void load(const LossArgs& a, uint64_t row, const T* x, int64_t target) {
    at = (uint64_t)target < a.cols ? to_f32(x[target]) : __int_as_float(0x7fffffff);
    if constexpr (KIND == POLICY) {
      old = a.old[row];
      advantage = a.advantage[row];
      weight = a.weight ? a.weight[row] : 1.f;
      ref = a.ref ? a.ref[row] : 0.f;
    }
  }
};

// What a row comes to whose exponentials sum to s over its largest element m: logp is
// returned with the loss's derivative by it. lse is that element and a logarithm, and where
// the first is large (an offset of all logits, masks of the lowest number) their rounded sum
// has lost the second: `rest` is what it lost, and logp is made of the distance from the
// largest. Of a cluster's blocks one writes.
template <int KIND>
__device__ __forceinline__ float2 finish_row(const LossArgs& a, uint64_t row, const RowIn& in, float m, float s,
                                             bool write = true) {
  const Pair l = log_of(s);
  Pair lp;
  lp.s = in.at;
  lp.add(-m);
  lp.add(-l.s, -l.e);
  const float logp = lp.value();
  float c = 0.f;
  [[maybe_unused]] Pair loss;
  if constexpr (KIND == POLICY) {
    // Next to a border of the clipping, and where rows' losses cancel in their sum, 24 bits
    // are too few.
    const float A = in.advantage;
    Pair e = lp;
    e.add(-in.old);
    const float above = (e.s - a.high.x) + (e.e - a.high.y), below = (e.s - a.low.x) + (e.e - a.low.y);
    if (A > 0.f && above > 0.f) {
      loss.s = -a.most.x, loss.e = -a.most.y;
      loss.times(A);
    } else if (A < 0.f && below < 0.f) {
      loss.s = -a.least.x, loss.e = -a.least.y;
      loss.times(A);
    } else if (A != 0.f || e.s != e.s) {  // an advantage of 0 hides no NaN
      const float f = e.value();
      if (f > -0.5f) {
        loss.s = -A;
        loss.add(-expm1f(f) * A);
      } else {
        loss.s = -expf(f) * A;
      }
      c = loss.value();
    }
    if (a.ref) {
      Pair d;
      d.s = in.ref;
      d.add(-lp.s, -lp.e);
      const float r = d.value(), x = expm1f(r);
      loss.add(a.kl * (x < INFINITY ? x - r : x));  // of an impossible token r is infinite too
      c = fmaf(-a.kl, x, c);
    }
    loss.times(in.weight);
    c *= a.scale * in.weight;
  }
  if (write) {
    a.logp[row] = logp;
    if (a.lse) {
      Pair lse;
      lse.s = m;
      lse.add(l.s, l.e);
      const float rounded = lse.value();
      a.lse[row] = rounded;
      if (a.rest) a.rest[row] = lse.e - (rounded - lse.s);
    }
    if constexpr (KIND == POLICY) {
      a.rowLoss[row] = make_float2(loss.s, loss.e);
      a.coef[row] = c;
    }
  }
  return make_float2(logp, c);
}
// A row that counts for nothing: its logits are not read.
template <int KIND>
__device__ __forceinline__ void skip_row(const LossArgs& a, uint64_t row) {
  a.logp[row] = 0.f;
  if (a.lse) a.lse[row] = 0.f;
  if (a.rest) a.rest[row] = 0.f;
  if constexpr (KIND == POLICY) {
    a.rowLoss[row] = make_float2(0.f, 0.f);
    a.coef[row] = 0.f;
  }
}
template <int KIND>
__device__ __forceinline__ bool skipped(const LossArgs& a, uint64_t row, int64_t target) {
  return target < 0 || (KIND == POLICY && a.weight && a.weight[row] == 0.f);
}

// A row, cut at memory's 16-byte boundaries: `head` elements, whole packs, and the rest.
template <typename T>
struct Cut {
  int head;
  uint64_t packs;
  __device__ __forceinline__ Cut(const T* p, uint64_t cols) {
    constexpr int V = kV<T>;
    head = (int)((16 - ((uintptr_t)p & 15)) & 15) / (int)sizeof(T);
    if ((uint64_t)head > cols) head = (int)cols;
    packs = (cols - head) / V;
  }
  // The element outside the packs of a thread, -1: none.
  __device__ __forceinline__ int64_t edge(int thread, uint64_t cols) const {
    const uint64_t i = thread < head ? thread : thread + packs * kV<T>;
    return i < cols && thread < 2 * kV<T> ? (int64_t)i : -1;
  }
};

// The sums of a block's threads joined, in an order fixed by the lanes; the same in all.
struct Joined {
  float tops[16], sums[16];
  __device__ __forceinline__ void warp(Online& o, int width) const {
    float m = o.m;
    for (int k = width / 2; k; k >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, k));
    float s = o.s * exp2_fast((o.m - m) * kLog2e);
    for (int k = width / 2; k; k >>= 1) s += __shfl_xor_sync(~0u, s, k);
    o.m = m, o.s = s;
  }
  __device__ __forceinline__ void operator()(Online& o) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    warp(o, 32);
    if (warps == 1) return;
    if (lane == 0) tops[threadIdx.x >> 5] = o.m, sums[threadIdx.x >> 5] = o.s;
    __syncthreads();
    const bool in = (lane & 15) < warps;
    o.m = in ? tops[lane & 15] : -FLT_MAX;
    o.s = in ? sums[lane & 15] : 0.f;
    warp(o, 16);
  }
};

// The same over the blocks of a cluster, each of which has announced itself (arrive) before.
struct Parts {
  float m[8], s[8];
  __device__ __forceinline__ static void arrive() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  }
  __device__ __forceinline__ void operator()(Online& o, int rank, int ctas) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the others are there
    if ((int)threadIdx.x < ctas) {
      store_remote(&m[rank], threadIdx.x, o.m);
      store_remote(&s[rank], threadIdx.x, o.s);
    }
    cluster_sync();
    o = Online{};
    for (int i = 0; i < ctas; ++i) o.join(m[i], s[i]);
  }
};

constexpr int kRowThreads = 256;

// A block for each row, or a warp for each of a block's, read once, the next packs on their
// way while the last are summed. Bound by HBM for long rows: 4096 x 131072 bf16 155 us, 1.03 of
// the measured copy peak; 8192 x 32000 0.97, 16384 x 5000 0.68 (a row's way from its target
// to its sum is some 4 us, of which blocks of 10 KB cannot hide all).
template <typename T, int KIND, bool CLUSTER>
__global__ void __launch_bounds__(kRowThreads, 4) vrRowLogs(const __grid_constant__ LossArgs a) {
  constexpr int U = 4;
  __shared__ Joined joined;
  __shared__ Parts parts;
  begin_kernel();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int ctas = CLUSTER ? a.ctas : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
  if (CLUSTER) Parts::arrive();
  for (uint64_t row = (uint64_t)(blockIdx.x / ctas) * blockDim.y + threadIdx.y; row < a.rows;
       row += (uint64_t)(gridDim.x / ctas) * blockDim.y) {
    const int64_t target = a.target[row];
    if (skipped<KIND>(a, row, target)) {
      if (tid == 0 && rank == 0) skip_row<KIND>(a, row);
      if (CLUSTER) return;  // one row a cluster
      continue;
    }
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const Cut<T> cut(x, a.cols);
    RowIn in;
    if (tid == 0) in.load<KIND>(a, row, x, target);
    Online o;
    const uint4* p = reinterpret_cast<const uint4*>(x + cut.head) + tid;
    int64_t left = (int64_t)cut.packs - tid;  // a pack of this thread is every threads-th
    if (CLUSTER) {
      const int64_t first = (int64_t)rank * a.part;
      p += first;
      left = ((int64_t)cut.packs - first < (int64_t)a.part ? (int64_t)cut.packs - first : (int64_t)a.part) - tid;
    }
    const int64_t edge = rank == 0 ? cut.edge(tid, a.cols) : -1;
    if (edge >= 0) o.add(to_f32(x[edge]));
    uint4 v[U];
    if (left > (U - 1) * threads) {
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = p[k * threads];
      p += U * threads;
      left -= U * threads;
      while (left > (U - 1) * threads) {
        uint4 w[U];
#pragma unroll
        for (int k = 0; k < U; ++k) w[k] = p[k * threads];
        o.add<T>(v, a.c65536);
#pragma unroll
        for (int k = 0; k < U; ++k) v[k] = w[k];
        p += U * threads;
        left -= U * threads;
      }
      o.add<T>(v, a.c65536);
    }
    if (left > 0) {
#pragma unroll
      for (int k = 0; k < U; ++k) v[k] = k * threads < left ? p[k * threads] : nothing<T>();
      o.add<T>(v, a.c65536);
    }
    joined(o);
    if (CLUSTER) parts(o, rank, ctas);
    if (tid == 0 && rank == 0) finish_row<KIND>(a, row, in, o.m, o.s);
    if (CLUSTER) return;
    if (threads > 32) __syncthreads();
  }
}

// f exp(x - m - rest) of a pack's elements. Results of 16 bits take |f| and rest in the
// exponent, where they cost nothing (off by 2^-20 of the result), and f's sign afterwards.
struct Factor {
  float m, add, f;
  uint32_t sign;
  template <typename T>
  __device__ __forceinline__ static Factor of(float m, float rest, float f) {
    if constexpr (sizeof(T) == 4) return {m, -rest, f, 0};
    return {m, fmaf(-rest, kLog2e, __log2f(fabsf(f))), f, __float_as_uint(f) & 0x80000000u};
  }
};
template <typename T>
__device__ __forceinline__ void scaled_exps(const uint4& v, const Factor& k, uint32_t c65536, float (&e)[kV<T>]) {
  constexpr int V = kV<T>;
  F2 x[V / 2];
  unpack<T>(v, c65536, x);
  const F2 less = f2(-k.m), add = f2(k.add), scale = f2(kLog2e);
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    float p, q;
    if constexpr (sizeof(T) == 4) {
      split((x[i] + less + add) * scale, p, q);
      split(f2(exp2_fast(p), exp2_fast(q)) * f2(k.f), e[2 * i], e[2 * i + 1]);
    } else {
      split(fma2(x[i] + less, scale, add), p, q);
      e[2 * i] = __uint_as_float(__float_as_uint(exp2_fast(p)) ^ k.sign);
      e[2 * i + 1] = __uint_as_float(__float_as_uint(exp2_fast(q)) ^ k.sign);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store_pack(T* p, const float (&e)[kV<T>], bool alike) {
  constexpr int V = kV<T>;
  if (alike) {
    F2 f[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) f[i] = f2(e[2 * i], e[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = pack<T>(f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = from_f32<T>(e[i]);
  }
}

template <typename T, typename I>
__device__ __forceinline__ void zero_packs(T* p, I from, I to, I step, bool alike) {
  const float zero[kV<T>] = {};
#pragma unroll 4
  for (I i = from; i < to; i += step) store_pack<T>(p + (int64_t)i * kV<T>, zero, alike);
}

// The logarithms and the gradient of a row in one pass over it: its packs are copied to
// shared memory, each by the thread that reads it (no barrier between), summed as they
// come, and read again there for the gradient. A row is a warp's, a block's, or a cluster's,
// each block with its part of it. A block's way is 8.5 to 10 us (its target 0.8, its copies 3.8,
// sums and their joining 1.1, a cluster's 1.5, the loss 0.7, the gradient 2.1), three or four
// blocks are on an SM. Of the measured copy peak, with half of the rows counting and with all:
// 8192 x 32000 bf16 0.90 and 0.87 (130, 178 us), 8192 x 50001 0.84 and 0.80 (215, 302 us; the two
// kernels of one pass each 274 and 393), 8192 x 50257 float32 0.88 and 0.87. What took it there from 0.49 is four packs a thread side by side, in straight lines.
constexpr int kLossThreads = 256;
template <typename T, int KIND, bool CLUSTER>
__global__ void __launch_bounds__(kLossThreads, 4) vrRowLossGrads(const __grid_constant__ LossArgs a) {
  constexpr int V = kV<T>, GROUPS = 4;
  extern __shared__ uint4 shared[];
  __shared__ Joined joined;
  __shared__ Parts parts;
  __shared__ float3 results[kLossThreads / 32];
  begin_kernel();
  const int tid = threadIdx.x, threads = blockDim.x;
  const int ctas = CLUSTER ? a.ctas : 1, rank = CLUSTER ? (int)cluster_rank() : 0;
  if (CLUSTER) Parts::arrive();
  const uint64_t row = (uint64_t)(blockIdx.x / ctas) * blockDim.y + threadIdx.y;
  if (row >= a.rows) return;
  uint4* const packs = shared + threadIdx.y * a.part;
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  T* dx = static_cast<T*>(a.dx) + row * a.dStride;
  const int64_t target = a.target[row];
  const Cut<T> cut(x, a.cols);
  const int first = rank * (int)a.part, all = (int)cut.packs - first;
  const int n = all < 0 ? 0 : all < (int)a.part ? all : (int)a.part;  // this block's packs
  const int64_t edge = rank == 0 ? cut.edge(tid, a.cols) : -1;
  T* const dp = dx + cut.head + (int64_t)first * V;
  const uint4* p = reinterpret_cast<const uint4*>(x + cut.head) + first;
  const int each = ((n + threads - 1) / threads + 4 * GROUPS - 1) / (4 * GROUPS) * 4 * threads;  // packs of a group
  const uint32_t to = (uint32_t)__cvta_generic_to_shared(packs);
  const auto fetch = [&]() {
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const int end = min(n, (g + 1) * each);
#pragma unroll 4
      for (int i = g * each + tid; i < end; i += threads)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * 16), "l"(p + i) : "memory");
      copies_commit();
    }
  };
  if (a.eager) fetch();
  if (skipped<KIND>(a, row, target)) {
    copies_wait<0>();
    zero_packs<T>(dp, tid, n, threads, a.alike);
    if (edge >= 0) dx[edge] = from_f32<T>(0.f);
    if (tid == 0 && rank == 0) skip_row<KIND>(a, row);
    return;
  }
  if (!a.eager) fetch();
  RowIn in;
  if (tid == 0) in.load<KIND>(a, row, x, target);
  Online o;
  float e = 0.f;
  if (edge >= 0) {
    e = to_f32(x[edge]);
    o.add(e);
  }
  const auto sum = [&](int g) {
    const int end = min(n, (g + 1) * each);
    for (int i = g * each + tid; i < end; i += 4 * threads) {
      uint4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) v[u] = i + u * threads < end ? packs[i + u * threads] : nothing<T>();
      o.add<T>(v, a.c65536);
    }
  };
  copies_wait<3>();
  sum(0);
  copies_wait<2>();
  sum(1);
  copies_wait<1>();
  sum(2);
  copies_wait<0>();
  sum(3);
  joined(o);
  if (CLUSTER) parts(o, rank, ctas);
  if (tid == 0) {
    const float2 r = finish_row<KIND>(a, row, in, o.m, o.s, rank == 0);
    results[threadIdx.y] = make_float3(r.x, r.y, -r.y / o.s);
  }
  if (threads == 32) __syncwarp();
  else __syncthreads();
  const float lp = results[threadIdx.y].x, c = results[threadIdx.y].y, f = results[threadIdx.y].z;
  // The target's element is c (1 - p) without the difference of two numbers near 1. Of a
  // target that is none c is NaN.
  const bool none = c == 0.f;
  const Factor factor = Factor::of<T>(o.m, 0.f, f);
  const int64_t t = target - cut.head - (int64_t)first * V;
  if (none) {
    zero_packs<T>(dp, tid, n, threads, a.alike);
  } else {
    for (int i = tid; i < n; i += 4 * threads) {  // four chains side by side, then the stores
      float d[4][V];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        scaled_exps<T>(packs[i + u * threads < n ? i + u * threads : i], factor, a.c65536, d[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (i + u * threads < n) store_pack<T>(dp + (int64_t)(i + u * threads) * V, d[u], a.alike);
    }
    if (t >= 0 && t < (int64_t)n * V && (int)(t / V) % threads == tid) dp[t] = from_f32<T>(-c * expm1f(lp));
  }
  if (edge >= 0)
    dx[edge] = from_f32<T>(none             ? 0.f
                           : edge == target ? -c * expm1f(lp)
                                            : f * exp2_fast((e - o.m) * kLog2e));
}

// dx from the rows' logarithms, read by an earlier kernel: a block takes some rows' parts,
// from the last row on, which that kernel read last. All of a group's arithmetic comes before
// its stores (4096 x 131072 bf16 308 us, 1.03 of the measured copy peak; with a branch for the
// target and the end between them 468).
constexpr int kGradThreads = 256;
template <typename T, int U>
__global__ void __launch_bounds__(kGradThreads) vrRowGrads(const __grid_constant__ LossArgs a) {
  constexpr int V = kV<T>;
  begin_kernel();
  const uint64_t line = blockIdx.x / a.segments;  // of rows
  const uint64_t back = line * blockDim.y + threadIdx.y;
  if (back >= a.rows) return;
  const uint64_t row = a.rows - 1 - back;
  const T* x = static_cast<const T*>(a.x) + row * a.stride;
  T* dx = static_cast<T*>(a.dx) + row * a.dStride;
  const int64_t target = a.target[row];
  float c = a.dlogp[row];
  const float lse = a.lse[row], rest = a.rest ? a.rest[row] : 0.f, gain = a.gain ? *a.gain : 1.f;
  if (target < 0) c = 0.f;
  if (c != 0.f) c *= gain;  // a row of 0 stays one, whatever the gain is
  if (target >= (int64_t)a.cols && c != 0.f) c = __int_as_float(0x7fffffff);
  const Cut<T> cut(x, a.cols);
  const uint64_t segment = blockIdx.x - line * a.segments;
  const bool none = c == 0.f;
  if (segment == 0) {
    const int64_t edge = cut.edge(threadIdx.x, a.cols);
    if (edge >= 0) {
      const float d = none ? 0.f : (to_f32(x[edge]) - lse) - rest;
      dx[edge] = from_f32<T>(none ? 0.f : edge == target ? -c * expm1f(d) : -c * exp2_fast(d * kLog2e));
    }
  }
  const int threads = blockDim.x;
  const uint64_t first = segment * a.part + threadIdx.x;
  const uint64_t end = first - threadIdx.x + a.part < cut.packs ? first - threadIdx.x + a.part : cut.packs;
  const uint4* p = reinterpret_cast<const uint4*>(x + cut.head);
  T* const dp = dx + cut.head;
  if (none) {
    zero_packs<T>(dp, first, end, (uint64_t)threads, a.alike);
    return;
  }
  // The target's element is left to the thread that writes its pack, which reads it before.
  const int64_t t = target - cut.head, at = t >= 0 ? t / V : -1, place = at - (int64_t)(segment * a.part);
  const bool mine = place >= 0 && at < (int64_t)end && (int)(place % threads) == (int)threadIdx.x;
  const float atTarget = mine ? to_f32(x[target]) : 0.f;
  const Factor factor = Factor::of<T>(lse, rest, -c);
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (first + u * threads < end) v[u] = p[first + u * threads];
  for (uint64_t i = first; i < end; i += U * threads) {
    uint4 w[U];  // the next, on their way
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + (U + u) * threads < end) w[u] = p[i + (U + u) * threads];
    float d[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) scaled_exps<T>(v[u], factor, a.c65536, d[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i + u * threads < end) store_pack<T>(dp + (i + u * threads) * V, d[u], a.alike);
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = w[u];
  }
  if (mine) dp[t] = from_f32<T>(-c * expm1f((atTarget - lse) - rest));
}

constexpr int kOneBlock = 1024;

// The sum of a value of each thread, in an order fixed by the lanes; the same in all.
__device__ double block_total(double v) {
  __shared__ double buf[kOneBlock / 32], all;
  static_assert(kOneBlock == 32 * 32, "a warp adds up the warps' sums");
  v = warp_sum(v);
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = warp_sum(buf[threadIdx.x]);
    if (threadIdx.x == 0) all = v;
  }
  __syncthreads();
  return all;
}

// The rows' losses added up.
__global__ void __launch_bounds__(kOneBlock) vrLossSum(const __grid_constant__ LossArgs a) {
  __shared__ Pair warps[32];
  begin_kernel();
  Pair p;
#pragma unroll 8
  for (uint64_t i = threadIdx.x; i < a.rows; i += kOneBlock) {
    const float2 v = a.rowLoss[i];
    p.add(v.x, v.y);
  }
  p.warp();
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = p;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  p = warps[threadIdx.x];
  p.warp();
  if (threadIdx.x == 0) *a.loss = (float)(((double)p.s + (double)p.e) * (double)a.scale);
}

// The sequences' sums, the pairs' losses and the derivatives by the rows' logp.
__global__ void __launch_bounds__(kOneBlock) vrPairLosses(const __grid_constant__ LossArgs a) {
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint64_t sequences = 2 * a.pairs;
  auto range = [&](uint64_t s, uint64_t& from, uint64_t& to) {
    if (a.starts) {  // cut at the rows that there are
      const int64_t f = a.starts[s], t = a.starts[s + 1], all = (int64_t)a.rows;
      from = (uint64_t)(f < 0 ? 0 : f > all ? all : f);
      to = (uint64_t)(t < 0 ? 0 : t > all ? all : t);
    } else {
      from = a.rows / sequences * s;
      to = from + a.rows / sequences;
    }
  };
  for (uint64_t i = threadIdx.x; i < a.rows; i += kOneBlock) a.coef[i] = 0.f;
  for (uint64_t s = warp; s < sequences; s += kOneBlock / 32) {
    uint64_t from, to;
    range(s, from, to);
    double sum = 0.0;
#pragma unroll 8
    for (uint64_t i = from + lane; i < to; i += 32) sum += (double)a.logp[i];
    sum = warp_sum(sum);
    if (lane == 0) {
      a.sums[s] = sum;
      a.seqLogp[s] = (float)sum;
    }
  }
  __syncthreads();
  double loss = 0.0;
  for (uint64_t i = threadIdx.x; i < a.pairs; i += kOneBlock) {
    double h = a.sums[i] - a.sums[a.pairs + i];
    if (a.refSums) h -= (double)a.refSums[i] - (double)a.refSums[a.pairs + i];
    const float f = (float)(h * (double)a.beta), e = expf(-fabsf(f));  // in (0, 1]
    const float soft = log1pf(e);
    const float up = soft + fmaxf(f, 0.f), down = soft + fmaxf(-f, 0.f);  // softplus of f and -f
    const float p = (f >= 0.f ? 1.f : e) / (1.f + e), q = (f >= 0.f ? e : 1.f) / (1.f + e);
    // A term of factor 0 is left out: it may be infinite (of an impossible token's sum of -inf).
    float pair = a.smoothing < 1.f ? (1.f - a.smoothing) * down : 0.f;
    if (a.smoothing > 0.f) pair += a.smoothing * up;
    loss += (double)pair;
    // in the place of the chosen one's sum; NaN stays one
    a.sums[i] = (double)(a.scale * a.beta * (a.smoothing * p - (1.f - a.smoothing) * (f == f ? q : f)));
  }
  loss = block_total(loss);  // and a barrier
  if (threadIdx.x == 0) *a.loss = (float)(loss * (double)a.scale);
  for (uint64_t s = warp; s < sequences; s += kOneBlock / 32) {
    uint64_t from, to;
    range(s, from, to);
    const float c = (float)a.sums[s < a.pairs ? s : s - a.pairs];
    for (uint64_t i = from + lane; i < to; i += 32)
      a.coef[i] = a.target[i] < 0 ? 0.f : s < a.pairs ? c : -c;
  }
}

// ------------------------------------------------------------------ host
constexpr uint64_t kMost = 1ull << 48;  // elements from the first to the last of a matrix

// A number as the sum of two floats.
float2 two(double v) {
  const float s = (float)v;
  return float2{s, std::isfinite(s) ? (float)(v - (double)s) : 0.f};
}

bool typeOk(vrDataType_t t) { return t == vrFloat16 || t == vrBfloat16 || t == vrFloat32; }

bool badMatrix(const void* p, uint64_t rows, uint64_t cols, uint64_t stride, int es) {
  return !p || misaligned(p, es) || stride < cols || stride > kMost / rows;
}

template <typename F>
vrResult_t dispatch(vrDataType_t t, F f) {
  if (t == vrFloat32) return f(float{});
  return t == vrFloat16 ? f(__half{}) : f(__nv_bfloat16{});
}

template <typename T, int KIND>
vrResult_t rowLogs(LossArgs& a, cudaStream_t st) {
  // Up to 256 threads, of 32 packs each, so that many rows are on their way at a time (8192 x
  // 32000 bf16 80 us, of 8 packs 88); 8 packs where there are few rows; rows of a warp eight in a
  // block. Few rows are
  // clusters', in parts of 32 KB at least, up to the four blocks of an SM; the fewest in
  // parts of 8 KB (200 x 32000 bf16 in clusters 5.9 us, without 5.2).
  const uint64_t packs = a.cols / kV<T>;
  int ctas = 1;
  while (ctas < 8 && a.rows * ctas * 2 <= 4 * kSMs && packs / ctas >= (a.rows * ctas * 8 <= kSMs ? 1024 : 4096)) ctas *= 2;
  const uint64_t part = (packs + ctas - 1) / ctas;
  a.ctas = ctas;
  a.part = (uint32_t)part;
  const uint64_t each = a.rows * ctas > 8 * kSMs ? 32 : 8;
  uint64_t threads = (part / each + 31) / 32 * 32;
  threads = threads < 32 ? 32 : threads > kRowThreads ? kRowThreads : threads;
  const unsigned y = threads == 32 ? kRowThreads / 32 : 1;
  const uint64_t groups = (a.rows + y - 1) / y, most = 1u << 20;
  const void* k = ctas > 1 ? (const void*)&vrRowLogs<T, KIND, true> : (const void*)&vrRowLogs<T, KIND, false>;
  return launch(k, dim3((unsigned)(groups < most ? groups : most) * ctas), dim3((unsigned)threads, y), 0, st, a, ctas);
}

template <typename T>
void alikeRows(LossArgs& a) {
  a.alike = (((uintptr_t)a.x - (uintptr_t)a.dx) & 15) == 0 &&
            (a.rows == 1 || (((a.stride - a.dStride) * sizeof(T)) & 15) == 0);
}

template <typename T>
vrResult_t rowGrads(LossArgs& a, cudaStream_t st) {
  alikeRows<T>(a);
  const uint64_t packs = a.cols / kV<T> ? a.cols / kV<T> : 1;
  // A row's threads, a power of two up to a block, of 32 packs each (16384 x 5000 bf16 55 us, of 4
  // packs 105), or as many as fill the GPU three blocks an SM; parts of 4096 packs, of 1024 where
  // those are few.
  unsigned x = 32;
  while (x < kGradThreads && x * 32 < packs) x *= 2;
  while (x < kGradThreads && x * 4 < packs && a.rows * x < 3ull * kSMs * kGradThreads) x *= 2;
  const unsigned y = kGradThreads / x;
  a.part = a.rows * packs >= (uint64_t)kSMs * 16 * 4096 ? 4096 : 1024;
  a.segments = (packs + a.part - 1) / a.part;
  const uint64_t blocks = (a.rows + y - 1) / y * a.segments;
  if (blocks > 0x7fffffffu) return vrInvalidArgument;
  return launch((const void*)&vrRowGrads<T, 4>, dim3((unsigned)blocks), dim3(x, y), 0, st, a);
}

// Logarithms and gradient in one pass; false if a row is too large for a cluster. Parts of up to
// 72 KB and 256 threads, four blocks an SM by their registers (8192 x 50001 bf16, all rows counting,
// 315 us before the pairs of floats; parts of 36 KB and 128 threads 327, of 52 KB and 192 threads
// 336; 4096 x 50257 float32 300, 330, 314).
constexpr size_t kMostShared = 200 * 1024;
template <typename T, int KIND>
bool rowLossGrads(LossArgs& a, cudaStream_t st, vrResult_t* r) {
  alikeRows<T>(a);
  const uint64_t packs = a.cols / kV<T> ? a.cols / kV<T> : 1;
  constexpr uint64_t kBest = 72 * 1024 / 16, kLargest = kMostShared / 16;
  int ctas = 1;
  while (ctas < 8 && (packs + ctas - 1) / ctas > kBest) ctas *= 2;
  // Few rows are spread over more SMs, in parts of 8 KB at least, up to six blocks on each.
  while (ctas < 8 && a.rows * ctas * 2 <= 6 * kSMs && packs / ctas >= 1024) ctas *= 2;
  const uint64_t part = (packs + ctas - 1) / ctas;
  // 16 packs a thread, so that many rows are on their way at a time (16384 x 8000 bf16, all counting, 93 us, of 8
  // packs 98, of 4 142; of 32 133); 4 where there are few.
  const uint64_t each = a.rows * ctas > 6 * kSMs ? 16 : 4;
  uint64_t threads = (part / each + 31) / 32 * 32;
  threads = threads < 32 ? 32 : threads > kLossThreads ? kLossThreads : threads;
  const unsigned y = threads == 32 ? kLossThreads / 32 : 1;
  const uint64_t blocks = (a.rows + y - 1) / y * ctas;
  if (part > kLargest || blocks > 0x7fffffffu) return false;
  a.ctas = ctas;
  a.part = (uint32_t)part;
  a.eager = blocks <= 6 * kSMs;  // a microsecond less where there is only one round
  const void* k = ctas > 1 ? (const void*)&vrRowLossGrads<T, KIND, true> : (const void*)&vrRowLossGrads<T, KIND, false>;
  if (!setOnce(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostShared) ||
      !setOnce(k, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared)) {
    *r = vrCudaError;
    return true;
  }
  *r = launch(k, dim3((unsigned)blocks), dim3((unsigned)threads, y), part * 16 * y, st, a, ctas);
  return true;
}

// Rows up to 2^32: eight of them or more are a block's where they are narrow.
bool sizesOk(uint64_t rows, uint64_t cols) {
  return cols >= 1 && cols <= kMost && rows <= kMost / cols && rows <= 1ull << 32;
}

}  // namespace

extern "C" VR_API vrResult_t vrTokenLogProbsForward(const void* logits, const int64_t* targets, float* logp,
                                                    float* lse, float* rest, size_t rows, size_t cols,
                                                    size_t stride, vrDataType_t dtype, void* stream) {
  NvtxRange range("vrTokenLogProbsForward");
  if (!typeOk(dtype) || !sizesOk(rows, cols)) return vrInvalidArgument;
  if (rows == 0) return vrSuccess;
  const int es = elemSizeOf(dtype);
  if (badMatrix(logits, rows, cols, stride, es) || !targets || misaligned(targets, 8) || !logp ||
      misaligned(logp, 4) || misaligned(lse, 4) || misaligned(rest, 4) || (rest && !lse))
    return vrInvalidArgument;
  const Bytes outs[] = {bytesOf(logp, rows * 4), bytesOf(lse, rows * 4), bytesOf(rest, rows * 4)};
  const Bytes ins[] = {bytesOf(logits, rows, cols, stride, es), bytesOf(targets, rows * 8)};
  if (anyOverlap(outs, 3, ins, 2)) return vrInvalidArgument;
  LossArgs a;
  memset(&a, 0, sizeof(a));
  a.c65536 = 65536;
  a.x = logits, a.target = targets, a.logp = logp, a.lse = lse, a.rest = rest;
  a.rows = rows, a.cols = cols, a.stride = stride;
  return dispatch(dtype, [&](auto t) { return rowLogs<decltype(t), LOGP>(a, (cudaStream_t)stream); });
}

extern "C" VR_API vrResult_t vrTokenLogProbsBackward(const float* dlogp, const float* gain, const void* logits,
                                                     const int64_t* targets, const float* lse,
                                                     const float* rest, void* dlogits, size_t rows, size_t cols, size_t stride, size_t dStride,
                                                     vrDataType_t dtype, void* stream) {
  NvtxRange range("vrTokenLogProbsBackward");
  if (!typeOk(dtype) || !sizesOk(rows, cols)) return vrInvalidArgument;
  if (rows == 0) return vrSuccess;
  const int es = elemSizeOf(dtype);
  if (badMatrix(logits, rows, cols, stride, es) || badMatrix(dlogits, rows, cols, dStride, es) || !targets ||
      misaligned(targets, 8) || !dlogp || misaligned(dlogp, 4) || !lse || misaligned(lse, 4) || misaligned(rest, 4) ||
      misaligned(gain, 4))
    return vrInvalidArgument;
  const bool over = logits == dlogits && stride == dStride;
  const Bytes outs[] = {bytesOf(dlogits, rows, cols, dStride, es)};
  const Bytes ins[] = {bytesOf(over ? nullptr : logits, rows, cols, stride, es), bytesOf(targets, rows * 8),
                       bytesOf(dlogp, rows * 4), bytesOf(lse, rows * 4), bytesOf(rest, rows * 4), bytesOf(gain, 4)};
  if (anyOverlap(outs, 1, ins, 6)) return vrInvalidArgument;
  LossArgs a;
  memset(&a, 0, sizeof(a));
  a.c65536 = 65536;
  a.x = logits, a.dx = dlogits, a.target = targets, a.lse = const_cast<float*>(lse), a.rest = const_cast<float*>(rest);
  a.dlogp = dlogp, a.gain = gain;
  a.rows = rows, a.cols = cols, a.stride = stride, a.dStride = dStride;
  return dispatch(dtype, [&](auto t) { return rowGrads<decltype(t)>(a, (cudaStream_t)stream); });
}

extern "C" VR_API vrResult_t vrPolicyLossWorkspace(size_t rows, size_t* bytes) {
  if (!bytes || rows > kMost) return vrInvalidArgument;
  *bytes = rows * sizeof(float2);
  return vrSuccess;
}

extern "C" VR_API vrResult_t vrPolicyLoss(const void* logits, const int64_t* targets, const float* oldLogp,
                                          const float* advantages, const float* weights, const float* refLogp,
                                          float* loss, float* logp, float* lse, float* rest, float* dlogp,
                                          void* dlogits, size_t rows, size_t cols, size_t stride, size_t dStride, double clipLow,
                                          double clipHigh, float klCoef, float scale, vrDataType_t dtype,
                                          void* workspace, size_t workspaceBytes, void* stream) {
  NvtxRange range("vrPolicyLoss");
  if (!typeOk(dtype) || !sizesOk(rows, cols) || !(clipLow >= 0.0) || !(clipHigh >= 0.0) ||
      !(klCoef - klCoef == 0.f) || !(scale - scale == 0.f) || !loss || misaligned(loss, 4))
    return vrInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  LossArgs a;
  memset(&a, 0, sizeof(a));
  a.c65536 = 65536;
  a.loss = loss, a.scale = scale, a.rows = rows, a.cols = cols;
  if (rows) {
    const int es = elemSizeOf(dtype);
    size_t need = 0;
    vrPolicyLossWorkspace(rows, &need);
    if (badMatrix(logits, rows, cols, stride, es) || !targets || misaligned(targets, 8) || !oldLogp ||
        misaligned(oldLogp, 4) || !advantages || misaligned(advantages, 4) || misaligned(weights, 4) ||
        misaligned(refLogp, 4) || !logp || misaligned(logp, 4) || !lse || misaligned(lse, 4) || !rest ||
        misaligned(rest, 4) || !dlogp || misaligned(dlogp, 4) || (dlogits && badMatrix(dlogits, rows, cols, dStride, es)) || !workspace ||
        misaligned(workspace, 16) || workspaceBytes < need)
      return vrInvalidArgument;
    const bool over = logits == dlogits && stride == dStride;
    const Bytes x = bytesOf(logits, rows, cols, stride, es), d = bytesOf(dlogits, rows, cols, dStride, es);
    const Bytes outs[] = {bytesOf(loss, 4), bytesOf(logp, rows * 4), bytesOf(lse, rows * 4), bytesOf(rest, rows * 4),
                          bytesOf(dlogp, rows * 4), bytesOf(workspace, need), d};
    const Bytes ins[] = {bytesOf(targets, rows * 8), bytesOf(oldLogp, rows * 4), bytesOf(advantages, rows * 4),
                         bytesOf(weights, rows * 4), bytesOf(refLogp, rows * 4)};
    if (anyOverlap(outs, 7, ins, 5) || (!over && overlap(d, x))) return vrInvalidArgument;
    for (int i = 0; i < 6; ++i)
      if (overlap(outs[i], x)) return vrInvalidArgument;
    a.x = logits, a.dx = dlogits, a.target = targets, a.stride = stride, a.dStride = dStride;
    a.logp = logp, a.lse = lse, a.rest = rest, a.coef = dlogp, a.dlogp = dlogp, a.rowLoss = (float2*)workspace;
    a.old = oldLogp, a.advantage = advantages, a.weight = weights, a.ref = klCoef != 0.f ? refLogp : nullptr;
    a.least = two(1.0 - clipLow), a.most = two(1.0 + clipHigh);
    a.low = two(clipLow < 1.0 ? log1p(-clipLow) : -INFINITY), a.high = two(log1p(clipHigh));
    a.kl = klCoef;
    const vrResult_t r = dispatch(dtype, [&](auto t) {
      using T = decltype(t);
      vrResult_t rc;
      if (dlogits && rowLossGrads<T, POLICY>(a, st, &rc)) return rc;
      rc = rowLogs<T, POLICY>(a, st);
      return rc == vrSuccess && dlogits ? rowGrads<T>(a, st) : rc;
    });
    if (r != vrSuccess) return r;
  }
  return launch((const void*)&vrLossSum, dim3(1), dim3(kOneBlock), 0, st, a);
}

extern "C" VR_API vrResult_t vrPreferenceLossWorkspace(size_t pairs, size_t* bytes) {
  if (!bytes || pairs < 1 || pairs > kMost) return vrInvalidArgument;
  *bytes = pairs * 2 * sizeof(double);
  return vrSuccess;
}

extern "C" VR_API vrResult_t vrPreferenceLoss(const void* logits, const int64_t* targets, const float* refLogps,
                                              const int64_t* starts, float* loss, float* logps, float* logp,
                                              float* lse, float* rest, float* dlogp, void* dlogits, size_t pairs,
                                              size_t rows, size_t cols, size_t stride, size_t dStride, float beta,
                                              float labelSmoothing, float scale, vrDataType_t dtype, void* workspace,
                                              size_t workspaceBytes, void* stream) {
  NvtxRange range("vrPreferenceLoss");
  size_t need = 0;
  if (!typeOk(dtype) || !sizesOk(rows, cols) || vrPreferenceLossWorkspace(pairs, &need) != vrSuccess ||
      (!starts && rows % (2 * pairs)) || !(beta - beta == 0.f) || !(scale - scale == 0.f) ||
      !(labelSmoothing >= 0.f && labelSmoothing <= 1.f) || !loss || misaligned(loss, 4) || !logps ||
      misaligned(logps, 4) || misaligned(refLogps, 4) || misaligned(starts, 8) || !workspace ||
      misaligned(workspace, 16) || workspaceBytes < need)
    return vrInvalidArgument;
  const int es = elemSizeOf(dtype);
  if (rows && (badMatrix(logits, rows, cols, stride, es) || !targets || misaligned(targets, 8) || !logp ||
               misaligned(logp, 4) || !lse || misaligned(lse, 4) || !rest || misaligned(rest, 4) || !dlogp ||
               misaligned(dlogp, 4) || (dlogits && badMatrix(dlogits, rows, cols, dStride, es))))
    return vrInvalidArgument;
  const bool over = logits == dlogits && stride == dStride;
  const Bytes x = bytesOf(logits, rows, cols, stride, es), d = bytesOf(dlogits, rows, cols, dStride, es);
  const Bytes outs[] = {bytesOf(loss, 4), bytesOf(logps, pairs * 8), bytesOf(workspace, need),
                        bytesOf(rows ? logp : nullptr, rows * 4), bytesOf(rows ? lse : nullptr, rows * 4),
                        bytesOf(rows ? rest : nullptr, rows * 4), bytesOf(rows ? dlogp : nullptr, rows * 4), d};
  const Bytes ins[] = {bytesOf(rows ? targets : nullptr, rows * 8), bytesOf(refLogps, pairs * 8),
                       bytesOf(starts, (2 * pairs + 1) * 8)};
  if (anyOverlap(outs, 8, ins, 3) || (!over && overlap(d, x))) return vrInvalidArgument;
  for (int i = 0; i < 7; ++i)
    if (overlap(outs[i], x)) return vrInvalidArgument;
  LossArgs a;
  memset(&a, 0, sizeof(a));
  a.c65536 = 65536;
  a.x = logits, a.dx = dlogits, a.target = targets, a.rows = rows, a.cols = cols, a.stride = stride, a.dStride = dStride;
  a.logp = logp, a.lse = lse, a.rest = rest, a.coef = dlogp, a.dlogp = dlogp;
  a.loss = loss, a.seqLogp = logps, a.refSums = refLogps, a.starts = starts, a.sums = (double*)workspace;
  a.pairs = pairs, a.beta = beta, a.smoothing = labelSmoothing, a.scale = scale;
  cudaStream_t st = (cudaStream_t)stream;
  vrResult_t r = vrSuccess;
  if (rows) r = dispatch(dtype, [&](auto t) { return rowLogs<decltype(t), LOGP>(a, st); });
  if (r == vrSuccess) r = launch((const void*)&vrPairLosses, dim3(1), dim3(kOneBlock), 0, st, a);
  if (r == vrSuccess && rows && dlogits) r = dispatch(dtype, [&](auto t) { return rowGrads<decltype(t)>(a, st); });
  return r;
}
