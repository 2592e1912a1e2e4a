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
// done in 64. All of it is bound by memory traffic (two exponentials an element).
#include <float.h>
#include <math.h>

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
  float* rowLoss;
  double low, high;  // logs of the ratio's borders
  float least, most;  // the borders
  float kl, scale;
  float* loss;
  // the gradient's kernel
  const float* dlogp;
  const float* gain;  // multiplies dlogp, or NULL
  uint64_t slots;     // packs that a row can touch
  bool alike;         // dx's rows lie as x's modulo 16 bytes
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
  template <typename T>
  __device__ __forceinline__ void add(const uint4& v) {
    constexpr int V = kV<T>;
    F2 f[V / 2];
    float e[V];
    unpack<T>(v, f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) split(f[i], e[2 * i], e[2 * i + 1]);
    float top = e[0];
#pragma unroll
    for (int i = 1; i < V; ++i) top = fmaxf(top, e[i]);
    raise(top);
    const F2 less = f2(-m), scale = f2(kLog2e);
    F2 sum = f2(0.f);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      float p, q;
      split((f[i] + less) * scale, p, q);
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

// log(s) in 64 bits but for the logarithm of a number between 3/4 and 3/2, whose error in
// 32 bits is 2^-25 at most.
__device__ __forceinline__ double log_of(float s) {
  if (!(s > 0.f && s < FLT_MAX)) return (double)logf(s);
  int k;
  float f = frexpf(s, &k);  // in [1/2, 1)
  if (f < 0.75f) f *= 2.f, --k;
  return fma((double)k, 0.693147180559945309417, (double)logf(f));
}

enum { LOGP = 0, POLICY = 1 };

// What a row comes to whose exponentials sum to s over its largest element m. lse is that
// element and a logarithm, and where the first is large (an offset of all logits, masks of
// the lowest number) their rounded sum has lost the second: `rest` is what it lost, and
// logp is made of the distance from the largest.
template <int KIND>
__device__ __forceinline__ void finish_row(const LossArgs& a, uint64_t row, float m, float s, double at) {
  const double l = log_of(s), lp = (at - (double)m) - l;
  a.logp[row] = (float)lp;
  if (a.lse) {
    const float lse = (float)((double)m + l);
    a.lse[row] = lse;
    if (a.rest) a.rest[row] = (float)(((double)m - (double)lse) + l);
  }
  if constexpr (KIND == POLICY) {
    const float A = a.advantage[row], w = a.weight ? a.weight[row] : 1.f;
    const double e = lp - (double)a.old[row];
    float loss = 0.f, c = 0.f;
    if (A > 0.f && e > a.high) loss = -(a.most * A);
    else if (A < 0.f && e < a.low) loss = -(a.least * A);
    else if (A != 0.f) loss = c = -(expf((float)e) * A);
    if (a.ref) {
      const float r = (float)((double)a.ref[row] - lp), x = expm1f(r);
      loss = fmaf(a.kl, x - r, loss);
      c = fmaf(-a.kl, x, c);
    }
    a.rowLoss[row] = w * loss;
    a.coef[row] = a.scale * w * c;
  }
}
// A row that counts for nothing: its logits are not read.
template <int KIND>
__device__ __forceinline__ void skip_row(const LossArgs& a, uint64_t row) {
  a.logp[row] = 0.f;
  if (a.lse) a.lse[row] = 0.f;
  if (a.rest) a.rest[row] = 0.f;
  if constexpr (KIND == POLICY) a.rowLoss[row] = a.coef[row] = 0.f;
}
template <int KIND>
__device__ __forceinline__ bool skipped(const LossArgs& a, uint64_t row) {
  return a.target[row] < 0 || (KIND == POLICY && a.weight && a.weight[row] == 0.f);
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

// A block for each row, read once.
template <typename T, int KIND>
__global__ void __launch_bounds__(512) vrRowLogs(const __grid_constant__ LossArgs a) {
  __shared__ float tops[16], sums[16];
  begin_kernel();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    if (skipped<KIND>(a, row)) {
      if (tid == 0) skip_row<KIND>(a, row);
      continue;
    }
    const T* x = static_cast<const T*>(a.x) + row * a.stride;
    const Cut<T> cut(x, a.cols);
    Online o;
    const int64_t edge = cut.edge(tid, a.cols);
    if (edge >= 0) o.add(to_f32(x[edge]));
    const uint4* p = reinterpret_cast<const uint4*>(x + cut.head);
    uint64_t i = tid;
    for (; i + 3 * threads < cut.packs; i += 4 * threads) {
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = p[i + k * threads];
#pragma unroll
      for (int k = 0; k < 4; ++k) o.add<T>(v[k]);
    }
    for (; i < cut.packs; i += threads) o.add<T>(p[i]);
#pragma unroll
    for (int k = 16; k; k >>= 1)
      o.join(__shfl_xor_sync(~0u, o.m, k), __shfl_xor_sync(~0u, o.s, k));
    if (threads > 32) {
      if (lane == 0) tops[warp] = o.m, sums[warp] = o.s;
      __syncthreads();
      if (warp == 0) {
        const bool in = lane < threads / 32;
        o.m = in ? tops[lane] : -FLT_MAX;
        o.s = in ? sums[lane] : 0.f;
#pragma unroll
        for (int k = 8; k; k >>= 1)
          o.join(__shfl_xor_sync(~0u, o.m, k), __shfl_xor_sync(~0u, o.s, k));
      }
    }
    if (tid == 0) {
      const uint64_t t = (uint64_t)a.target[row];
      finish_row<KIND>(a, row, o.m, o.s, t < a.cols ? (double)to_f32(x[t]) : (double)NAN);
    }
    if (threads > 32) __syncthreads();
  }
}

// dx from the rows' logarithms: a thread takes U packs of dx, as in dropout.
constexpr int kGradThreads = 256;
template <typename T, int U>
__global__ void __launch_bounds__(kGradThreads) vrRowGrads(const __grid_constant__ LossArgs a) {
  constexpr int V = kV<T>;
  begin_kernel();
  const uint64_t first = (uint64_t)blockIdx.x * (kGradThreads * U) + threadIdx.x;
  const uint64_t all = a.rows * a.slots;
  const float gain = a.gain ? *a.gain : 1.f;
  const T* x[U];
  T* dx[U];
  int64_t col[U], target[U];
  float c[U], lse[U], rest[U];
  bool some[U], whole[U];
  uint4 v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t slot = first + u * kGradThreads;
    some[u] = whole[u] = false;
    if (slot >= all) continue;
    const uint64_t row = all >> 32 ? slot / a.slots : (uint32_t)slot / (uint32_t)a.slots;
    T* d0 = static_cast<T*>(a.dx) + row * a.dStride;
    col[u] = (int64_t)((slot - row * a.slots) * V) - (int64_t)(((uintptr_t)d0 & 15) / sizeof(T));
    dx[u] = d0 + col[u];
    x[u] = static_cast<const T*>(a.x) + row * a.stride + col[u];
    some[u] = col[u] < (int64_t)a.cols;
    whole[u] = col[u] >= 0 && col[u] + V <= (int64_t)a.cols;
    target[u] = a.target[row];
    c[u] = target[u] < 0 ? 0.f : a.dlogp[row];
    if (c[u] != 0.f) c[u] *= gain;  // a row of 0 stays one, whatever it holds and the gain is
    lse[u] = a.lse[row];
    rest[u] = a.rest ? a.rest[row] : 0.f;
    if (whole[u] && c[u] != 0.f) {
      if (a.alike) {
        v[u] = *reinterpret_cast<const uint4*>(x[u]);
      } else {
        T e[V];
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = x[u][i];
        memcpy(&v[u], e, 16);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!some[u]) continue;
    const int64_t t = target[u] - col[u];
    // At the target 1 - p without the difference of two numbers near 1.
    auto one = [&](float e, int i) {
      if (c[u] == 0.f) return 0.f;
      if (target[u] >= (int64_t)a.cols) return __int_as_float(0x7fffffff);
      const float d = (e - lse[u]) - rest[u];
      return i == t ? -c[u] * expm1f(d) : -c[u] * exp2_fast(d * kLog2e);
    };
    if (whole[u]) {
      float e[V];
      F2 f[V / 2];
      if (c[u] != 0.f) {
        unpack<T>(v[u], f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) split(f[i], e[2 * i], e[2 * i + 1]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = one(e[i], i);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[i] = f2(e[2 * i], e[2 * i + 1]);
      *reinterpret_cast<uint4*>(dx[u]) = pack<T>(f);
    } else {
      for (int i = 0; i < V; ++i) {
        if (col[u] + i < 0 || col[u] + i >= (int64_t)a.cols) continue;
        dx[u][i] = from_f32<T>(one(c[u] == 0.f ? 0.f : to_f32(x[u][i]), i));
      }
    }
  }
}

constexpr int kOneBlock = 1024;

// The sum of a value of each thread, in an order fixed by the lanes; the same in all.
__device__ double block_total(double v) {
  __shared__ double buf[kOneBlock / 32];
  return block_sum<kOneBlock / 32>(v, buf);
}

// The rows' losses added up.
__global__ void __launch_bounds__(kOneBlock) vrLossSum(const __grid_constant__ LossArgs a) {
  begin_kernel();
  double s = 0.0;
  for (uint64_t i = threadIdx.x; i < a.rows; i += kOneBlock) s += (double)a.rowLoss[i];
  s = block_total(s);
  if (threadIdx.x == 0) *a.loss = (float)(s * (double)a.scale);
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
    loss += (double)((1.f - a.smoothing) * down + a.smoothing * up);
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
  // Eight packs a thread, up to 512 threads.
  uint64_t threads = (a.cols / kV<T> / 8 + 31) / 32 * 32;
  threads = threads < 32 ? 32 : threads > 512 ? 512 : threads;
  const uint64_t most = 1u << 20;
  return launch((const void*)&vrRowLogs<T, KIND>, dim3((unsigned)(a.rows < most ? a.rows : most)),
                dim3((unsigned)threads), 0, st, a);
}

template <typename T>
vrResult_t rowGrads(LossArgs& a, cudaStream_t st) {
  constexpr uint64_t V = kV<T>;
  a.slots = (a.cols + 2 * (V - 1)) / V;
  a.alike = (((uintptr_t)a.x - (uintptr_t)a.dx) & 15) == 0 &&
            (a.rows == 1 || (((a.stride - a.dStride) * sizeof(T)) & 15) == 0);
  const uint64_t slots = a.rows * a.slots;
  const bool many = slots >= (uint64_t)kSMs * 8 * kGradThreads * 2;
  const uint64_t each = many ? 4 * kGradThreads : kGradThreads;
  const void* k = many ? (const void*)&vrRowGrads<T, 4> : (const void*)&vrRowGrads<T, 1>;
  const uint64_t blocks = (slots + each - 1) / each;
  if (blocks > 0x7fffffffu) return vrInvalidArgument;
  return launch(k, dim3((unsigned)blocks), dim3(kGradThreads), 0, st, a);
}

bool sizesOk(uint64_t rows, uint64_t cols) { return cols >= 1 && cols <= kMost && rows <= kMost / cols; }

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
  a.x = logits, a.dx = dlogits, a.target = targets, a.lse = const_cast<float*>(lse), a.rest = const_cast<float*>(rest);
  a.dlogp = dlogp, a.gain = gain;
  a.rows = rows, a.cols = cols, a.stride = stride, a.dStride = dStride;
  return dispatch(dtype, [&](auto t) { return rowGrads<decltype(t)>(a, (cudaStream_t)stream); });
}

extern "C" VR_API vrResult_t vrPolicyLossWorkspace(size_t rows, size_t* bytes) {
  if (!bytes || rows > kMost) return vrInvalidArgument;
  *bytes = rows * sizeof(float);
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
    a.logp = logp, a.lse = lse, a.rest = rest, a.coef = dlogp, a.dlogp = dlogp, a.rowLoss = (float*)workspace;
    a.old = oldLogp, a.advantage = advantages, a.weight = weights, a.ref = klCoef != 0.f ? refLogp : nullptr;
    a.least = (float)(1.0 - clipLow), a.most = (float)(1.0 + clipHigh);
    a.low = clipLow < 1.0 ? log1p(-clipLow) : -INFINITY, a.high = log1p(clipHigh);
    a.kl = klCoef;
    const vrResult_t r = dispatch(dtype, [&](auto t) {
      const vrResult_t rc = rowLogs<decltype(t), POLICY>(a, st);
      return rc == vrSuccess && dlogits ? rowGrads<decltype(t)>(a, st) : rc;
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
