// vr_dropout.cu -- dropout by a counter-based generator: the mask is a function of
// the seed and of each element's number, so it is never stored.
//
//   y = residual + (u(n) >= p 2^32 ? x / (1 - p) : 0)
//
// u(n), 32 bits, comes from Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): its upper half is halfword n mod 8 of
// the block of counter (n div 8, 0), its lower half the same of counter (n div 8, 1).
// The lower half decides only where the upper one equals the threshold's, for one
// element in 65536: nearly always one block serves 8 elements, and p still holds to
// 2^-33. The backward pass is the same call on dy.
#include <math.h>

#include "vr_packs.cuh"

namespace {

using namespace vrop;

struct DropArgs {
  const void* x;
  const void* residual;
  void* y;
  uint64_t rows, cols, xStride, rStride, yStride;
  const uint64_t* seedDevice;  // the seed where it is not NULL
  uint64_t seed, offset;
  uint64_t slots;  // packs that a row can touch
  uint32_t least;  // upper halves from here on are kept
  uint32_t tie;    // the one that leaves it to the lower half; above 65535: none does
  uint32_t lower;  // which is kept from here on
  float scale;
  bool xAlike, rAlike;  // x's and the residual's rows lie as y's modulo 16 bytes
};

constexpr int kThreads = 256;
constexpr uint64_t kBlocks = (1ull << 61) - 1;  // numbers wrap at 2^64

// The block of counter (n, stream) under `seed`.
__device__ __forceinline__ void philox(uint64_t n, uint32_t stream, uint64_t seed, uint32_t* w) {
  uint32_t c0 = (uint32_t)n, c1 = (uint32_t)(n >> 32), c2 = stream, c3 = 0;
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// The halfwords of the V elements from number n on, two in a word.
template <int V>
__device__ __forceinline__ void halfwords(uint64_t n, uint32_t stream, uint64_t seed,
                                          uint32_t (&h)[V / 2]) {
  uint32_t w[8];
  const uint32_t first = (uint32_t)n & 7;
  philox(n >> 3, stream, seed, w);
  w[4] = w[5] = w[6] = w[7] = 0;
  if (first + V > 8) philox(((n >> 3) + 1) & kBlocks, stream, seed, w + 4);
  if (first) {
#pragma unroll
    for (int i = 0; i < 7; ++i) w[i] = first & 2 ? w[i + 1] : w[i];
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = first & 4 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = first & 1 ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
  }
#pragma unroll
  for (int i = 0; i < V / 2; ++i) h[i] = w[i];
}

// Which of the V elements from number n on stay: a bit for each.
template <int V>
__device__ __forceinline__ uint32_t kept(const DropArgs& a, uint64_t n, uint64_t seed) {
  uint32_t h[V / 2], keep = 0, ties = 0;
  halfwords<V>(n, 0, seed, h);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t u = i & 1 ? h[i / 2] >> 16 : h[i / 2] & 0xffff;
    keep |= (u >= a.least ? 1u : 0u) << i;
    ties |= (u == a.tie ? 1u : 0u) << i;
  }
  if (ties) {
    halfwords<V>(n, 1, seed, h);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = i & 1 ? h[i / 2] >> 16 : h[i / 2] & 0xffff;
      keep |= (u >= a.lower ? ties : 0u) & (1u << i);
    }
  }
  return keep;
}

// A thread takes U packs of y, cut at memory's 16-byte boundaries; a row's first and
// last may be parts. Bound by HBM: 2 or 3 tensors, and about 90 instructions for 32 or
// 48 bytes of them.
template <typename T, int U, bool ADD>
__global__ void __launch_bounds__(kThreads) vrDropKernel(const __grid_constant__ DropArgs a) {
  constexpr int V = kV<T>;
  begin_kernel();
  const uint64_t seed = a.seedDevice ? *a.seedDevice : a.seed;
  const uint64_t first = (uint64_t)blockIdx.x * (kThreads * U) + threadIdx.x;
  const uint64_t all = a.rows * a.slots;
  const T* x[U];
  const T* r[U];
  T* y[U];
  int64_t col[U];  // of the pack's first element, negative where the row starts inside it
  uint64_t n[U];
  uint4 vx[U], vr[U];
  bool some[U], whole[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint64_t slot = first + u * kThreads;
    some[u] = whole[u] = false;
    if (slot >= all) continue;
    uint64_t row = 0, j = slot;
    if (a.rows > 1) {
      row = all >> 32 ? slot / a.slots : (uint32_t)slot / (uint32_t)a.slots;
      j = slot - row * a.slots;
    }
    T* y0 = static_cast<T*>(a.y) + row * a.yStride;
    col[u] = (int64_t)(j * V) - (int64_t)(((uintptr_t)y0 & 15) / sizeof(T));
    y[u] = y0 + col[u];
    x[u] = static_cast<const T*>(a.x) + row * a.xStride + col[u];
    if (ADD) r[u] = static_cast<const T*>(a.residual) + row * a.rStride + col[u];
    n[u] = a.offset + row * a.cols + (uint64_t)col[u];
    some[u] = col[u] < (int64_t)a.cols;
    whole[u] = col[u] >= 0 && col[u] + V <= (int64_t)a.cols;
    auto load = [&](const T* p, bool alike) {
      if (alike) return *reinterpret_cast<const uint4*>(p);
      T e[V];
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = p[i];
      uint4 v;
      memcpy(&v, e, 16);
      return v;
    };
    if (whole[u]) {
      vx[u] = load(x[u], a.xAlike);
      if (ADD) vr[u] = load(r[u], a.rAlike);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (!some[u]) continue;
    const uint32_t keep = kept<V>(a, n[u], seed);
    if (whole[u]) {
      F2 f[V / 2], add[V / 2];
      unpack<T>(vx[u], f);
      if (ADD) unpack<T>(vr[u], add);
#pragma unroll
      for (int i = 0; i < V / 2; ++i) {
        float p, q;
        split(f[i] * f2(a.scale), p, q);  // selected, not multiplied by 0: x may be infinite
        f[i] = f2(keep >> (2 * i) & 1 ? p : 0.f, keep >> (2 * i + 1) & 1 ? q : 0.f);
        if (ADD) f[i] = f[i] + add[i];
      }
      *reinterpret_cast<uint4*>(y[u]) = pack<T>(f);
    } else {
      for (int i = 0; i < V; ++i) {
        if (col[u] + i < 0 || col[u] + i >= (int64_t)a.cols) continue;
        // two roundings, as in whole packs: no element depends on how its row lies
        float f = keep >> i & 1 ? __fmul_rn(to_f32(x[u][i]), a.scale) : 0.f;
        if (ADD) f = __fadd_rn(f, to_f32(r[u][i]));
        y[u][i] = from_f32<T>(f);
      }
    }
  }
}

template <typename T, bool ADD>
vrResult_t run(DropArgs& a, cudaStream_t st) {
  constexpr uint64_t V = kV<T>;
  // As one row where nothing lies between rows.
  if (a.xStride == a.cols && a.yStride == a.cols && (!ADD || a.rStride == a.cols)) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  a.slots = (a.cols + 2 * (V - 1)) / V;
  const auto alike = [&](const void* p, uint64_t stride) {
    return (((uintptr_t)p - (uintptr_t)a.y) & 15) == 0 &&
           (a.rows == 1 || (((stride - a.yStride) * sizeof(T)) & 15) == 0);
  };
  a.xAlike = alike(a.x, a.xStride);
  a.rAlike = ADD && alike(a.residual, a.rStride);
  const uint64_t slots = a.rows * a.slots;
  // Four packs a thread, all loaded before the first is computed, where they fill the
  // GPU at least twice; else one, on more SMs.
  const bool many = slots >= (uint64_t)kSMs * 8 * kThreads * 2;
  const uint64_t each = many ? 4 * kThreads : kThreads;
  const void* k = many ? (const void*)&vrDropKernel<T, 4, ADD> : (const void*)&vrDropKernel<T, 1, ADD>;
  const uint64_t blocks = (slots + each - 1) / each;
  if (blocks > 0x7fffffffu) return vrInvalidArgument;
  return launch(k, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
}

}  // namespace

extern "C" VR_API vrResult_t vrDropout(const void* x, const void* residual, void* y, size_t rows,
                                       size_t cols, size_t xStride, size_t residualStride,
                                       size_t yStride, double p, uint64_t seed,
                                       const uint64_t* seedDevice, uint64_t offset,
                                       vrDataType_t dtype, void* stream) {
  NvtxRange range("vrDropout");
  const int es = elemSizeOf(dtype);
  if (!(es == 2 || es == 4) || !(p >= 0.0) || !(p <= 1.0)) return vrInvalidArgument;
  if (rows == 0 || cols == 0) return vrSuccess;
  constexpr uint64_t kMost = 1ull << 48;  // elements from the first to the last: addresses stay in 64 bits
  if (cols > kMost || rows > kMost / cols) return vrInvalidArgument;
  const auto bad = [&](const void* t, size_t stride) {
    return !t || misaligned(t, es) || stride < cols || stride > kMost / rows;
  };
  if (bad(x, xStride) || bad(y, yStride) || (residual && bad(residual, residualStride)) ||
      misaligned(seedDevice, 8))
    return vrInvalidArgument;
  const bool overX = x == y && xStride == yStride, overR = residual == y && residualStride == yStride;
  const Bytes outs[] = {bytesOf(y, rows, cols, yStride, es)};
  const Bytes ins[] = {bytesOf(overX ? nullptr : x, rows, cols, xStride, es),
                       bytesOf(overR ? nullptr : residual, rows, cols, residualStride, es),
                       bytesOf(seedDevice, 8)};
  if (anyOverlap(outs, 1, ins, 3)) return vrInvalidArgument;
  // round(p 2^32), its upper half and its lower
  const uint64_t threshold = (uint64_t)llrint(p * 4294967296.0);
  const uint32_t upper = (uint32_t)(threshold >> 16), lower = (uint32_t)threshold & 0xffff;
  DropArgs a = {x, residual, y, rows, cols, xStride, residualStride, yStride, seedDevice, seed, offset,
                0, lower ? upper + 1 : upper, lower ? upper : ~0u, lower,
                p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f, false, false};
  cudaStream_t st = (cudaStream_t)stream;
  const auto pick = [&](auto t) {
    using T = decltype(t);
    return residual ? run<T, true>(a, st) : run<T, false>(a, st);
  };
  if (dtype == vrFloat32) return pick(float{});
  return dtype == vrFloat16 ? pick(__half{}) : pick(__nv_bfloat16{});
}
