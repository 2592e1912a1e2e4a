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
  uint32_t keys[20];           // of the ten rounds, without it
  uint64_t offset;
  uint64_t slots;  // packs that a row can touch; units
  uint64_t head;   // elements before the first unit
  uint32_t least;  // upper halves from here on are kept
  uint32_t below;  // least << 16, less one
  uint32_t tie;    // the one that leaves it to the lower half; above 65535: none does
  uint32_t lower;  // which is kept from here on
  uint32_t ties;   // the tying half twice
  uint32_t c65536, one;  // constants that keep products products
  float scale;
  bool xAlike, rAlike;  // x's and the residual's rows lie as y's modulo 16 bytes
};


constexpr int kThreads = 256;
constexpr uint64_t kBlocks = (1ull << 61) - 1;  // numbers wrap at 2^64

// The keys of the rounds: from the host, constants of the launch that the instructions
// take as they are, or with a seed on the device from that one (18 additions a block).
template <bool DEVICE>
struct Keys {
  uint32_t k0, k1;
  __device__ __forceinline__ Keys(const DropArgs& a) {
    if (DEVICE) k0 = (uint32_t)*a.seedDevice, k1 = (uint32_t)(*a.seedDevice >> 32);
  }
  __device__ __forceinline__ uint32_t first(const DropArgs& a, int r) const {
    return DEVICE ? k0 + r * 0x9E3779B9u : a.keys[2 * r];
  }
  __device__ __forceinline__ uint32_t second(const DropArgs& a, int r) const {
    return DEVICE ? k1 + r * 0xBB67AE85u : a.keys[2 * r + 1];
  }
};

// The block of counter (n, stream).
template <bool DEVICE>
__device__ __forceinline__ void philox(const DropArgs& a, const Keys<DEVICE>& keys, uint64_t n, uint32_t stream,
                                       uint32_t* w) {
  uint32_t c0 = (uint32_t)n, c1 = (uint32_t)(n >> 32), c2 = stream, c3 = 0;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p = (uint64_t)0xD2511F53u * c0, q = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ keys.first(a, r);
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ keys.second(a, r);
    c3 = (uint32_t)p;
  }
  w[0] = c0, w[1] = c1, w[2] = c2, w[3] = c3;
}

// The halfwords of the V elements from number n on, two in a word.
template <int V, bool DEVICE>
__device__ __forceinline__ void halfwords(const DropArgs& a, const Keys<DEVICE>& keys, uint64_t n,
                                          uint32_t stream, uint32_t (&h)[V / 2]) {
  uint32_t w[8];
  const uint32_t first = (uint32_t)n & 7;
  philox(a, keys, n >> 3, stream, w);
  w[4] = w[5] = w[6] = w[7] = 0;
  if (first + V > 8) philox(a, keys, ((n >> 3) + 1) & kBlocks, stream, w + 4);
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
template <int V, bool DEVICE>
__device__ __forceinline__ uint32_t kept(const DropArgs& a, const Keys<DEVICE>& keys, uint64_t n) {
  uint32_t h[V / 2], keep = 0, ties = 0;
  halfwords<V>(a, keys, n, 0, h);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const uint32_t u = i & 1 ? h[i / 2] >> 16 : h[i / 2] & 0xffff;
    keep |= (u >= a.least ? 1u : 0u) << i;
    ties |= (u == a.tie ? 1u : 0u) << i;
  }
  if (ties) {
    halfwords<V>(a, keys, n, 1, h);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t u = i & 1 ? h[i / 2] >> 16 : h[i / 2] & 0xffff;
      keep |= (u >= a.lower ? ties : 0u) & (1u << i);
    }
  }
  return keep;
}

// An element that is kept: one rounding in 32 bits, wherever it lies.
template <bool ADD>
__device__ __forceinline__ float apply(float x, float scale, float add) {
  return ADD ? __fmaf_rn(x, scale, add) : __fmul_rn(x, scale);
}

// One element's fate.
template <bool DEVICE>
__device__ __forceinline__ bool keeps(const DropArgs& a, const Keys<DEVICE>& keys, uint64_t n) {
  uint32_t w[4];
  const auto half = [&](uint32_t stream) {
    philox(a, keys, n >> 3, stream, w);
    const uint32_t v = n & 4 ? (n & 2 ? w[3] : w[2]) : (n & 2 ? w[1] : w[0]);
    return n & 1 ? v >> 16 : v & 0xffff;
  };
  const uint32_t u = half(0);
  return u == a.tie ? half(1) >= a.lower : u >= a.least;
}

// The four words of a unit that starts FW words and `first` mod 2 halfwords behind the start
// of this lane's block, from that and the next lane's.
template <int FW>
__device__ __forceinline__ void shifted(const uint32_t (&now)[4], const uint32_t (&next)[4], uint32_t first,
                                        uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31;
  uint32_t all[5];
#pragma unroll
  for (int i = 0; i < 5; ++i)
    all[i] = i + FW < 4 ? now[(i + FW) & 3]
                        : __shfl_sync(~0u, lane == 0 ? next[(i + FW) & 3] : now[(i + FW) & 3], (lane + 1) & 31);
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(all[i], all[i + 1], (first & 1) * 16);
}

// A pack's elements. The kernel's time is that of the pipe that compares, selects and
// shifts: what can be a product here is one.
template <typename T>
__device__ __forceinline__ void floats(const uint4& v, uint32_t c65536, float (&e)[kV<T>]) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = __uint_as_float(w[i] * c65536);
      e[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    F2 f[kV<T> / 2];
    unpack<T>(v, f);
#pragma unroll
    for (int i = 0; i < kV<T> / 2; ++i) split(f[i], e[2 * i], e[2 * i + 1]);
  }
}

// h > below ? x scale + add : add. Not a product with 0: x may be infinite.
template <bool ADD>
__device__ __forceinline__ float if_above(uint32_t h, uint32_t below, float x, float scale, float add) {
  float y = add;
  if (ADD)
    asm("{\n.reg .pred p;\nsetp.gt.u32 p, %1, %2;\n@p fma.rn.f32 %0, %3, %4, %0;\n}"
        : "+f"(y) : "r"(h), "r"(below), "f"(x), "f"(scale));
  else
    asm("{\n.reg .pred p;\nsetp.gt.u32 p, %1, %2;\n@p mul.rn.f32 %0, %3, %4;\n}"
        : "+f"(y) : "r"(h), "r"(below), "f"(x), "f"(scale));
  return y;
}

// Tensors without gaps that lie alike: a warp takes U x 32 units of 8 elements, a lane
// every 32nd. Where the units' numbers start at a multiple of 8, a unit's randomness is one
// block of the generator; else (SHIFTED) parts of two, and a lane takes the second from
// the next lane, so that U + 1 blocks serve U units. Two bounds lie close together: HBM,
// and the pipe of comparisons, shifts and logic, half of whose work is the generator's exclusive
// ors. Of the measured copy peak, on 16384 x 8192: bf16 with an addition 1.06 (113 us), at
// odd numbers 1.00; alone 0.89 (89 us), at odd numbers 0.77 (104 us; with both blocks made
// in each lane 0.58); float32 alone 1.02. With 32 random bits an element, two blocks for 8, 107
// us alone; keys added up in the kernel 94. At odd numbers, 39892 x 2051 float16 (60 us, 0.81; at
// even ones 53), that pipe is busy for 62 % of the cycles and an instruction issued in 66 % of them:
// 154 a warp and unit, from 22 warps on an SM. 9973 x 2051 is 17 us (0.69), of which
// by both sizes 3 do not grow with the elements.
template <typename T, int U, bool ADD, bool SHIFTED, bool DEVICE>
__global__ void __launch_bounds__(kThreads, 3) vrDropFlat(const __grid_constant__ DropArgs a) {
  constexpr int N = 8 * (int)sizeof(T) / 16;  // packs of a unit
  constexpr int V = kV<T>;
  begin_kernel();
  const Keys<DEVICE> keys(a);
  const int lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.residual);
  T* y = static_cast<T*>(a.y);
  if (blockIdx.x == 0 && threadIdx.x < 16) {  // what lies before the first unit and after the last
    const uint64_t i = threadIdx.x < 8 ? threadIdx.x : a.head + 8 * a.slots + (threadIdx.x - 8);
    if (threadIdx.x < 8 ? i < a.head : i < a.cols) {
      const float add = ADD ? to_f32(r[i]) : 0.f;
      y[i] = from_f32<T>(keeps(a, keys, a.offset + i) ? apply<ADD>(to_f32(x[i]), a.scale, add) : add);
    }
  }
  const uint64_t unit0 = ((uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5)) * (U * 32) + lane;
  x += a.head + unit0 * 8;
  y += a.head + unit0 * 8;
  if (ADD) r += a.head + unit0 * 8;
  uint4 vx[U][N], vr[U][N];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (unit0 + u * 32 < a.slots) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        vx[u][k] = reinterpret_cast<const uint4*>(x + u * 256)[k];
        if (ADD) vr[u][k] = reinterpret_cast<const uint4*>(r + u * 256)[k];
      }
    }
  const uint64_t n0 = a.offset + a.head + unit0 * 8;
  const uint32_t first = SHIFTED ? (uint32_t)n0 & 7 : 0;  // the same in all threads
  uint32_t now[4], next[4];
  if (SHIFTED) philox(a, keys, n0 >> 3, 0, now);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint32_t w[4];
    if (SHIFTED) {
      philox(a, keys, ((n0 >> 3) + (u + 1) * 32) & kBlocks, 0, next);
      switch (first >> 1) {
        case 0: shifted<0>(now, next, first, w); break;
        case 1: shifted<1>(now, next, first, w); break;
        case 2: shifted<2>(now, next, first, w); break;
        default: shifted<3>(now, next, first, w);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) now[i] = next[i];
    } else {
      philox(a, keys, ((n0 >> 3) + u * 32) & kBlocks, 0, w);
    }
    // Upper halves are compared where they stand in a word, or multiplied there; ties are
    // halfwords that are 0 after an exclusive or.
    uint32_t h[8], below = a.below, ties = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[2 * i] = w[i] * a.c65536;
      h[2 * i + 1] = w[i];
      const uint32_t z = w[i] ^ a.ties;
      ties |= (z * a.one + 0xfffeffffu) & ~z;
    }
    if (((ties & 0x80008000u) && a.lower) || a.least == 0) {  // one unit of 8192; or p == 0
      below = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) h[i] = a.least == 0 || keeps(a, keys, n0 + u * 256 + i);
    }
    if (unit0 + u * 32 < a.slots) {
#pragma unroll
      for (int k = 0; k < N; ++k) {
        F2 f[V / 2];
        float e[V], add[V];
        floats<T>(vx[u][k], a.c65536, e);
        if (ADD) floats<T>(vr[u][k], a.c65536, add);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = if_above<ADD>(h[k * V + i], below, e[i], a.scale, ADD ? add[i] : 0.f);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) f[i] = f2(e[2 * i], e[2 * i + 1]);
        reinterpret_cast<uint4*>(y + u * 256)[k] = pack<T>(f);
      }
    }
  }
}

// Rows with other elements between them, or tensors that do not lie alike: a thread takes U
// packs of y, cut at memory's 16-byte boundaries; a row's first and last may be parts. Bound by its
// instructions: whatever a number starts at, a pack makes its own blocks of the generator and finds
// its row by a division. 16384 x 8192 bf16 with rows 8200 apart 150 us (0.53 of the measured copy
// peak), at odd numbers 200, with an addition 165 (0.72); from one element off 16 bytes, read in
// single elements, 163, 196, 227; float32 279, 332, 299 and 239, 289, 285.
template <typename T, int U, bool ADD, bool DEVICE>
__global__ void __launch_bounds__(kThreads) vrDropKernel(const __grid_constant__ DropArgs a) {
  constexpr int V = kV<T>;
  begin_kernel();
  const Keys<DEVICE> keys(a);
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
    const uint32_t keep = kept<V>(a, keys, n[u]);
    if (whole[u]) {
      F2 f[V / 2];
      float e[V], add[V];
      floats<T>(vx[u], a.c65536, e);
      if (ADD) floats<T>(vr[u], a.c65536, add);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float r = ADD ? add[i] : 0.f;
        e[i] = keep >> i & 1 ? apply<ADD>(e[i], a.scale, r) : r;
      }
#pragma unroll
      for (int i = 0; i < V / 2; ++i) f[i] = f2(e[2 * i], e[2 * i + 1]);
      *reinterpret_cast<uint4*>(y[u]) = pack<T>(f);
    } else {
      for (int i = 0; i < V; ++i) {
        if (col[u] + i < 0 || col[u] + i >= (int64_t)a.cols) continue;
        const float add = ADD ? to_f32(r[u][i]) : 0.f;
        y[u][i] = from_f32<T>(keep >> i & 1 ? apply<ADD>(to_f32(x[u][i]), a.scale, add) : add);
      }
    }
  }
}

template <typename T, bool ADD, bool DEVICE>
vrResult_t run(DropArgs& a, cudaStream_t st) {
  constexpr uint64_t V = kV<T>;
  // As one row where nothing lies between rows.
  if (a.xStride == a.cols && a.yStride == a.cols && (!ADD || a.rStride == a.cols)) {
    a.cols *= a.rows;
    a.rows = 1;
  }
  const auto alike = [&](const void* p, uint64_t stride) {
    return (((uintptr_t)p - (uintptr_t)a.y) & 15) == 0 &&
           (a.rows == 1 || (((stride - a.yStride) * sizeof(T)) & 15) == 0);
  };
  a.xAlike = alike(a.x, a.xStride);
  a.rAlike = ADD && alike(a.residual, a.rStride);
  const void* k;
  uint64_t blocks;
  if (a.rows == 1 && a.xAlike && (!ADD || a.rAlike)) {
    a.head = ((16 - ((uintptr_t)a.x & 15)) & 15) / sizeof(T);
    if (a.head > a.cols) a.head = a.cols;
    a.slots = (a.cols - a.head) / 8;
    const bool shifted = (a.offset + a.head) % 8 != 0;
    // 64 bytes of x a thread, all loaded before the first is computed, where they fill the GPU
    // at least twice (96 where a block of the generator more is to be spread over them; with an
    // addition they are too many registers); else one unit, on more SMs.
    constexpr int U = 64 / (8 * (int)sizeof(T)), SU = ADD ? U : U * 3 / 2;
    const bool many = a.slots >= (uint64_t)kSMs * 8 * kThreads * 2;
    const uint64_t each = (many ? (shifted ? SU : U) : 1) * kThreads;
    blocks = (a.slots + each - 1) / each;
    if (!blocks) blocks = 1;
    k = many ? (shifted ? (const void*)&vrDropFlat<T, SU, ADD, true, DEVICE>
                        : (const void*)&vrDropFlat<T, U, ADD, false, DEVICE>)
             : (shifted ? (const void*)&vrDropFlat<T, 1, ADD, true, DEVICE>
                        : (const void*)&vrDropFlat<T, 1, ADD, false, DEVICE>);
  } else {
    a.slots = (a.cols + 2 * (V - 1)) / V;
    blocks = (a.rows * a.slots + 2 * kThreads - 1) / (2 * kThreads);
    k = (const void*)&vrDropKernel<T, 2, ADD, DEVICE>;
  }
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
  const uint32_t least = lower ? upper + 1 : upper;
  DropArgs a = {x, residual, y, rows, cols, xStride, residualStride, yStride, seedDevice, {}, offset,
                0, 0, least, (least << 16) - 1, lower ? upper : ~0u, lower,
                upper << 16 | (upper & 0xffff), 65536, 1,
                p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f, false, false};
  for (int i = 0; i < 20; ++i)
    a.keys[i] = (uint32_t)(i % 2 ? seed >> 32 : seed) + (uint32_t)(i / 2) * (i % 2 ? 0xBB67AE85u : 0x9E3779B9u);
  cudaStream_t st = (cudaStream_t)stream;
  const auto pick = [&](auto t) {
    using T = decltype(t);
    if (seedDevice) return residual ? run<T, true, true>(a, st) : run<T, false, true>(a, st);
    return residual ? run<T, true, false>(a, st) : run<T, false, false>(a, st);
  };
  if (dtype == vrFloat32) return pick(float{});
  return dtype == vrFloat16 ? pick(__half{}) : pick(__nv_bfloat16{});
}
