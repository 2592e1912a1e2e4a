// vr_gradnorm.cu -- the norm of a list of gradients, and clipping by it.
//
//   N = |s| sqrt(sum_t sum_i g_ti^2),  out = g s min(1, max / N)
//
// for tensors of any sizes, types and alignments. A list is cut into tiles, and
// the tiles into units of consecutive ones: unit u of U takes the tiles [nt u / U,
// nt (u + 1) / U), which may lie in several tensors, and leaves one partial sum
// for each tensor it meets, in slot u + t: along a unit t grows, from one unit
// to the next u does, so every slot has one writer and the sums have one order
// (no atomics: equal inputs give equal bits). A second kernel adds the slots up.
// Lists of up to 1 MiB are one launch of one cluster, whose slots lie in
// shared memory.
//
// All of it is bound by HBM (2 or 3 flop an element). The norm reads every
// element once. Clipping reads it again, as the factor needs all of them, and
// writes it; lists of some 25 MB are still in L2 then, of 197 MB nothing is.
// Measured on a GB300: the norms of 0.94 GB of bf16 in 288 tensors 138 us (1.01
// of the measured copy peak: reads alone are a little faster than copies);
// clipping 1.06 GB of float32 498 us and 1.15 GB of mixed odd-sized tensors 544
// us, 0.94 of what two reads and a write take at that peak.
#include <algorithm>
#include <memory>
#include <new>

#include "vr_ln_rows.cuh"

namespace {

using namespace vrop;
using vrln::cluster_rank;
using vrln::cluster_sync;
using vrop::warp_sum;

// Who works on a unit (a block, or a warp), and the tile that it reads at a time:
// PACKS 16-byte packs a thread.
template <int THREADS, int PACKS>
struct Team {
  enum { threads = THREADS, warps = THREADS / 32, packs = PACKS, tileBytes = THREADS * PACKS * 16 };
  static __device__ __forceinline__ int id() {
    return THREADS == 32 ? threadIdx.x & 31 : threadIdx.x;
  }
};
// Long lists: 5 blocks an SM for the sums, 3 for scaling, with the registers that
// 8 loads in flight take (2 / 3 / 4 / 5 blocks: 1.06 GB 511 / 498 / 504 / 510 us,
// 25 MB 20.7 / 19.3 / 20.1 / 20.1 us; 3 in the registers of 4: 526 and 20.2).
using Block = Team<256, 8>;
constexpr int kSumBlocks = 5, kScaleBlocks = 3;
constexpr int kBlocks = kSMs * kSumBlocks;
// A unit is at least 8 tiles where a block has more than one unit. Several
// units a block keep what all blocks read at a time together in memory: 532
// us against 543 for 1.15 GB in one unit a block.
constexpr int kUnitTiles = 8, kMostWaves = 8;
// Short lists: the warps of one cluster.
using Warp = Team<32, 8>;
constexpr int kShortBlocks = 16, kShortWarps = 16, kShortUnits = kShortBlocks * kShortWarps;
constexpr int kShortTiles = kShortUnits;

// Tensors of one launch. Their table lies in the kernel's parameter space
// (32,764 bytes at most): nothing is copied to the device beforehand and the
// caller's arrays are free on return. Longer lists take several launches.
constexpr int kShortList = 64;
constexpr int kLongList = 960;  // and LongTable's table of units

template <int CAP>
struct alignas(8) Table {
  int nTensors;
  int nUnits;
  uint32_t nTiles;
  uint32_t nSlots;    // of all launches of the call
  uint32_t slotBase;  // of this launch
  int tensorBase;
  float scale;
  float maxNorm;
  uint64_t* slots;
  float* norm;
  float* tensorNorms;
  const void* in[CAP];
  void* out[CAP];
  uint64_t count[CAP];
  uint32_t tile[CAP + 1];  // tiles before tensor t
  uint8_t type[CAP];
};
// With one unit a block the host looks up the units' first tensors: a search in
// parameter space is a chain of misses in the constant cache, 4 of the 11 us of
// 25 MB (lists with more units are long enough not to notice).
template <int CAP>
struct LongTable : Table<CAP> {
  uint16_t first[kBlocks];
};

__host__ __device__ inline int sizeOfType(int t) {
  return t == vrFloat64 ? 8 : t == vrFloat32 ? 4 : 2;
}

// Elements before the first 16-byte boundary.
__host__ __device__ inline uint64_t headOf(const void* p, uint64_t count, int es) {
  const uint64_t h = ((16 - ((uintptr_t)p & 15)) & 15) / es;
  return h < count ? h : count;
}

inline uint64_t tilesOf(const void* p, uint64_t count, int es, int tileBytes) {
  if (!count) return 0;
  const uint64_t body = (count - headOf(p, count, es)) * es;
  return body ? (body + tileBytes - 1) / tileBytes : 1;
}

// The first tile of unit u, and the unit that holds tile k.
__host__ __device__ inline uint32_t divide(uint64_t a, uint32_t b) {
  return a >> 32 ? (uint32_t)(a / b) : (uint32_t)a / b;  // 64-bit division is slow
}
__host__ __device__ inline uint32_t firstTile(uint32_t nTiles, int nUnits, int u) {
  return divide((uint64_t)nTiles * u, nUnits);
}
__device__ inline uint32_t unitOf(uint32_t nTiles, int nUnits, uint32_t k) {
  return divide(((uint64_t)k + 1) * nUnits - 1, nTiles);
}

// The tensor that tile k lies in: the last t with tile[t] <= k.
template <typename A>
__device__ inline int tensorOf(const A& a, uint32_t k) {
  int lo = 0, hi = a.nTensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.tile[mid] <= k) lo = mid; else hi = mid;
  }
  return lo;
}

// The same for a launch of single units: the first tensor of unit u, and from
// there on.
template <int CAP>
__device__ inline int tensorOf(const LongTable<CAP>& a, uint32_t k) {
  if (a.nUnits > kBlocks) return tensorOf(static_cast<const Table<CAP>&>(a), k);
  int t = a.first[unitOf(a.nTiles, a.nUnits, k)];
  while (a.tile[t + 1] <= k) ++t;
  return t;
}

// A sum in two floats: hi + lo, the rounding errors of hi caught exactly
// (Knuth's two-sum), so that a long run costs no precision. This GPU works on
// 64-bit numbers at a sixty-fourth of its 32-bit rate: with them, a square root,
// a division and the sums over a block were 5 of the 10 us of a small call.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, z = s - hi;
    lo += (hi - (s - z)) + (x - z);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& b) {
    add(b.hi);
    lo += b.lo;
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};

// The sum over a warp, the same bits in every lane.
__device__ __forceinline__ Sum2 warp_sum(Sum2 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    Sum2 w;
    w.hi = __shfl_xor_sync(~0u, v.hi, o);
    w.lo = __shfl_xor_sync(~0u, v.lo, o);
    v.add(w);
  }
  // hi + lo are the same in all lanes, but lo's roundings go by the order
  v.hi = __shfl_sync(~0u, v.hi, 0);
  v.lo = __shfl_sync(~0u, v.lo, 0);
  return v;
}

// A sum of squares as a slot holds it: two floats, hi in the upper word, where it
// is zero or within [2^-90, 2^100] (the sum of all slots then fits a float), else
// a double with the sign bit set.
constexpr float kLeast = 0x1p-90f, kMost = 0x1p100f;
__device__ __forceinline__ uint64_t slotOf(const Sum2& v) {
  return (uint64_t)__float_as_uint(v.hi) << 32 | __float_as_uint(v.lo);
}
__device__ __forceinline__ uint64_t slotOf(double d) {
  return (uint64_t)__double_as_longlong(d) | 1ull << 63;
}

// Slots added up: the pairs, and the doubles apart.
struct Total {
  Sum2 pair;
  double rest = 0;
  bool wide = false;
  __device__ __forceinline__ void add(uint64_t slot) {
    if (slot >> 63) {
      wide = true;
      rest += __longlong_as_double((long long)(slot & ~(1ull << 63)));
    } else {
      Sum2 v;
      v.hi = __uint_as_float((uint32_t)(slot >> 32));
      v.lo = __uint_as_float((uint32_t)slot);
      pair.add(v);
    }
  }
  __device__ __forceinline__ double value() const { return pair.value() + rest; }
  // |scale| sqrt(sum)
  __device__ __forceinline__ float norm(float scale) const {
    if (!wide) {
      const float h = pair.hi + pair.lo, l = (pair.hi - h) + pair.lo;
      float r = sqrtf(h);
      if (r > 0.f) r += (fmaf(-r, r, h) + l) / (2.f * r);
      r *= fabsf(scale);
      if (r == 0.f ? h == 0.f || scale == 0.f : r >= 0x1p-100f && r <= 0x1p120f) return r;
    }
    return (float)wideNorm(scale);
  }
  __device__ double wideNorm(float scale) const { return fabs((double)scale) * sqrt(value()); }
};

// Sums over a team, the same in every thread. `buf` holds a block's warps + 1
// values; it may be used again after a barrier.
template <typename S>
__device__ __forceinline__ Sum2 team_sum(Sum2 v, uint64_t* buf) {
  v = warp_sum(v);
  if constexpr (S::warps > 1) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = slotOf(v);
    __syncthreads();
    if (threadIdx.x < 32) {
      Total t;
      if (threadIdx.x < S::warps) t.pair = {__uint_as_float(buf[threadIdx.x] >> 32),
                                            __uint_as_float((uint32_t)buf[threadIdx.x])};
      const Sum2 all = warp_sum(t.pair);
      if (threadIdx.x == 0) buf[S::warps] = slotOf(all);
    }
    __syncthreads();
    v.hi = __uint_as_float((uint32_t)(buf[S::warps] >> 32));
    v.lo = __uint_as_float((uint32_t)buf[S::warps]);
  }
  return v;
}
template <typename S>
__device__ double team_sum(double s, uint64_t* buf) {
  s = vrop::warp_sum(s);
  if constexpr (S::warps > 1) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = (uint64_t)__double_as_longlong(s);
    __syncthreads();
    s = 0;
    for (int i = 0; i < S::warps; ++i) s += __longlong_as_double((long long)buf[i]);
    __syncthreads();
  }
  return s;
}
template <typename S>
__device__ __forceinline__ bool team_any(bool b) {
  if constexpr (S::warps == 1) return __any_sync(~0u, b);
  else return __syncthreads_or(b);
}
template <typename S>
__device__ __forceinline__ Total team_sum(Total t, uint64_t* buf) {
  t.wide = team_any<S>(t.wide);
  t.pair = team_sum<S>(t.pair, buf);
  if (t.wide) t.rest = team_sum<S>(t.rest, buf);
  return t;
}

template <typename T>
__device__ __forceinline__ void squares(const uint4& v, float* acc, uint32_t& bits) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 2) {
      bits |= w[i] & 0x7fff7fffu;
      T e[2];
      memcpy(e, &w[i], 4);
      const float a = to_f32(e[0]), b = to_f32(e[1]);
      acc[0] = fmaf(a, a, acc[0]);
      acc[1] = fmaf(b, b, acc[1]);
    } else {
      bits |= w[i] & 0x7fffffffu;
      const float a = __uint_as_float(w[i]);
      acc[i & 1] = fmaf(a, a, acc[i & 1]);
    }
  }
}

__device__ __forceinline__ uint4 load16(const void* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// A team's sum of squares of the tiles [k0, k1) of one tensor, as a slot, the same
// in every thread.
template <typename S, typename T>
__device__ uint64_t sumTiles(const T* g, uint64_t count, uint32_t k0, uint32_t k1, uint64_t* buf) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr uint64_t E = S::tileBytes / sizeof(T);
  const uint64_t head = headOf(g, count, (int)sizeof(T)), body = count - head;
  if constexpr (sizeof(T) < 8) {
    const T* p = g + head;
    uint32_t bits = 0;
    Sum2 sum;
    for (uint32_t k = k0; k < k1; ++k) {
      const uint64_t left = body - k * E;
      const T* q = p + k * E;
      float acc[2] = {0.f, 0.f};
      if (left >= E) {
        uint4 v[S::packs];
#pragma unroll
        for (int i = 0; i < S::packs; ++i) v[i] = load16(q + (S::id() + i * S::threads) * V);
#pragma unroll
        for (int i = 0; i < S::packs; ++i) squares<T>(v[i], acc, bits);
      } else {
        const int packs = (int)(left / V);
        for (int i = S::id(); i < packs; i += S::threads)
          squares<T>(load16(q + (uint64_t)i * V), acc, bits);
        const int at = packs * V + S::id();
        if (at < (int)left) {
          const float x = to_f32(q[at]);
          acc[0] = fmaf(x, x, acc[0]);
          bits |= x != 0.f;
        }
      }
      sum.add(acc[0] + acc[1]);
    }
    if (k0 == 0 && S::id() < head) {
      const float x = to_f32(g[S::id()]);
      sum.add(x * x);
      bits |= x != 0.f;
    }
    sum = team_sum<S>(sum, buf);
    // The squares of 32-bit floats and of bfloat16 leave the range of a float
    // long before their sum leaves that of a double. Where they did (the sum
    // is infinite, or so small that squares went below the smallest float),
    // the tiles are summed again in 64 bits. float16's squares always fit.
    const bool fits = sum.hi >= kLeast && sum.hi <= kMost;
    if (std::is_same_v<T, __half> || fits || (sum.hi < kLeast && !team_any<S>(bits != 0))) {
      // hi is infinite or NaN where float16 elements are; lo, the difference of two
      // infinities, is NaN for both.
      return sum.hi <= kMost ? slotOf(sum) : slotOf((double)sum.hi);
    }
    if (S::warps > 1) __syncthreads();  // before `buf` is used again
  }
  double d = 0;
  const uint64_t from = k0 ? head + k0 * E : 0, end = head + k1 * E, to = end < count ? end : count;
  for (uint64_t i = from + S::id(); i < to; i += S::threads) {
    const double x = to_f64(g[i]);
    d = fma(x, x, d);
  }
  return slotOf(team_sum<S>(d, buf));
}

template <typename S, typename A>
__device__ uint64_t sumTensor(const A& a, int t, uint32_t k0, uint32_t k1, uint64_t* buf) {
  if (k0 >= k1) return 0;
  const void* g = a.in[t];
  const uint64_t n = a.count[t];
  switch (a.type[t]) {
    case vrFloat16: return sumTiles<S>((const __half*)g, n, k0, k1, buf);
    case vrBfloat16: return sumTiles<S>((const __nv_bfloat16*)g, n, k0, k1, buf);
    case vrFloat32: return sumTiles<S>((const float*)g, n, k0, k1, buf);
    default: return sumTiles<S>((const double*)g, n, k0, k1, buf);
  }
}

// The partial sums of unit u: put(slot, sum) for each of its slots, u + t from
// its first tensor to the next unit's first. A tensor without a tile in the
// unit gets a zero.
template <typename S, typename A, typename Put>
__device__ __forceinline__ void sumUnit(const A& a, int u, uint64_t (*buf)[S::warps + 1], int& turn,
                                        Put put) {
  const uint32_t k0 = firstTile(a.nTiles, a.nUnits, u), k1 = firstTile(a.nTiles, a.nUnits, u + 1);
  const int t0 = u ? tensorOf(a, k0) : 0;
  const int t1 = u + 1 < a.nUnits ? tensorOf(a, k1) : a.nTensors - 1;
  for (int t = t0; t <= t1; ++t) {
    const uint32_t first = a.tile[t], last = a.tile[t + 1];
    const uint32_t x = k0 > first ? k0 : first, y = k1 < last ? k1 : last;
    const uint64_t s = sumTensor<S>(a, t, x - first, y > x ? y - first : x - first, buf[turn]);
    turn ^= 1;
    put(u + t, s);
  }
}

template <int CAP>
__global__ void __launch_bounds__(Block::threads, kSumBlocks)
    vrNormPartials(const __grid_constant__ LongTable<CAP> a) {
  __shared__ uint64_t buf[2][Block::warps + 1];
  begin_kernel();
  int turn = 0;
  for (int u = blockIdx.x; u < a.nUnits; u += gridDim.x)
    sumUnit<Block>(a, u, buf, turn, [&](int slot, uint64_t s) {
      if (threadIdx.x == 0) a.slots[a.slotBase + slot] = s;
    });
}

// The sum of n slots, the same in every thread.
template <typename S>
__device__ Total sumSlots(const uint64_t* slots, uint32_t n, uint64_t* buf) {
  constexpr int kAtOnce = 4;  // loads in flight
  Total t;
  for (uint32_t i = S::id(); i < n; i += kAtOnce * S::threads) {
    uint64_t v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) v[j] = i + j * S::threads < n ? slots[i + j * S::threads] : 0;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) t.add(v[j]);
  }
  return team_sum<S>(t, buf);
}

// Tensor t's sum of squares from the slots of one launch, in a warp.
template <typename A>
__device__ Total tensorSum(const A& a, const uint64_t* slots, int t) {
  Total s;
  if (a.tile[t] < a.tile[t + 1]) {
    const uint32_t u0 = unitOf(a.nTiles, a.nUnits, a.tile[t]);
    const uint32_t u1 = unitOf(a.nTiles, a.nUnits, a.tile[t + 1] - 1);
    for (uint32_t u = u0 + (threadIdx.x & 31); u <= u1; u += 32) s.add(slots[u + t]);
  }
  return team_sum<Warp>(s, nullptr);
}

// The norms: block 0 the whole list's (in the call's last launch), the other
// blocks' warps one tensor's each.
template <int CAP>
__global__ void __launch_bounds__(Block::threads)
    vrNormFinish(const __grid_constant__ LongTable<CAP> a) {
  __shared__ uint64_t buf[Block::warps + 1];
  begin_kernel();
  if (blockIdx.x == 0) {
    if (!a.norm) return;
    const Total s = sumSlots<Block>(a.slots, a.nSlots, buf);
    if (threadIdx.x == 0) *a.norm = s.norm(a.scale);
    return;
  }
  const int t = (blockIdx.x - 1) * Block::warps + (threadIdx.x >> 5);
  if (t >= a.nTensors) return;
  const Total s = tensorSum(a, a.slots + a.slotBase, t);
  if ((threadIdx.x & 31) == 0) a.tensorNorms[a.tensorBase + t] = s.norm(a.scale);
}

// What the gradients are multiplied by. A norm that is not finite in 64 bits (an
// element is not) clips nothing: the caller sees it and drops the step, and the
// gradients still show where it came from. One that is too large for a float alone
// is reported as infinite and clips like any other.
struct Factor {
  float norm, f;
  float after = 1.f;  // the factor is f times this power of two
  bool clips;
  __device__ Factor(const Total& s, float scale, float maxNorm) {
    norm = s.norm(scale);
    clips = norm > maxNorm;
    const float ratio = clips ? maxNorm / norm : 1.f;
    f = scale * ratio;
    // Rare: in 64 bits, also where the factor or its ratio is near the smallest normal
    // float, below which bits are lost.
    if (!(norm >= 0x1p-100f && norm <= 0x1p120f) ||
        (clips && maxNorm > 0.f && !(ratio >= 0x1p-100f && fabsf(f) >= 0x1p-100f))) {
      const double n = s.wideNorm(scale);
      clips = n > (double)maxNorm && isfinite(n);
      const double d = clips ? (double)scale * ((double)maxNorm / n) : (double)scale;
      after = clips && fabs(d) < 0x1p-100 ? 0x1p-64f : 1.f;
      f = (float)(d / (double)after);
    }
  }
  __device__ __forceinline__ float operator()(float x) const { return x * f * after; }
  // For elements of 64 bits.
  __device__ static double of(const Total& s, float scale, float maxNorm, bool clips) {
    return clips ? (double)scale * ((double)maxNorm / s.wideNorm(scale)) : (double)scale;
  }
};

// One tile of out = g * factor: 16-byte packs where g and out lie alike modulo
// 16 bytes, elements elsewhere. Each product is rounded once. `loaded`: `v` holds
// the packs of a whole tile.
template <typename S, typename T, typename F>
__device__ __forceinline__ void scaleTile(const T* g, T* out, uint64_t count, uint32_t k, F by,
                                          bool loaded, const uint4 (&v)[S::packs]) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr uint64_t E = S::tileBytes / sizeof(T);
  auto mul = [by](T x) -> T {
    if constexpr (sizeof(T) == 8) return x * by;
    else return from_f32<T>(by(to_f32(x)));
  };
  auto mulPack = [&](uint4 v) {
    T e[V];
    memcpy(e, &v, 16);
#pragma unroll
    for (int c = 0; c < V; ++c) e[c] = mul(e[c]);
    memcpy(&v, e, 16);
    return v;
  };
  const uint64_t head = headOf(g, count, (int)sizeof(T)), body = count - head;
  if (k == 0 && S::id() < head) out[S::id()] = mul(g[S::id()]);
  const uint64_t left = body - k * E;
  const int n = (int)(left < E ? left : E);
  const T* p = g + head + k * E;
  T* q = out + head + k * E;
  if (loaded) {
#pragma unroll
    for (int j = 0; j < S::packs; ++j)
      *reinterpret_cast<uint4*>(q + (S::id() + j * S::threads) * V) = mulPack(v[j]);
    return;
  }
  const int packs = ((uintptr_t)q & 15) == 0 ? n / V : 0;
  for (int i = S::id(); i < packs; i += S::threads)
    *reinterpret_cast<uint4*>(q + i * V) = mulPack(load16(p + i * V));
  for (int i = packs * V + S::id(); i < n; i += S::threads) q[i] = mul(p[i]);
}

// Tile k of the list, and its packs loaded if it is a whole one and its output
// lies like it: what can be done before the factor is known.
template <typename S>
struct Tile {
  int t;
  uint32_t k;  // in tensor t
  bool whole;
  uint4 v[S::packs];
  template <typename A>
  __device__ __forceinline__ void load(const A& a, uint32_t at) {
    t = tensorOf(a, at);
    k = at - a.tile[t];
    const char* g = static_cast<const char*>(a.in[t]);
    const int es = sizeOfType(a.type[t]);
    const uint64_t head = headOf(g, a.count[t], es) * es, bytes = a.count[t] * es;
    const uint64_t from = head + (uint64_t)k * S::tileBytes;
    whole = from + S::tileBytes <= bytes && (((uintptr_t)g - (uintptr_t)a.out[t]) & 15) == 0;
    if (whole) {
#pragma unroll
      for (int j = 0; j < S::packs; ++j) v[j] = load16(g + from + (S::id() + j * S::threads) * 16);
    }
  }
};

template <typename S, typename A>
__device__ __forceinline__ void scale(const A& a, const Tile<S>& at, const Factor& by,
                                      const Total& s) {
  const void* g = a.in[at.t];
  void* o = a.out[at.t];
  const uint64_t n = a.count[at.t];
  switch (a.type[at.t]) {
    case vrFloat16: return scaleTile<S>((const __half*)g, (__half*)o, n, at.k, by, at.whole, at.v);
    case vrBfloat16:
      return scaleTile<S>((const __nv_bfloat16*)g, (__nv_bfloat16*)o, n, at.k, by, at.whole, at.v);
    case vrFloat32: return scaleTile<S>((const float*)g, (float*)o, n, at.k, by, at.whole, at.v);
    default:
      return scaleTile<S>((const double*)g, (double*)o, n, at.k,
                          Factor::of(s, a.scale, a.maxNorm, by.clips), at.whole, at.v);
  }
}

// Every block adds the slots up for itself, while its first tile is on its way,
// then takes tiles in turn, from the list's end to its start, so that a list
// that fits L2 is found there.
template <int CAP>
__global__ void __launch_bounds__(Block::threads, kScaleBlocks)
    vrClip(const __grid_constant__ LongTable<CAP> a) {
  __shared__ uint64_t buf[Block::warps + 1];
  begin_kernel();
  Tile<Block> tile;
  if (blockIdx.x < a.nTiles) tile.load(a, a.nTiles - 1 - blockIdx.x);
  const Total s = sumSlots<Block>(a.slots, a.nSlots, buf);
  const Factor by(s, a.scale, a.maxNorm);
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = by.norm;
  for (uint32_t i = blockIdx.x; i < a.nTiles; i += gridDim.x) {
    if (i != blockIdx.x) tile.load(a, a.nTiles - 1 - i);
    scale(a, tile, by, s);
  }
}

// A short list in one launch: a unit for each warp of a cluster, the slots in every
// block's shared memory. Where `out` is there, each warp scales its unit. The
// table is copied to shared memory first, as lookups of single parameters would
// each wait for the constant cache.
__global__ void __launch_bounds__(32 * kShortWarps, 1)
    vrShortList(const __grid_constant__ Table<kShortList> p) {
  __shared__ Table<kShortList> a;
  __shared__ uint64_t slots[kShortUnits + kShortList];
  __shared__ uint64_t total[kShortWarps + 1];
  uint64_t none[2][2];
  begin_kernel();
  const int threads = 32 * kShortWarps;
  for (int i = threadIdx.x; i < (int)(sizeof(p) / 8); i += threads)
    reinterpret_cast<uint64_t*>(&a)[i] = reinterpret_cast<const uint64_t*>(&p)[i];
  cluster_sync();  // the table, and every block's slots, are there
  const int u = (int)cluster_rank() * kShortWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  int turn = 0;
  sumUnit<Warp>(a, u, none, turn, [&](int slot, uint64_t s) {
    if (lane * kShortWarps < a.nUnits) {
      uint32_t at;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                   : "=r"(at) : "r"((uint32_t)__cvta_generic_to_shared(&slots[slot])), "r"(lane));
      asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(at), "l"(s) : "memory");
    }
  });
  cluster_sync();
  const Total s =
      sumSlots<Team<32 * kShortWarps, 1>>(slots, a.nUnits + a.nTensors - 1, total);
  const Factor by(s, a.scale, a.maxNorm);
  if (cluster_rank() == 0) {
    if (a.norm && threadIdx.x == 0) *a.norm = by.norm;
    if (a.tensorNorms)
      for (int t = threadIdx.x >> 5; t < a.nTensors; t += kShortWarps) {
        const Total one = tensorSum(a, slots, t);
        if (lane == 0) a.tensorNorms[t] = one.norm(a.scale);
      }
  }
  if (a.maxNorm < 0.f) return;  // the norm alone
  const uint32_t k1 = firstTile(a.nTiles, a.nUnits, u + 1);
  for (uint32_t k = firstTile(a.nTiles, a.nUnits, u); k < k1; ++k) {
    Tile<Warp> tile;
    tile.load(a, k);
    scale(a, tile, by, s);
  }
}

// ------------------------------------------------------------------ host
struct Call {
  const void* const* in;
  void* const* out;  // NULL: the norm alone
  const size_t* counts;
  const vrDataType_t* types;
  int nTensors;
  float scale, maxNorm;
  float* norm;
  float* tensorNorms;
  uint64_t* slots;
  cudaStream_t stream;
};

// Slots of a launch of T tensors in U units: u + t runs from 0 to (U - 1) + (T - 1).
uint64_t slotsBound(int nTensors) {
  const uint64_t launches = ((uint64_t)nTensors + kLongList - 1) / kLongList;
  return launches * (uint64_t)(kBlocks * kMostWaves) + (uint64_t)nTensors;
}

template <int CAP>
void fill(const Call& c, int at, int n, int tileBytes, Table<CAP>* a) {
  uint64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    const int t = at + i;
    a->in[i] = c.in[t];
    a->out[i] = c.out ? c.out[t] : nullptr;
    a->count[i] = c.counts[t];
    a->type[i] = (uint8_t)c.types[t];
    a->tile[i] = (uint32_t)tiles;
    tiles += tilesOf(c.in[t], c.counts[t], sizeOfType(c.types[t]), tileBytes);
  }
  a->tile[n] = (uint32_t)tiles;
  a->nTensors = n;
  a->nTiles = (uint32_t)tiles;
  a->tensorBase = at;
  a->scale = c.scale;
  a->maxNorm = c.out ? c.maxNorm : -1.f;
  a->slots = c.slots;
  a->norm = c.norm;
  a->tensorNorms = c.tensorNorms;
}

// Units of a long list's launch: one a block, or whole waves of them.
int unitsFor(uint32_t tiles) {
  if (tiles <= (uint32_t)kBlocks) return tiles ? (int)tiles : 1;
  const uint32_t waves = tiles / (uint32_t)(kBlocks * kUnitTiles);
  return kBlocks * (int)(waves < 1 ? 1 : waves > kMostWaves ? kMostWaves : waves);
}

// At most a tile for each warp of the cluster: a launch costs the host 3 us, the
// cluster's two barriers the GPU 2 (1 MiB of gradients clipped in 10.6 us, by the
// long path in 6.7).
bool isShort(const Call& c) {
  if (c.nTensors > kShortList) return false;
  uint64_t tiles = 0;
  for (int t = 0; t < c.nTensors; ++t)
    tiles += tilesOf(c.in[t], c.counts[t], sizeOfType(c.types[t]), Warp::tileBytes);
  return tiles <= kShortTiles;
}

vrResult_t runShort(const Call& c) {
  Table<kShortList> a;
  memset(&a, 0, sizeof(a));
  fill(c, 0, c.nTensors, Warp::tileBytes, &a);
  int blocks = 1;
  while (blocks < kShortBlocks && (uint32_t)(blocks * kShortWarps) < a.nTiles) blocks *= 2;
  a.nUnits = blocks * kShortWarps;
  const void* k = (const void*)&vrShortList;
  if (!vrln::allowLargeClusters(k)) return vrCudaError;
  return launch(k, dim3(blocks), dim3(32 * kShortWarps), 0, c.stream, a, blocks);
}

// The first tensor of each unit, where a block has one unit.
template <int CAP>
void findFirst(LongTable<CAP>* a) {
  if (a->nUnits > kBlocks) return;
  int t = 0;
  for (int u = 0; u < a->nUnits; ++u) {
    const uint32_t k = firstTile(a->nTiles, a->nUnits, u);
    while (t + 1 < a->nTensors && a->tile[t + 1] <= k) ++t;
    a->first[u] = (uint16_t)t;
  }
}

template <int CAP>
vrResult_t runLong(const Call& c) {
  LongTable<CAP> a;
  const int launches = (c.nTensors + CAP - 1) / CAP;
  uint32_t slots = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t base = 0;
    for (int l = 0; l < launches; ++l) {
      const int at = l * CAP, n = c.nTensors - at < CAP ? c.nTensors - at : CAP;
      if (pass == 0 || launches > 1) {
        fill(c, at, n, Block::tileBytes, static_cast<Table<CAP>*>(&a));
        a.nUnits = unitsFor(a.nTiles);
        findFirst(&a);
      }
      a.slotBase = base;
      a.nSlots = slots;
      base += (uint32_t)(a.nUnits + n - 1);
      const void* kernel;
      int blocks;
      if (pass == 0) {
        kernel = (const void*)&vrNormPartials<CAP>;
        blocks = a.nUnits < kBlocks ? a.nUnits : kBlocks;
      } else {
        if (l < launches - 1) a.norm = nullptr;
        if (c.out) {
          kernel = (const void*)&vrClip<CAP>;
          blocks = a.nTiles < kSMs * kScaleBlocks ? (int)a.nTiles : kSMs * kScaleBlocks;
          if (!blocks) blocks = 1;
        } else {
          kernel = (const void*)&vrNormFinish<CAP>;
          blocks = 1 + (c.tensorNorms ? (n + Block::warps - 1) / Block::warps : 0);
        }
      }
      const vrResult_t r =
          launch(kernel, dim3((unsigned)blocks), dim3(Block::threads), 0, c.stream, a);
      if (r != vrSuccess) return r;
    }
    slots = base;
  }
  return vrSuccess;
}

vrResult_t checkList(const void* const* in, const size_t* counts, const vrDataType_t* types, int n) {
  if (n < 1 || !in || !counts || !types) return vrInvalidArgument;
  uint64_t tiles = 0;
  for (int t = 0; t < n; ++t) {
    const int es = elemSizeOf(types[t]);
    if (!es || (counts[t] && (!in[t] || misaligned(in[t], es)))) return vrInvalidArgument;
    if (counts[t] > ((size_t)1 << 48)) return vrInvalidArgument;
    tiles += tilesOf(in[t], counts[t], es, Block::tileBytes);
    if (tiles >= 0x7fffffffull) return vrInvalidArgument;
  }
  return vrSuccess;
}

size_t bytesOfTensor(const Call& c, int t) { return c.counts[t] * elemSizeOf(c.types[t]); }

// Tensors that are written: one after another in memory, upwards or downwards, as
// the views of a bucket are. The others' hull alone counts.
struct Run {
  uintptr_t lo = UINTPTR_MAX, hi = 0, lastLo = 0, lastHi = 0;
  bool up = true, down = true;
  void add(uintptr_t p, size_t n) {
    if (hi) {
      up = up && p >= lastHi;
      down = down && p + n <= lastLo;
    }
    lastLo = p, lastHi = p + n;
    lo = p < lo ? p : lo;
    hi = p + n > hi ? p + n : hi;
  }
  bool apartFrom(const Run& r) const { return lo >= r.hi || r.lo >= hi; }
};

// Whether outs overlap each other, or gradients other than outs[t] == grads[t].
// A run for each type, with the runs apart, is what buckets give and takes one walk;
// anything else is sorted by address.
vrResult_t checkOuts(const Call& c) {
  constexpr int kTypes = vrFloat64 - vrFloat16 + 1;
  Run reads[kTypes], writes[kTypes];
  bool apart = true;
  for (int t = 0; t < c.nTensors; ++t) {
    const size_t n = bytesOfTensor(c, t);
    if (!n) continue;
    const int k = c.types[t] - vrFloat16;
    writes[k].add((uintptr_t)c.out[t], n);
    if (c.out[t] != c.in[t]) reads[k].add((uintptr_t)c.in[t], n);
  }
  for (int k = 0; k < kTypes; ++k) {
    apart = apart && (writes[k].up || writes[k].down);
    for (int j = 0; j < kTypes; ++j)
      apart = apart && writes[k].apartFrom(reads[j]) && (j >= k || writes[k].apartFrom(writes[j]));
  }
  if (apart) return vrSuccess;
  struct Range {
    uintptr_t lo, hi;
    bool write;
  };
  std::unique_ptr<Range[]> all(new (std::nothrow) Range[2 * (size_t)c.nTensors]);
  if (!all) return vrInternalError;
  size_t m = 0;
  for (int t = 0; t < c.nTensors; ++t) {
    const size_t n = bytesOfTensor(c, t);
    if (!n) continue;
    const uintptr_t i = (uintptr_t)c.in[t], o = (uintptr_t)c.out[t];
    all[m++] = {o, o + n, true};
    if (i != o) all[m++] = {i, i + n, false};
  }
  std::sort(&all[0], &all[0] + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t written = 0, touched = 0;  // to there
  for (size_t i = 0; i < m; ++i) {
    if (all[i].lo < (all[i].write ? touched : written)) return vrInvalidArgument;
    touched = all[i].hi > touched ? all[i].hi : touched;
    if (all[i].write) written = all[i].hi > written ? all[i].hi : written;
  }
  return vrSuccess;
}

vrResult_t runChecked(const Call& c, const void* workspace, size_t workspaceBytes) {
  const size_t need = slotsBound(c.nTensors) * sizeof(uint64_t);
  if (!workspace || misaligned(workspace, 16) || workspaceBytes < need) return vrInvalidArgument;
  const Bytes outs[] = {bytesOf(c.norm, 4), bytesOf(c.tensorNorms, (size_t)c.nTensors * 4),
                        bytesOf(workspace, need)};
  if (anyOverlap(outs, 3, nullptr, 0)) return vrInvalidArgument;
  for (int t = 0; t < c.nTensors; ++t) {
    const size_t n = bytesOfTensor(c, t);
    const Bytes in = bytesOf(c.in[t], n), out = bytesOf(c.out ? c.out[t] : nullptr, n);
    for (const Bytes& o : outs)
      if (overlap(o, in) || overlap(o, out)) return vrInvalidArgument;
  }
  const vrResult_t r = c.out ? checkOuts(c) : vrSuccess;
  if (r != vrSuccess) return r;
  if (isShort(c)) return runShort(c);
  return c.nTensors <= kShortList ? runLong<kShortList>(c) : runLong<kLongList>(c);
}

}  // namespace

extern "C" VR_API vrResult_t vrGradNormWorkspace(int nTensors, size_t* bytes) {
  if (nTensors < 1 || !bytes) return vrInvalidArgument;
  *bytes = (size_t)(slotsBound(nTensors) * sizeof(uint64_t));
  return vrSuccess;
}

extern "C" VR_API vrResult_t vrGradNorm(const void* const* grads, const size_t* counts,
                                        const vrDataType_t* dtypes, int nTensors, float scale,
                                        float* norm, float* tensorNorms, void* workspace,
                                        size_t workspaceBytes, void* stream) {
  NvtxRange range("vrGradNorm");
  const vrResult_t r = checkList(grads, counts, dtypes, nTensors);
  if (r != vrSuccess) return r;
  if ((!norm && !tensorNorms) || misaligned(norm, 4) || misaligned(tensorNorms, 4) ||
      !(scale - scale == 0.f))
    return vrInvalidArgument;
  const Call c = {grads, nullptr, counts, dtypes, nTensors, scale, 0.f, norm, tensorNorms,
                  (uint64_t*)workspace, (cudaStream_t)stream};
  return runChecked(c, workspace, workspaceBytes);
}

extern "C" VR_API vrResult_t vrClipGradNorm(const void* const* grads, void* const* outs,
                                            const size_t* counts, const vrDataType_t* dtypes,
                                            int nTensors, float scale, float maxNorm, float* norm,
                                            void* workspace, size_t workspaceBytes, void* stream) {
  NvtxRange range("vrClipGradNorm");
  const vrResult_t r = checkList(grads, counts, dtypes, nTensors);
  if (r != vrSuccess) return r;
  if (!outs || misaligned(norm, 4) || !(scale - scale == 0.f) || !(maxNorm >= 0.f))
    return vrInvalidArgument;
  for (int t = 0; t < nTensors; ++t) {
    const size_t es = (size_t)elemSizeOf(dtypes[t]);
    if (counts[t] && (!outs[t] || misaligned(outs[t], es))) return vrInvalidArgument;
  }
  const Call c = {grads, outs, counts, dtypes, nTensors, scale, maxNorm, norm, nullptr,
                  (uint64_t*)workspace, (cudaStream_t)stream};
  return runChecked(c, workspace, workspaceBytes);
}
