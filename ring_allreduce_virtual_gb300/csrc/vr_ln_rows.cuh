// vr_ln_rows.cuh -- what the layer norm kernels that keep a row in registers
// share: how a row is cut into packs, and sums over the threads of a row.
//
// A row belongs to a group of threads: part of a warp, some warps of a block,
// or the blocks of a cluster. It is cut at the 16-byte boundaries of memory:
// the whole packs inside it, dealt to the threads, and up to V - 1 elements (V =
// 16 / element size) before the first and after the last, one for each of the
// first threads. So every access but those is a whole aligned pack, whatever
// the row's width and address. Groups take rows a multiple of V rows apart
// where rows do not all start alike: V rows are a multiple of 16 bytes, so a
// group sees one cut in all of its rows and a thread one set of columns, whose
// weights, and whose gradients' sums, it keeps in registers.
#pragma once

#include <mutex>

#include "vr_opcommon.cuh"

namespace vrln {

using namespace vrop;

// Where the threads of a row are.
enum { IN_WARP = 0, IN_BLOCK = 1, IN_CLUSTER = 2 };

struct Layout {
  int tpr;     // threads of a row in one block
  int groups;  // rows of a block at a time
  int ctas;    // blocks of a row (a cluster), 1 but for IN_CLUSTER
  int offset;  // bytes by which row 0 starts after a 16-byte boundary
  int skew;    // bytes by which the offset grows from row to row, modulo 16
  uint32_t step;  // rows between two rows of a group
};

constexpr int kMaxWarps = 32;

template <typename T>
constexpr int kV = 16 / (int)sizeof(T);

// Two floats in one 64-bit register pair: sm_103a adds and multiplies both in
// one instruction, which halves the arithmetic of a row.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ void split(F2 a, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(a.v));
}
__device__ __forceinline__ float both(F2 a) {
  float x, y;
  split(a, x, y);
  return x + y;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// One 32-bit word of T (two 16-bit elements) as floats.
template <typename T>
__device__ __forceinline__ F2 word2(uint32_t w) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  } else {
    __half2 h;
    memcpy(&h, &w, 4);
    const float2 f = __half22float2(h);
    return f2(f.x, f.y);
  }
}

// A pack as pairs of floats, and back (the one rounding of a result).
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, F2* f) {
  if constexpr (sizeof(T) == 4) {
    f[0] = f2(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2(__uint_as_float(v.z), __uint_as_float(v.w));
  } else {
    f[0] = word2<T>(v.x);
    f[1] = word2<T>(v.y);
    f[2] = word2<T>(v.z);
    f[3] = word2<T>(v.w);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t round2(F2 a) {
  float x, y;
  split(a, x, y);
  uint32_t w;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    memcpy(&w, &h, 4);
  } else {
    const __half2 h = __floats2half2_rn(x, y);
    memcpy(&w, &h, 4);
  }
  return w;
}
template <typename T>
__device__ __forceinline__ uint4 pack(const F2* f) {
  uint4 v;
  if constexpr (sizeof(T) == 4) {
    float e[4];
    split(f[0], e[0], e[1]);
    split(f[1], e[2], e[3]);
    memcpy(&v, e, 16);
  } else {
    v = make_uint4(round2<T>(f[0]), round2<T>(f[1]), round2<T>(f[2]), round2<T>(f[3]));
  }
  return v;
}

// Rows on their way into shared memory. Each thread copies the packs that it
// will read itself, some rows ahead, so no barrier separates the copy from the
// read, and the bytes in flight (what HBM's latency asks for) take no registers.
template <int S, int G>  // constant offsets of both addresses
__device__ __forceinline__ void copy16(uint32_t smem, const void* g) {
  asm volatile("cp.async.cg.shared.global [%0+%2], [%1+%3], 16;" ::"r"(smem), "l"(g), "n"(S), "n"(G)
               : "memory");
}
// f(integral_constant 0), ..., f(integral_constant N - 1)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void each(F f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    each<N, I + 1>(f);
  }
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The parameters of a thread's V columns from c0 on: packed as they are where
// they have the rows' type, else as floats. `none` where the pointer is NULL.
// Plain loads: the read-only path asks that nobody writes the parameters from the
// kernel's launch on, and the stream's previous kernel may still be writing them then.
template <typename T, typename W>
struct Params {
  static constexpr int V = kV<T>;
  static constexpr bool packed = sizeof(W) == sizeof(T);
  std::conditional_t<packed, uint4, float4> v[packed ? 1 : V / 4];
  __device__ __forceinline__ void load(const W* p, int c0, bool used, float none) {
    W e[V];
    if (p && used && ((uintptr_t)(p + c0) & 15) == 0) {
#pragma unroll
      for (int i = 0; i < (int)(V * sizeof(W) / 16); ++i) {
        const uint4 q = reinterpret_cast<const uint4*>(p + c0)[i];
        memcpy(reinterpret_cast<char*>(e) + 16 * i, &q, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) e[i] = p && used ? p[c0 + i] : from_f32<W>(none);
    }
    memcpy(v, e, sizeof(v));
  }
  __device__ __forceinline__ void get(F2* f) const {
    if constexpr (packed) {
      unpack<T>(v[0], f);
    } else {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        f[2 * i] = f2(v[i].x, v[i].y);
        f[2 * i + 1] = f2(v[i].z, v[i].w);
      }
    }
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n"
               "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void store_remote(float* p, uint32_t cta, float v) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(cta));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

__device__ __forceinline__ float load_remote(const float* p, uint32_t cta) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(cta));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// Sums of N values (N rows') over the threads of a row, the same in each of
// them. In a warp the N values share the steps: after log2(N) of them a lane
// holds one value, that of row (lane & (N - 1)). Between warps two halves of the
// buffer are used in turn: the barrier of the next sum separates the reads of
// this one from the writes of the one after.
template <int MODE, int N>
struct RowSum {
  static_assert(N == 1 || N == 2 || N == 4, "");
  float buf[2][MODE == IN_WARP ? 1 : (MODE == IN_CLUSTER ? 8 * 16 : kMaxWarps) * N];

  __device__ __forceinline__ float fold(const float (&v)[N], int lane) const {
    if constexpr (N == 1) {
      return v[0];
    } else if constexpr (N == 2) {
      return (lane & 1 ? v[1] : v[0]) + __shfl_xor_sync(~0u, lane & 1 ? v[0] : v[1], 1);
    } else {
      const float a = (lane & 1 ? v[1] : v[0]) + __shfl_xor_sync(~0u, lane & 1 ? v[0] : v[1], 1);
      const float b = (lane & 1 ? v[3] : v[2]) + __shfl_xor_sync(~0u, lane & 1 ? v[2] : v[3], 1);
      return (lane & 2 ? b : a) + __shfl_xor_sync(~0u, lane & 2 ? a : b, 2);
    }
  }

  __device__ __forceinline__ void operator()(float (&v)[N], const Layout& l, int group, int& turn) {
    const int lane = threadIdx.x & 31;
    float t = fold(v, lane);
    if constexpr (MODE == IN_WARP) {
      for (int o = N; o < l.tpr; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
    } else {
#pragma unroll
      for (int o = N; o < 32; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
      const int nw = l.tpr >> 5;
      int first = 0, all = nw * N;
      if constexpr (MODE == IN_BLOCK) {
        if (lane < N) buf[turn][(threadIdx.x >> 5) * N + lane] = t;
        first = group * nw * N;
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(l.tpr) : "memory");
      } else {
        if (lane < l.ctas * N)
          store_remote(&buf[turn][(cluster_rank() * nw + (threadIdx.x >> 5)) * N + (lane & (N - 1))],
                       lane / N, t);
        all *= l.ctas;
        cluster_sync();
      }
      t = 0.f;
      for (int k = lane; k < all; k += 32) t += buf[turn][first + k];
#pragma unroll
      for (int o = N; o < 32; o <<= 1) t += __shfl_xor_sync(~0u, t, o);
      turn ^= 1;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(~0u, t, N == 1 ? lane : (lane & ~(N - 1)) | i);
  }
};

// A thread's place in its row, the rows of its group, and the row's cut. P
// packs of a thread lie a warp's width apart (a fixed distance, so that their
// addresses are one register and constants), a warp's packs together.
template <typename T, int MODE, int P>
struct Place {
  static constexpr int V = kV<T>;
  int group;     // in the block
  int lane;      // in the row
  uint64_t row;  // the group's first
  int n;         // rows of the group
  int rounds;    // the most rows of a group in this warp
  int stripe;    // lanes of a warp that hold one row
  int head;      // elements before the first whole pack
  int packs;     // whole packs
  int pack0;     // the thread's first
  int edge;      // this thread's element outside the packs, -1: none
  // Of thread `thread` of block `block`, `rank` in its cluster.
  __host__ __device__ __forceinline__ Place(const Layout& l, uint64_t rows, int cols, uint32_t block,
                                            uint32_t thread, uint32_t rank) {
    uint64_t first;
    if constexpr (MODE == IN_CLUSTER) {
      group = 0;
      lane = (int)(rank * l.tpr + thread);
      row = first = block / l.ctas;
    } else {
      group = thread / l.tpr;
      lane = thread - group * l.tpr;
      row = (uint64_t)block * l.groups + group;
      first = MODE == IN_WARP ? (uint64_t)block * l.groups + (thread & ~31) / l.tpr : row;
    }
    // fewer than kMostRows rows: 32-bit divisions
    n = row < rows ? (int)(((uint32_t)(rows - row) + l.step - 1) / l.step) : 0;
    rounds = first < rows ? (int)(((uint32_t)(rows - first) + l.step - 1) / l.step) : 0;
    stripe = MODE == IN_WARP ? l.tpr : 32;
    const int shift = (int)((l.offset + (uint32_t)row * (uint32_t)l.skew) & 15) / (int)sizeof(T);
    head = (V - shift) & (V - 1);
    head = head < cols ? head : cols;
    packs = (cols - head) / V;
    pack0 = MODE == IN_WARP ? lane : (lane >> 5) * (32 * P) + (lane & 31);
    edge = lane < head ? lane : lane + packs * V;
    edge = edge < cols ? edge : -1;
  }
  __device__ __forceinline__ Place(const Layout& l, uint64_t rows, int cols)
      : Place(l, rows, cols, blockIdx.x, threadIdx.x, MODE == IN_CLUSTER ? cluster_rank() : 0) {}
  __host__ __device__ __forceinline__ int pack(int i) const {
    return pack0 + i * (MODE == IN_WARP ? stripe : 32);
  }
  __host__ __device__ __forceinline__ int column(int i) const { return head + pack(i) * V; }
  __host__ __device__ __forceinline__ bool used(int i) const { return pack(i) < packs; }
};

// ------------------------------------------------------------------ host
// Row counts of the kernels here are 32-bit numbers of rows of a group.
constexpr uint64_t kMostRows = 1ull << 31;

// Warps on an SM at a time: its registers hold so many, and its shared memory
// the blocks' rings.
inline int residentWarps(int regs, size_t smem, int threads) {
  const int byRegs = 65536 / 32 / regs;
  const int blocks = (int)((227 * 1024) / (smem + 4096));  // and what each block has besides
  const int byShared = blocks * ((threads + 31) / 32);
  return byShared < byRegs ? byShared : byRegs;
}

// Dynamic shared memory of a block, at most.
constexpr size_t kMostShared = 200 * 1024;

// Sets an attribute of a kernel, once on each device.
inline bool setOnce(const void* kernel, cudaFuncAttribute what, int value) {
  constexpr int kSeen = 256;
  static std::mutex m;
  static const void* seen[kSeen];
  static int device[kSeen], attribute[kSeen], n = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> g(m);
  for (int i = 0; i < n; ++i)
    if (seen[i] == kernel && device[i] == dev && attribute[i] == (int)what) return true;
  if (cudaFuncSetAttribute(kernel, what, value) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  if (n < kSeen) seen[n] = kernel, attribute[n] = (int)what, device[n++] = dev;
  return true;
}
inline bool allowShared(const void* kernel) {
  return setOnce(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMostShared);
}
inline bool allowLargeClusters(const void* kernel) {
  return setOnce(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

// How rows of `cols` elements are laid over threads: PACKS packs for each
// thread, in a warp, a block, or a cluster of up to 8 blocks; blocks of as many
// rows as blockThreads hold (smaller blocks that fill an SM better are slower:
// 1280 float32 forward 0.71 with 15 warps in 5 blocks, 0.91 with 12 in 2). False if
// the row is too wide for it.
inline bool layoutFor(uint64_t cols, int V, int packs, int blockThreads, int maxThreads,
                      bool ragged, Layout* l, int* mode) {
  const uint64_t n = cols / V;  // whole packs of a row, at most
  uint64_t threads = (n + packs - 1) / packs;
  const uint64_t least = ragged ? 2 * V : 4;  // a thread for each element outside the packs
  threads = threads < least ? least : threads;
  l->ctas = 1;
  if (threads <= 32) {
    *mode = IN_WARP;
    l->tpr = threads <= 4 ? 4 : threads <= 8 ? 8 : threads <= 16 ? 16 : 32;
    l->groups = blockThreads / l->tpr;  // whole warps
    return true;
  }
  if (threads <= (uint64_t)maxThreads) {
    *mode = IN_BLOCK;
    l->tpr = (int)((threads + 31) / 32 * 32);
    l->groups = blockThreads / l->tpr;
    if (l->groups < 1) l->groups = 1;
    if (l->groups > 15) l->groups = 15;  // named barriers
    return true;
  }
  *mode = IN_CLUSTER;
  l->groups = 1;
  for (l->ctas = 2; l->ctas <= 8; l->ctas *= 2) {
    const uint64_t t = ((threads + l->ctas - 1) / l->ctas + 31) / 32 * 32;
    if (t <= (uint64_t)maxThreads) {
      l->tpr = (int)t;
      return true;
    }
  }
  return false;
}

// Blocks (or clusters) of rows that the GPU holds at a time, at most:
// residentWarps warps on an SM.
inline uint64_t mostAtOnce(const Layout& l, int residentWarps) {
  const int blockWarps = (l.tpr * l.groups + 31) / 32;
  int perSm = residentWarps / blockWarps;
  perSm = perSm < 1 ? 1 : perSm > 32 ? 32 : perSm;
  return (uint64_t)kSMs * perSm / l.ctas;
}

// Clusters that it does hold, up to `most`. A cluster lies in one group of SMs,
// and what is left of a group stays empty: of 4 blocks, one on an SM, 36 clusters
// fit and not 38, of 8 blocks 15 and not 19, and the others would take a second
// round (2000 x 65536 bf16 forward 297 us in 38 clusters, 182 in 36).
inline uint64_t clustersAtOnce(const void* kernel, const Layout& l, size_t smem, uint64_t most) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)(most * l.ctas));
  cfg.blockDim = dim3((unsigned)(l.tpr * l.groups));
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)l.ctas;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return most;
  }
  return n < 1 ? 1 : (uint64_t)n < most ? (uint64_t)n : most;
}

// The grid for `rows` rows, `most` blocks (or clusters) at a time: whole rounds
// over the rows (a multiple of those that a group takes at once), each as full as
// the last. Sets l->step. Fewer at a time never make a larger grid.
inline unsigned gridFor(uint64_t rows, Layout* l, int V, uint64_t most, bool ragged,
                        int rowsAtOnce) {
  const uint64_t unit = (uint64_t)l->groups;  // rows of a block (or cluster) at a time
  // Blocks come in lots whose rows are a multiple of V.
  uint64_t lot = 1;
  while (ragged && lot * unit % V) ++lot;
  most = most / lot * lot ? most / lot * lot : lot;
  uint64_t rounds = (rows + most * unit - 1) / (most * unit);
  if (rounds < (uint64_t)rowsAtOnce) rounds = rowsAtOnce;
  uint64_t blocks = ((rows + rounds - 1) / rounds + unit - 1) / unit;
  if (rounds > 1) blocks = (blocks + lot - 1) / lot * lot;
  l->step = (uint32_t)(blocks * unit);
  return (unsigned)(blocks * l->ctas);
}

}  // namespace vrln
