// vr_gradnorm.cu -- the norm of a list of gradients, and clipping by it.
//
//   N = |s| sqrt(sum_t sum_i g_ti^2),  out = g s min(1, max / N)
//
// for tensors of any sizes, types and alignments. A list is cut into tiles of
// kTileBytes; block b of B takes the tiles [nt b / B, nt (b + 1) / B), which
// may lie in several tensors, and leaves one partial sum for each tensor it
// meets, in slot b + t: along a block's walk t grows, from one block to the
// next b does, so every slot has one writer and the sums have one order (no
// atomics: equal inputs give equal bits). The second kernel adds the slots up.
//
// Both kernels are bound by HBM: the norm reads every element once (2 flop
// each), clipping reads it once more and writes it.
#include "vr_opcommon.cuh"

namespace {

using namespace vrop;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPacks = 4;  // 16-byte packs of a thread in flight
constexpr int kTileBytes = kThreads * kPacks * 16;
constexpr int kBlocks = kSMs * 4;
// Tensors of one launch. Their table lies in the kernel's parameter space
// (32,764 bytes at most): nothing is copied to the device beforehand and the
// caller's arrays are free on return. Longer lists take several launches.
constexpr int kSmallList = 64;
constexpr int kLongList = 960;

template <int CAP>
struct Table {
  int nTensors;
  int nBlocks;
  uint32_t nTiles;
  uint32_t nSlots;    // of all launches of the call
  uint32_t slotBase;  // of this launch
  int tensorBase;
  float scale;
  float maxNorm;
  double* slots;
  float* norm;
  float* tensorNorms;
  const void* in[CAP];
  void* out[CAP];
  uint64_t count[CAP];
  uint32_t tile[CAP + 1];  // tiles before tensor t
  uint8_t type[CAP];
};

__host__ __device__ inline int sizeOfType(int t) {
  return t == vrFloat64 ? 8 : t == vrFloat32 ? 4 : 2;
}

// Elements before the first 16-byte boundary.
__host__ __device__ inline uint64_t headOf(const void* p, uint64_t count, int es) {
  const uint64_t h = ((16 - ((uintptr_t)p & 15)) & 15) / es;
  return h < count ? h : count;
}

inline uint64_t tilesOf(const void* p, uint64_t count, int es) {
  if (!count) return 0;
  const uint64_t body = (count - headOf(p, count, es)) * es;
  return body ? (body + kTileBytes - 1) / kTileBytes : 1;
}

// The first tile of block b, and the block that holds tile k.
__host__ __device__ inline uint32_t firstTile(uint32_t nTiles, int nBlocks, int b) {
  return (uint32_t)((uint64_t)nTiles * b / nBlocks);
}
__device__ inline uint32_t blockOf(uint32_t nTiles, int nBlocks, uint32_t k) {
  return (uint32_t)((((uint64_t)k + 1) * nBlocks - 1) / nTiles);
}

// The tensor that tile k lies in: the last t with tile[t] <= k.
template <int CAP>
__device__ inline int tensorOf(const Table<CAP>& a, uint32_t k) {
  int lo = 0, hi = a.nTensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.tile[mid] <= k) lo = mid; else hi = mid;
  }
  return lo;
}

// A sum in two floats: hi + lo, the rounding errors of hi caught exactly
// (Knuth's two-sum), so that a thread's long run costs no precision.
struct Sum2 {
  float hi = 0.f, lo = 0.f;
  __device__ void add(float x) {
    const float s = hi + x, z = s - hi;
    lo += (hi - (s - z)) + (x - z);
    hi = s;
  }
  __device__ double value() const { return (double)hi + (double)lo; }
};

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
  return __ldg(reinterpret_cast<const uint4*>(p));
}

// A block's sum of squares of the tiles [k0, k1) of one tensor, the same value in
// every thread.
template <typename T>
__device__ double sumTiles(const T* g, uint64_t count, uint32_t k0, uint32_t k1, double* buf) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr uint64_t E = kTileBytes / sizeof(T);
  const uint64_t head = headOf(g, count, (int)sizeof(T)), body = count - head;
  const T* p = g + head;
  uint32_t bits = 0;
  Sum2 sum;
  if constexpr (sizeof(T) < 8) {
    for (uint32_t k = k0; k < k1; ++k) {
      const uint64_t left = body - k * E;
      const T* q = p + k * E;
      float acc[2] = {0.f, 0.f};
      if (left >= E) {
        uint4 v[kPacks];
#pragma unroll
        for (int i = 0; i < kPacks; ++i) v[i] = load16(q + (threadIdx.x + i * kThreads) * V);
#pragma unroll
        for (int i = 0; i < kPacks; ++i) squares<T>(v[i], acc, bits);
      } else {
        const int packs = (int)(left / V);
        for (int i = threadIdx.x; i < packs; i += kThreads)
          squares<T>(load16(q + (uint64_t)i * V), acc, bits);
        const int at = packs * V + threadIdx.x;
        if (at < (int)left) {
          const float x = to_f32(q[at]);
          acc[0] = fmaf(x, x, acc[0]);
          bits |= x != 0.f;
        }
      }
      sum.add(acc[0] + acc[1]);
    }
    if (k0 == 0 && threadIdx.x < head) {
      const float x = to_f32(g[threadIdx.x]);
      sum.add(x * x);
      bits |= x != 0.f;
    }
    const double s = block_sum<kWarps>(sum.value(), buf);
    // The squares of 32-bit floats and of bfloat16 leave the range of a float
    // long before their sum leaves that of a double. Where they did (the sum
    // is infinite, or so small that squares went below the smallest float),
    // the tiles are summed again in 64 bits. float16's squares always fit.
    if (std::is_same_v<T, __half>) return s;
    const bool small = s < 0x1p-90;
    if (s < 0x1p120 && !(small && __syncthreads_or(bits != 0))) return s;
  }
  __syncthreads();  // before `buf` is used again
  double d = 0;
  const uint64_t from = k0 ? head + k0 * E : 0, end = head + k1 * E, to = end < count ? end : count;
  for (uint64_t i = from + threadIdx.x; i < to; i += kThreads) {
    const double x = to_f64(g[i]);
    d = fma(x, x, d);
  }
  return block_sum<kWarps>(d, buf);
}

template <int CAP>
__device__ double sumTensor(const Table<CAP>& a, int t, uint32_t k0, uint32_t k1, double* buf) {
  if (k0 >= k1) return 0.0;
  switch (a.type[t]) {
    case vrFloat16: return sumTiles((const __half*)a.in[t], a.count[t], k0, k1, buf);
    case vrBfloat16: return sumTiles((const __nv_bfloat16*)a.in[t], a.count[t], k0, k1, buf);
    case vrFloat32: return sumTiles((const float*)a.in[t], a.count[t], k0, k1, buf);
    default: return sumTiles((const double*)a.in[t], a.count[t], k0, k1, buf);
  }
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) vrNormPartials(const __grid_constant__ Table<CAP> a) {
  __shared__ double buf[2][kWarps];
  const int b = blockIdx.x;
  const uint32_t k0 = firstTile(a.nTiles, a.nBlocks, b), k1 = firstTile(a.nTiles, a.nBlocks, b + 1);
  // This block owns the slots b + t from its first tensor to the next
  // block's first; a tensor without a tile in here gets a zero.
  const int t0 = b ? tensorOf(a, k0) : 0;
  const int t1 = b + 1 < a.nBlocks ? tensorOf(a, k1) : a.nTensors - 1;
  for (int t = t0; t <= t1; ++t) {
    const uint32_t first = a.tile[t], last = a.tile[t + 1];
    const uint32_t x = k0 > first ? k0 : first, y = k1 < last ? k1 : last;
    const double s = sumTensor(a, t, x - first, y > x ? y - first : x - first, buf[t & 1]);
    if (threadIdx.x == 0) a.slots[a.slotBase + b + t] = s;
    __syncthreads();
  }
}

// The sum of all slots, the same in every thread.
template <int CAP>
__device__ double sumSlots(const Table<CAP>& a, double* buf) {
  double s = 0;
  for (uint32_t i = threadIdx.x; i < a.nSlots; i += kThreads) s += a.slots[i];
  return block_sum<kWarps>(s, buf);
}

// The norms: block 0 the whole list's (in the call's last launch), warp w of
// all blocks those of the tensors w, w + warps, ...
template <int CAP>
__global__ void __launch_bounds__(kThreads) vrNormFinish(const __grid_constant__ Table<CAP> a) {
  __shared__ double buf[kWarps];
  const double scale = fabs((double)a.scale);
  if (blockIdx.x == 0 && a.norm) {
    const double s = sumSlots(a, buf);
    if (threadIdx.x == 0) *a.norm = (float)(scale * sqrt(s));
  }
  if (!a.tensorNorms) return;
  const int lane = threadIdx.x & 31;
  for (int t = blockIdx.x * kWarps + (threadIdx.x >> 5); t < a.nTensors; t += gridDim.x * kWarps) {
    double s = 0;
    if (a.tile[t] < a.tile[t + 1]) {
      const uint32_t b0 = blockOf(a.nTiles, a.nBlocks, a.tile[t]);
      const uint32_t b1 = blockOf(a.nTiles, a.nBlocks, a.tile[t + 1] - 1);
      for (uint32_t b = b0 + lane; b <= b1; b += 32) s += a.slots[a.slotBase + b + t];
    }
    s = warp_sum(s);
    if (lane == 0) a.tensorNorms[a.tensorBase + t] = (float)(scale * sqrt(s));
  }
}

// One tile of out = g * factor: 16-byte packs where g and out lie alike modulo
// 16 bytes, elements elsewhere. Each product is rounded once.
template <typename T, typename F>
__device__ void scaleTile(const T* g, T* out, uint64_t count, uint32_t k, F factor) {
  constexpr int V = 16 / (int)sizeof(T);
  constexpr uint64_t E = kTileBytes / sizeof(T);
  auto mul = [factor](T x) -> T {
    if constexpr (sizeof(T) == 8) return x * factor;
    else return from_f32<T>(to_f32(x) * factor);
  };
  const uint64_t head = headOf(g, count, (int)sizeof(T)), body = count - head;
  if (k == 0 && threadIdx.x < head) out[threadIdx.x] = mul(g[threadIdx.x]);
  const uint64_t left = body - k * E;
  const int n = (int)(left < E ? left : E);
  const T* p = g + head + k * E;
  T* q = out + head + k * E;
  const int packs = ((uintptr_t)q & 15) == 0 ? n / V : 0;
#pragma unroll
  for (int j = 0; j < kPacks; ++j) {
    const int i = threadIdx.x + j * kThreads;
    if (i < packs) {
      uint4 v = *reinterpret_cast<const uint4*>(p + i * V);
      T e[V];
      memcpy(e, &v, 16);
#pragma unroll
      for (int c = 0; c < V; ++c) e[c] = mul(e[c]);
      memcpy(&v, e, 16);
      *reinterpret_cast<uint4*>(q + i * V) = v;
    }
  }
  for (int i = packs * V + threadIdx.x; i < n; i += kThreads) q[i] = mul(p[i]);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) vrClip(const __grid_constant__ Table<CAP> a) {
  __shared__ double buf[kWarps];
  const double norm = fabs((double)a.scale) * sqrt(sumSlots(a, buf));
  // A norm that is not finite clips nothing: the caller sees it and drops
  // the step, and the gradients still show where it came from.
  const bool clips = norm > (double)a.maxNorm && isfinite(norm);
  const double factor = (double)a.scale * (clips ? (double)a.maxNorm / norm : 1.0);
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const int b = blockIdx.x;
  const uint32_t k0 = firstTile(a.nTiles, a.nBlocks, b), k1 = firstTile(a.nTiles, a.nBlocks, b + 1);
  if (k0 == k1) return;
  int t = tensorOf(a, k0);
  for (uint32_t k = k0; k < k1; ++k) {
    while (k >= a.tile[t + 1]) ++t;
    const uint32_t at = k - a.tile[t];
    const void* g = a.in[t];
    void* o = a.out[t];
    switch (a.type[t]) {
      case vrFloat16: scaleTile((const __half*)g, (__half*)o, a.count[t], at, (float)factor); break;
      case vrBfloat16:
        scaleTile((const __nv_bfloat16*)g, (__nv_bfloat16*)o, a.count[t], at, (float)factor);
        break;
      case vrFloat32: scaleTile((const float*)g, (float*)o, a.count[t], at, (float)factor); break;
      default: scaleTile((const double*)g, (double*)o, a.count[t], at, factor); break;
    }
  }
}

// ------------------------------------------------------------------ host
int blocksFor(uint64_t tiles) { return tiles < (uint64_t)kBlocks ? (tiles ? (int)tiles : 1) : kBlocks; }

// Slots of a launch of T tensors on B blocks: b + t runs from 0 to
// (B - 1) + (T - 1).
uint64_t slotsBound(int nTensors) {
  uint64_t s = 0;
  for (int at = 0; at < nTensors; at += kLongList) {
    const int n = nTensors - at < kLongList ? nTensors - at : kLongList;
    s += (uint64_t)kBlocks + n;
  }
  return s;
}

struct Call {
  const void* const* in;
  void* const* out;  // NULL: the norm alone
  const size_t* counts;
  const vrDataType_t* types;
  int nTensors;
  float scale, maxNorm;
  float* norm;
  float* tensorNorms;
  double* slots;
  cudaStream_t stream;
};

template <int CAP>
void fill(const Call& c, int at, int n, Table<CAP>* a) {
  uint64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    const int t = at + i;
    a->in[i] = c.in[t];
    a->out[i] = c.out ? c.out[t] : nullptr;
    a->count[i] = c.counts[t];
    a->type[i] = (uint8_t)c.types[t];
    a->tile[i] = (uint32_t)tiles;
    tiles += tilesOf(c.in[t], c.counts[t], sizeOfType(c.types[t]));
  }
  a->tile[n] = (uint32_t)tiles;
  a->nTensors = n;
  a->nTiles = (uint32_t)tiles;
  a->nBlocks = blocksFor(tiles);
  a->tensorBase = at;
  a->scale = c.scale;
  a->maxNorm = c.maxNorm;
  a->slots = c.slots;
  a->norm = nullptr;
  a->tensorNorms = c.tensorNorms;
}

template <int CAP>
vrResult_t runCall(const Call& c) {
  Table<CAP> a;
  const int launches = (c.nTensors + CAP - 1) / CAP;
  uint32_t slots = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint32_t base = 0;
    for (int l = 0; l < launches; ++l) {
      const int at = l * CAP, n = c.nTensors - at < CAP ? c.nTensors - at : CAP;
      if (pass == 0 || launches > 1) fill<CAP>(c, at, n, &a);
      a.slotBase = base;
      a.nSlots = slots;
      base += (uint32_t)(a.nBlocks + n - 1);
      const void* kernel;
      int blocks = a.nBlocks;
      if (pass == 0) {
        kernel = (const void*)&vrNormPartials<CAP>;
      } else {
        if (l == launches - 1) a.norm = c.norm;
        if (c.out) {
          kernel = (const void*)&vrClip<CAP>;
        } else {
          kernel = (const void*)&vrNormFinish<CAP>;
          blocks = c.tensorNorms ? (n + kWarps - 1) / kWarps : 1;
        }
      }
      const vrResult_t r = launch(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, c.stream, a);
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
    tiles += counts[t] ? tilesOf(in[t], counts[t], es) : 0;
    if (tiles >= 0xffffffffull) return vrInvalidArgument;
  }
  return vrSuccess;
}

vrResult_t runChecked(const Call& c, const void* workspace, size_t workspaceBytes) {
  if (!workspace || misaligned(workspace, 16) ||
      workspaceBytes < slotsBound(c.nTensors) * sizeof(double))
    return vrInvalidArgument;
  return c.nTensors <= kSmallList ? runCall<kSmallList>(c) : runCall<kLongList>(c);
}

}  // namespace

extern "C" VR_API vrResult_t vrGradNormWorkspace(int nTensors, size_t* bytes) {
  if (nTensors < 1 || !bytes) return vrInvalidArgument;
  *bytes = (size_t)(slotsBound(nTensors) * sizeof(double));
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
                  (double*)workspace, (cudaStream_t)stream};
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
    if (outs[t] != grads[t] && overlap(grads[t], counts[t] * es, outs[t], counts[t] * es))
      return vrInvalidArgument;
  }
  const Call c = {grads, outs, counts, dtypes, nTensors, scale, maxNorm, norm, nullptr,
                  (double*)workspace, (cudaStream_t)stream};
  return runChecked(c, workspace, workspaceBytes);
}
