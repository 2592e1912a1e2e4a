// vr_opcommon.cuh -- what the training-step operators (layer norm, gradient
// norm, clipping) share: element conversions, block sums, launch and argument
// helpers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>
#include <stddef.h>
#include <stdint.h>
#include <string.h>

#include <type_traits>

#include "vr.h"

namespace vrop {

// Grids are sized for the 152 SMs of the one GPU this library is written for, not
// asked of the device, so that sums have the same order wherever it runs -- but for
// dw and db of rows over clusters, whose number the driver says (clustersAtOnce).
constexpr int kSMs = 152;

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
};

inline int elemSizeOf(vrDataType_t t) {
  switch (t) {
    case vrFloat16: case vrBfloat16: return 2;
    case vrFloat32: return 4;
    case vrFloat64: return 8;
    default: return 0;  // not a type of these operators
  }
}

inline bool misaligned(const void* p, size_t to) { return (uintptr_t)p % to != 0; }

// The bytes of an argument: rows of `width` bytes, `stride` apart.
struct Bytes {
  uintptr_t at;
  uint64_t rows, width, stride;
  uintptr_t end() const { return at + (rows - 1) * stride + width; }
};
inline Bytes bytesOf(const void* p, uint64_t width) {
  return {(uintptr_t)p, p && width ? 1u : 0u, width, width};
}
inline Bytes bytesOf(const void* p, uint64_t rows, uint64_t cols, uint64_t stride, int es) {
  return {(uintptr_t)p, p ? rows : 0u, cols * es, stride * es};
}

// Whether two arguments share a byte. Matrices of one stride may lie side by
// side; of two strides they may not even interleave.
inline bool overlap(const Bytes& a, const Bytes& b) {
  if (!a.rows || !b.rows || a.at >= b.end() || b.at >= a.end()) return false;
  if (a.rows > 1 && b.rows > 1 && a.stride != b.stride) return true;
  const uint64_t s = a.rows > 1 ? a.stride : b.stride;
  if (a.rows == 1 && b.rows == 1) return true;
  const uint64_t r = b.at >= a.at ? (b.at - a.at) % s : (s - (a.at - b.at) % s) % s;
  return r < a.width || r + b.width > s;
}

// Whether one of the outputs shares a byte with an input or another output.
inline bool anyOverlap(const Bytes* outs, int nOuts, const Bytes* ins, int nIns) {
  for (int i = 0; i < nOuts; ++i) {
    for (int j = 0; j < nIns; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ double to_f64(double x) { return x; }
template <typename T>
__device__ __forceinline__ double to_f64(T x) { return (double)to_f32(x); }
// The one rounding of a result to its type, to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (std::is_same_v<T, __half>) return __float2half_rn(x);
  else if constexpr (std::is_same_v<T, __nv_bfloat16>) return __float2bfloat16_rn(x);
  else return x;
}

template <typename A>
__device__ __forceinline__ A warp_sum(A v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over a block of NW warps, the same value in every thread, added up in an
// order fixed by the lanes. `buf` holds NW values; the caller separates two
// uses of it by a barrier (two buffers in turn do).
template <int NW, typename A>
__device__ __forceinline__ A block_sum(A v, A* buf) {
  v = warp_sum(v);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
    __syncthreads();
    v = buf[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) v += buf[i];
  }
  return v;
}

// First in every kernel here, before it touches memory. All of them are launched
// before the stream's previous kernel has ended (where that one allows it, as
// these do): their blocks come to wait where blocks of that one have left, and
// go on when it has ended and all that it wrote can be seen. It takes the
// start of a launch, 2 to 3 us, out of a chain of calls.
__device__ __forceinline__ void begin_kernel() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launch of `kernel` with one by-value argument struct, in clusters of `ctas`.
template <typename Args>
inline vrResult_t launch(const void* kernel, dim3 grid, dim3 block, size_t smem,
                         cudaStream_t stream, Args& args, int ctas = 1) {
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (ctas > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = (unsigned)ctas;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
  ++cfg.numAttrs;
  void* a[] = {&args};
  if (cudaLaunchKernelExC(&cfg, kernel, a) != cudaSuccess) {
    cudaGetLastError();
    return vrCudaError;
  }
  return vrSuccess;
}

}  // namespace vrop
