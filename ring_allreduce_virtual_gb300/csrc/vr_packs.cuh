// vr_packs.cuh -- what the training-step operators share that work on aligned 16-byte
// packs of elements: pairs of floats, packs as pairs and back, clusters, attributes
// of kernels.
#pragma once

#include <mutex>

#include "vr_opcommon.cuh"

namespace vrop {

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
__device__ __forceinline__ F2 operator-(F2 a, F2 b) {
  F2 r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
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

// The same with bfloat16's lower elements by a product (c65536, which the compiler must not
// know: an argument of the launch), for kernels whose time is that of the pipe that shifts,
// compares and selects.
template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, uint32_t c65536, F2* f) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2(__uint_as_float(w[i] * c65536), __uint_as_float(w[i] & 0xffff0000u));
  } else {
    unpack<T>(v, f);
  }
}

// Copies to shared memory on their way (cp.async): a group of them, and the wait for all
// but the last N groups.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
inline bool allowLargeClusters(const void* kernel) {
  return setOnce(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
}

}  // namespace vrop
