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
#include "vr_opcommon.cuh"

namespace {

using namespace vrop;

struct FwdArgs {
  const void* x;
  const void* w;
  const void* b;
  void* y;
  float* mean;
  float* rstd;
  uint64_t rows, cols, xStride, yStride;
  float eps;
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
};

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// Rows of any width, stride and alignment: a block for each row, three walks
// over it.
template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) vrLnForwardAny(const __grid_constant__ FwdArgs a) {
  __shared__ float buf[2][kRowWarps];
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

// dx of rows of any width: a block for each row, two walks over it.
template <typename T, typename W>
__global__ void __launch_bounds__(kRowThreads) vrLnBackwardAny(const __grid_constant__ BwdArgs a) {
  __shared__ float buf[4][kRowWarps];
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

// dw and db, second step: the splits' sums added up, split by split.
template <typename W>
__global__ void __launch_bounds__(256) vrLnJoin(const __grid_constant__ BwdArgs a) {
  const uint64_t col = (uint64_t)blockIdx.x * 256 + threadIdx.x;
  if (col >= a.cols) return;
  W* out = static_cast<W*>(blockIdx.y ? a.db : a.dw);
  if (!out) return;
  float s = 0.f;
  for (int i = 0; i < a.splits; ++i) s += a.partials[((uint64_t)i * 2 + blockIdx.y) * a.cols + col];
  out[col] = from_f32<W>(s);
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

int splitsFor(uint64_t rows, uint64_t cols) {
  const uint64_t tiles = (cols + 31) / 32;
  uint64_t s = (uint64_t)kSMs * 8 / tiles + 1;
  const uint64_t most = (rows + 63) / 64;
  s = s < most ? s : most;
  return s ? (int)s : 1;
}

// Bytes from a matrix's first element to the end of its last.
size_t extent(uint64_t rows, uint64_t cols, uint64_t stride, int es) {
  return rows ? ((rows - 1) * stride + cols) * es : 0;
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
  if (!(x == y && xStride == yStride) &&
      overlap(x, extent(rows, cols, xStride, es), y, extent(rows, cols, yStride, es)))
    return vrInvalidArgument;
  FwdArgs a = {x, weight, bias, y, mean, rstd, rows, cols, xStride, yStride, eps};
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    const uint64_t most = (uint64_t)kSMs * 8;
    return launch((const void*)&vrLnForwardAny<T, W>, dim3((unsigned)(rows < most ? rows : most)),
                  dim3(kRowThreads), 0, (cudaStream_t)stream, a);
  });
}

extern "C" VR_API vrResult_t vrLayerNormBackwardWorkspace(size_t rows, size_t cols,
                                                          vrDataType_t dtype, size_t* bytes) {
  if (!typesOk(dtype, dtype) || cols < 1 || !bytes) return vrInvalidArgument;
  *bytes = (size_t)splitsFor(rows, cols) * 2 * cols * sizeof(float);
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
  const size_t out = extent(rows, cols, dxStride, es);
  if (overlap(dx, out, dy, extent(rows, cols, dyStride, es)) ||
      overlap(dx, out, x, extent(rows, cols, xStride, es)))
    return vrInvalidArgument;
  const bool params = dweight || dbias;
  BwdArgs a = {dy, x, weight, mean, rstd, dx, dweight, dbias, rows, cols,
               dyStride, xStride, dxStride, (float*)workspace, splitsFor(rows, cols)};
  if (params && (!workspace || misaligned(workspace, 16) ||
                 workspaceBytes < (size_t)a.splits * 2 * cols * sizeof(float)))
    return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    vrResult_t r = vrSuccess;
    const uint64_t most = (uint64_t)kSMs * 8;
    if (dx)
      r = launch((const void*)&vrLnBackwardAny<T, W>, dim3((unsigned)(rows < most ? rows : most)),
                 dim3(kRowThreads), 0, st, a);
    if (r == vrSuccess && params)
      r = launch((const void*)&vrLnColumns<T>, dim3((unsigned)((cols + 31) / 32), a.splits),
                 dim3(32 * kColWarps), 0, st, a);
    if (r == vrSuccess && params)
      r = launch((const void*)&vrLnJoin<W>, dim3((unsigned)((cols + 255) / 256), 2), dim3(256), 0,
                 st, a);
    return r;
  });
}
