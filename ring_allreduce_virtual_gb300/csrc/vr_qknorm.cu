// vr_qknorm.cu -- the root-mean-square norm of each query and key head with the
// rotation by its token's position in the same pass, and the backward pass.
//
//   r = 1 / sqrt(sum(x^2) / D + eps), u = x r, y = R (u w)
// R turns pairs (a, b) of the first elements by the angles of the position's row of
// the tables: (a cos - b sin, b cos + a sin).
//   g = R^T dy, dx = r (g w - u sum(g w u) / D), dw = sum over tokens and heads of g u
//
// Everything is computed in 32 bits and rounded once to the tensors' type. All of it
// is bound by memory traffic: a head is read once and written once (dy and x are read
// in the backward pass), and a token's angles once for all of its heads.
#include "vr_packs.cuh"

namespace {

using namespace vrop;

// Heads of one kind (queries or keys) of a tensor: element i of head h of token t of
// batch b at p + b batch + t token + h head + i.
struct Side {
  const void* p;
  uint64_t batch, token, head;
};

struct QkArgs {
  Side x[2], dy[2], out[2];  // queries, keys; out: y or dx
  const void* w[2];
  uint32_t heads[2];
  const float *cos, *sin;
  uint64_t tableRows;
  const void* positions;
  bool wide;  // positions of 64 bits
  uint64_t positionStride;
  uint32_t tokens, all;  // of a batch; of all batches
  uint32_t dim, rot;
  bool inter;  // pairs of neighbours, else of the rotated part's halves
  float eps;
  // the layout of the kernels of whole packs
  int lanes;       // of a head, a power of two
  int pairs;       // of packs of a head, one a lane
  uint32_t steps[2];  // of a warp for a token's heads of each kind
  uint32_t chunk, chunks;  // steps of a warp, warps of a token
  float* partials;  // [blocks][2][dim]: sums of g u
  uint32_t blocks;
  void* dw[2];
};

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// The row of the tables of a token; tableRows where the position is outside of them.
__device__ __forceinline__ uint64_t table_row(const QkArgs& a, uint32_t b, uint32_t t) {
  if (!a.rot) return 0;
  const uint64_t at = b * a.positionStride + t;
  const int64_t p = a.wide ? static_cast<const int64_t*>(a.positions)[at]
                           : static_cast<const int32_t*>(a.positions)[at];
  return p >= 0 && (uint64_t)p < a.tableRows ? (uint64_t)p : a.tableRows;
}
__device__ __forceinline__ float nan32() { return __int_as_float(0x7fffffff); }

// The two packs of a head that a lane holds. Where halves are paired they are
// partners, so that a pair never leaves its lane; what is not rotated follows.
template <typename T, bool INTER>
struct Packs {
  static constexpr int V = kV<T>;
  int a, b;       // first elements
  bool hasA, hasB;
  __device__ __forceinline__ Packs(const QkArgs& q, int j) {
    const int packs = q.dim / V, half = INTER ? 0 : q.rot / 2 / V;
    const int rest = packs - 2 * half, pairs = (rest + 1) / 2;
    hasA = j < half + pairs;
    if (j < half) {
      a = j, b = j + half;
      hasB = true;
    } else {
      a = half + j, b = a + pairs;  // 2 half + (j - half)
      hasB = hasA && b < packs;
    }
    a *= V, b *= V;
  }
  // The angles of the lane's pairs: of halves one for each element of a pack, of
  // neighbours V / 2 for each pack. Past the rotated part, no rotation.
  __device__ __forceinline__ void angles(const QkArgs& q, uint64_t row, float (&c)[V], float (&s)[V]) const {
    const float* cp = q.cos + row * (q.rot / 2);
    const float* sp = q.sin + row * (q.rot / 2);
    const bool out = row == q.tableRows;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      int at = a + i;
      bool in = hasA && a < (int)q.rot / 2;
      if (INTER) {
        at = (i < V / 2 ? a : b) / 2 + i % (V / 2);
        in = (i < V / 2 ? hasA : hasB) && at < (int)q.rot / 2;
      }
      c[i] = !in ? 1.f : out ? nan32() : cp[at];
      s[i] = !in ? 0.f : out ? nan32() : sp[at];
    }
  }
};

// Pairs (x, y) turned by (c, s); BACK: by the opposite angle.
template <int V, bool INTER, bool BACK>
__device__ __forceinline__ void turn(float (&x)[V], float (&y)[V], const float (&c)[V], const float (&s)[V]) {
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float s0 = BACK ? -s[i] : s[i], s1 = BACK ? -s[V / 2 + i] : s[V / 2 + i];
      const float p = x[2 * i], q = x[2 * i + 1], t = y[2 * i], v = y[2 * i + 1];
      x[2 * i] = p * c[i] - q * s0;
      x[2 * i + 1] = q * c[i] + p * s0;
      y[2 * i] = t * c[V / 2 + i] - v * s1;
      y[2 * i + 1] = v * c[V / 2 + i] + t * s1;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float si = BACK ? -s[i] : s[i];
      const float p = x[i], q = y[i];
      x[i] = p * c[i] - q * si;
      y[i] = q * c[i] + p * si;
    }
  }
}

template <typename T>
__device__ __forceinline__ void to_floats(const uint4& v, float (&f)[kV<T>]) {
  F2 p[kV<T> / 2];
  unpack<T>(v, p);
#pragma unroll
  for (int i = 0; i < kV<T> / 2; ++i) split(p[i], f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 to_pack(const float (&f)[kV<T>]) {
  F2 p[kV<T> / 2];
#pragma unroll
  for (int i = 0; i < kV<T> / 2; ++i) p[i] = f2(f[2 * i], f[2 * i + 1]);
  return pack<T>(p);
}

// Sum over the lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) v += __shfl_xor_sync(~0u, v, o);
  return v;
}

template <typename W, int V>
__device__ __forceinline__ void weights(const void* w, int at, bool has, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = w && has ? to_f32(static_cast<const W*>(w)[at + i]) : 1.f;
}

// Whole packs: a warp takes 32 / lanes heads of a token at a step, U steps' loads before
// the first is computed.
template <typename T, typename W, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) vrQkForward(const __grid_constant__ QkArgs a) {
  constexpr int V = kV<T>;
  begin_kernel();
  const uint64_t unit = (uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const uint32_t token = (uint32_t)(unit / a.chunks);
  if (token >= a.all) return;
  const int lane = threadIdx.x & 31, group = lane / a.lanes, groups = 32 / a.lanes;
  const uint32_t b = token / a.tokens, t = token - b * a.tokens;
  const Packs<T, INTER> at(a, lane % a.lanes);
  float c[V], s[V];
  at.angles(a, table_row(a, b, t), c, s);
  const uint32_t from = (uint32_t)(unit % a.chunks) * a.chunk;
  const uint32_t to = from + a.chunk;
  uint32_t before = 0;  // steps of the kinds before
  const float mean = 1.f / (float)a.dim;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const uint32_t first = from > before ? from - before : 0;
    const uint32_t last = to < before + a.steps[kind] ? to - (to > before ? before : to) : a.steps[kind];
    before += a.steps[kind];
    if (first >= last) continue;
    float wa[V], wb[V];
    weights<W, V>(a.w[kind], at.a, at.hasA, wa);
    weights<W, V>(a.w[kind], at.b, at.hasB, wb);
    const Side &x = a.x[kind], &y = a.out[kind];
    const T* xp = static_cast<const T*>(x.p) + b * x.batch + t * x.token;
    T* yp = static_cast<T*>(const_cast<void*>(y.p)) + b * y.batch + t * y.token;
    for (uint32_t step = first; step < last; step += U) {
      uint4 va[U], vb[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t head = (step + u) * groups + group;
        const bool in = step + u < last && head < a.heads[kind];
        va[u] = vb[u] = make_uint4(0, 0, 0, 0);
        if (in && at.hasA) va[u] = *reinterpret_cast<const uint4*>(xp + head * x.head + at.a);
        if (in && at.hasB) vb[u] = *reinterpret_cast<const uint4*>(xp + head * x.head + at.b);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (step + u >= last) break;
        const uint32_t head = (step + u) * groups + group;
        float fa[V], fb[V], q = 0.f;
        to_floats<T>(va[u], fa);
        to_floats<T>(vb[u], fb);
#pragma unroll
        for (int i = 0; i < V; ++i) q = fmaf(fb[i], fb[i], fmaf(fa[i], fa[i], q));
        const float r = rsqrtf(head_sum(q, a.lanes) * mean + a.eps);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          fa[i] = fa[i] * r * wa[i];
          fb[i] = fb[i] * r * wb[i];
        }
        turn<V, INTER, false>(fa, fb, c, s);
        if (head < a.heads[kind]) {
          if (at.hasA) *reinterpret_cast<uint4*>(yp + head * y.head + at.a) = to_pack<T>(fa);
          if (at.hasB) *reinterpret_cast<uint4*>(yp + head * y.head + at.b) = to_pack<T>(fb);
        }
      }
    }
  }
}

// The same backward. Each warp's tokens are blocks' warps apart, so that its sums of
// g u stay in registers until the last; a block leaves one set.
template <typename T, typename W, bool INTER, int U>
__global__ void __launch_bounds__(kThreads) vrQkBackward(const __grid_constant__ QkArgs a) {
  constexpr int V = kV<T>;
  extern __shared__ float sums[];  // [warps][2][dim], then added up
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = lane / a.lanes, groups = 32 / a.lanes;
  const Packs<T, INTER> at(a, lane % a.lanes);
  const float mean = 1.f / (float)a.dim;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    float wa[V], wb[V], da[V], db[V];
    weights<W, V>(a.w[kind], at.a, at.hasA, wa);
    weights<W, V>(a.w[kind], at.b, at.hasB, wb);
#pragma unroll
    for (int i = 0; i < V; ++i) da[i] = db[i] = 0.f;
    const Side &x = a.x[kind], &g = a.dy[kind], &o = a.out[kind];
    const uint64_t units = (uint64_t)a.all * a.chunks;
    for (uint64_t unit = (uint64_t)blockIdx.x * kWarps + warp; unit < units; unit += (uint64_t)gridDim.x * kWarps) {
      const uint32_t token = (uint32_t)(unit / a.chunks), from = (uint32_t)(unit % a.chunks) * a.chunk;
      const uint32_t last = min(from + a.chunk, a.steps[kind]);
      if (from >= last) continue;
      const uint32_t b = token / a.tokens, t = token - b * a.tokens;
      float c[V], s[V];
      at.angles(a, table_row(a, b, t), c, s);
      const T* xp = static_cast<const T*>(x.p) + b * x.batch + t * x.token;
      const T* gp = static_cast<const T*>(g.p) + b * g.batch + t * g.token;
      T* op = static_cast<T*>(const_cast<void*>(o.p)) + b * o.batch + t * o.token;
      for (uint32_t step = from; step < last; step += U) {
        uint4 xa[U], xb[U], ga[U], gb[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t head = (step + u) * groups + group;
          const bool in = step + u < last && head < a.heads[kind];
          xa[u] = xb[u] = ga[u] = gb[u] = make_uint4(0, 0, 0, 0);
          if (in && at.hasA) {
            xa[u] = *reinterpret_cast<const uint4*>(xp + head * x.head + at.a);
            ga[u] = *reinterpret_cast<const uint4*>(gp + head * g.head + at.a);
          }
          if (in && at.hasB) {
            xb[u] = *reinterpret_cast<const uint4*>(xp + head * x.head + at.b);
            gb[u] = *reinterpret_cast<const uint4*>(gp + head * g.head + at.b);
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (step + u >= last) break;
          const uint32_t head = (step + u) * groups + group;
          float fa[V], fb[V], ha[V], hb[V], q = 0.f, p = 0.f;
          to_floats<T>(xa[u], fa);
          to_floats<T>(xb[u], fb);
          to_floats<T>(ga[u], ha);
          to_floats<T>(gb[u], hb);
          turn<V, INTER, true>(ha, hb, c, s);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            q = fmaf(fb[i], fb[i], fmaf(fa[i], fa[i], q));
            p = fmaf(hb[i] * wb[i], fb[i], fmaf(ha[i] * wa[i], fa[i], p));
          }
          const float r = rsqrtf(head_sum(q, a.lanes) * mean + a.eps);
          // never r^2, which leaves the range of a float before dx does
          const float k = -(r * (r * (head_sum(p, a.lanes) * mean)));
          if (head < a.heads[kind]) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              da[i] = fmaf(ha[i], fa[i] * r, da[i]);
              db[i] = fmaf(hb[i], fb[i] * r, db[i]);
              fa[i] = r * fmaf(fa[i], k, ha[i] * wa[i]);
              fb[i] = r * fmaf(fb[i], k, hb[i] * wb[i]);
            }
            if (at.hasA) *reinterpret_cast<uint4*>(op + head * o.head + at.a) = to_pack<T>(fa);
            if (at.hasB) *reinterpret_cast<uint4*>(op + head * o.head + at.b) = to_pack<T>(fb);
          }
        }
      }
    }
    if (!a.partials) continue;
    // over the heads of a warp, then over the warps
    for (int o = a.lanes; o < 32; o <<= 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        da[i] += __shfl_xor_sync(~0u, da[i], o);
        db[i] += __shfl_xor_sync(~0u, db[i], o);
      }
    }
    if (group == 0) {
      float* mine = sums + (warp * 2 + kind) * a.dim;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at.hasA) mine[at.a + i] = da[i];
        if (at.hasB) mine[at.b + i] = db[i];
      }
    }
  }
  if (!a.partials) return;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
    float t = 0.f;
    for (int w = 0; w < kWarps; ++w) t += sums[w * 2 * a.dim + i];
    a.partials[(uint64_t)blockIdx.x * 2 * a.dim + i] = t;
  }
}

// Heads of any width, strides and alignment: a warp for each head, walks over it in
// single elements. Pair i is elements (2 i, 2 i + 1) or (i, i + rot / 2); the elements
// past the rotated part are taken as pairs that are not turned, with their like.
template <typename T>
struct Pairs {
  const QkArgs& a;
  uint32_t half, count;
  __device__ __forceinline__ Pairs(const QkArgs& q) : a(q), half(q.rot / 2), count(half + (q.dim - q.rot + 1) / 2) {}
  __device__ __forceinline__ void at(uint32_t i, uint32_t& x, uint32_t& y, bool& two) const {
    if (i < half) {
      x = a.inter ? 2 * i : i;
      y = a.inter ? 2 * i + 1 : i + half;
      two = true;
    } else {
      x = a.rot + 2 * (i - half);
      y = x + 1;
      two = y < a.dim;
    }
  }
  __device__ __forceinline__ void angle(uint64_t row, uint32_t i, float& c, float& s) const {
    c = 1.f, s = 0.f;
    if (i >= half) return;
    c = s = nan32();
    if (row == a.tableRows) return;
    c = a.cos[row * half + i];
    s = a.sin[row * half + i];
  }
};

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) vrQkForwardAny(const __grid_constant__ QkArgs a) {
  begin_kernel();
  const int lane = threadIdx.x & 31;
  const Pairs<T> pairs(a);
  const uint32_t heads = a.heads[0] + a.heads[1];
  const uint64_t units = (uint64_t)a.all * heads;
  for (uint64_t unit = (uint64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); unit < units;
       unit += (uint64_t)gridDim.x * kWarps) {
    const uint32_t token = (uint32_t)(unit / heads);
    uint32_t head = (uint32_t)(unit - (uint64_t)token * heads);
    const int kind = head >= a.heads[0];
    head -= kind ? a.heads[0] : 0;
    const uint32_t b = token / a.tokens, t = token - b * a.tokens;
    const uint64_t row = table_row(a, b, t);
    const T* x = static_cast<const T*>(a.x[kind].p) + b * a.x[kind].batch + t * a.x[kind].token + head * a.x[kind].head;
    T* y = static_cast<T*>(const_cast<void*>(a.out[kind].p)) + b * a.out[kind].batch + t * a.out[kind].token +
           head * a.out[kind].head;
    const W* w = static_cast<const W*>(a.w[kind]);
    float q = 0.f;
    for (uint32_t i = lane; i < a.dim; i += 32) q = fmaf(to_f32(x[i]), to_f32(x[i]), q);
    const float r = rsqrtf(warp_sum(q) / (float)a.dim + a.eps);
    for (uint32_t i = lane; i < pairs.count; i += 32) {
      uint32_t m, n;
      bool two;
      float c, s;
      pairs.at(i, m, n, two);
      pairs.angle(row, i, c, s);
      const float p = to_f32(x[m]) * r * (w ? to_f32(w[m]) : 1.f);
      const float v = two ? to_f32(x[n]) * r * (w ? to_f32(w[n]) : 1.f) : 0.f;
      y[m] = from_f32<T>(p * c - v * s);
      if (two) y[n] = from_f32<T>(v * c + p * s);
    }
  }
}

template <typename T, typename W>
__global__ void __launch_bounds__(kThreads) vrQkBackwardAny(const __grid_constant__ QkArgs a) {
  extern __shared__ float sums[];  // [warps][2][dim]
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* mine = sums + warp * 2 * a.dim;
  if (a.partials)
    for (uint32_t i = lane; i < 2 * a.dim; i += 32) mine[i] = 0.f;
  __syncwarp();
  const Pairs<T> pairs(a);
  const uint32_t heads = a.heads[0] + a.heads[1];
  const uint64_t units = (uint64_t)a.all * heads;
  for (uint64_t unit = (uint64_t)blockIdx.x * kWarps + warp; unit < units; unit += (uint64_t)gridDim.x * kWarps) {
    const uint32_t token = (uint32_t)(unit / heads);
    uint32_t head = (uint32_t)(unit - (uint64_t)token * heads);
    const int kind = head >= a.heads[0];
    head -= kind ? a.heads[0] : 0;
    const uint32_t b = token / a.tokens, t = token - b * a.tokens;
    const uint64_t row = table_row(a, b, t);
    const T* x = static_cast<const T*>(a.x[kind].p) + b * a.x[kind].batch + t * a.x[kind].token + head * a.x[kind].head;
    const T* g = static_cast<const T*>(a.dy[kind].p) + b * a.dy[kind].batch + t * a.dy[kind].token + head * a.dy[kind].head;
    T* dx = static_cast<T*>(const_cast<void*>(a.out[kind].p)) + b * a.out[kind].batch + t * a.out[kind].token +
            head * a.out[kind].head;
    const W* w = static_cast<const W*>(a.w[kind]);
    float* dw = mine + kind * a.dim;
    float r = 0.f, k = 0.f;
    for (int pass = 0; pass < 2; ++pass) {  // the sums, then dx
      float q = 0.f, p = 0.f;
      for (uint32_t i = lane; i < pairs.count; i += 32) {
        uint32_t m, n;
        bool two;
        float c, s;
        pairs.at(i, m, n, two);
        pairs.angle(row, i, c, s);
        const float gm = to_f32(g[m]), gn = two ? to_f32(g[n]) : 0.f;
        const float xm = to_f32(x[m]), xn = two ? to_f32(x[n]) : 0.f;
        const float hm = gm * c + gn * s, hn = gn * c - gm * s;
        const float wm = w ? to_f32(w[m]) : 1.f, wn = w && two ? to_f32(w[n]) : 1.f;
        if (pass == 0) {
          q = fmaf(xn, xn, fmaf(xm, xm, q));
          p = fmaf(hn * wn, xn, fmaf(hm * wm, xm, p));
        } else {
          dx[m] = from_f32<T>(r * fmaf(xm, k, hm * wm));
          if (two) dx[n] = from_f32<T>(r * fmaf(xn, k, hn * wn));
          if (a.partials) {
            dw[m] = fmaf(hm, xm * r, dw[m]);
            if (two) dw[n] = fmaf(hn, xn * r, dw[n]);
          }
        }
      }
      if (pass == 0) {
        r = rsqrtf(warp_sum(q) / (float)a.dim + a.eps);
        k = -(r * (r * (warp_sum(p) / (float)a.dim)));
      }
    }
  }
  if (!a.partials) return;
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
    float t = 0.f;
    for (int v = 0; v < kWarps; ++v) t += sums[v * 2 * a.dim + i];
    a.partials[(uint64_t)blockIdx.x * 2 * a.dim + i] = t;
  }
}

// The blocks' sums added up in a fixed order: a block takes 32 columns, a warp of it
// every 32nd block's.
constexpr int kJoinWarps = 32;
template <typename W>
__global__ void __launch_bounds__(32 * kJoinWarps) vrQkJoin(const __grid_constant__ QkArgs a) {
  __shared__ float buf[kJoinWarps][33];
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t first = blockIdx.x * 32;
  W* out = static_cast<W*>(a.dw[blockIdx.y]);
  if (!out) return;
  float s = 0.f;
  if (first + lane < a.dim) {
    const float* p = a.partials + (uint64_t)blockIdx.y * a.dim + first + lane;
#pragma unroll 8
    for (uint32_t i = warp; i < a.blocks; i += kJoinWarps) s += p[(uint64_t)i * 2 * a.dim];
  }
  buf[warp][lane] = s;
  __syncthreads();
  s = warp_sum(buf[lane][warp]);
  if (lane == 0 && first + warp < a.dim) out[first + warp] = from_f32<W>(s);
}

// ------------------------------------------------------------------ host
constexpr size_t kMostDim = 1024;
constexpr unsigned kBackwardBlocks = kSMs * 2;
constexpr uint64_t kMost = 1ull << 48;  // elements from the first to the last of a tensor

bool typesOk(vrDataType_t t, vrDataType_t w) {
  return (t == vrFloat16 || t == vrBfloat16 || t == vrFloat32) && (w == t || w == vrFloat32);
}

struct Shape {
  size_t batch, tokens, dim;
};

// Whether an argument's strides are usable: no address beyond 2^48 elements, and of an
// output no two elements in one place.
bool badSide(const void* p, size_t heads, const size_t* st, const Shape& s, int es, bool output) {
  if (!p || !st || misaligned(p, es)) return true;
  struct Axis {
    uint64_t n, stride;
  } ax[3] = {{s.batch, st[0]}, {s.tokens, st[1]}, {heads, st[2]}};
  uint64_t end = s.dim;
  for (const Axis& x : ax) {
    if (x.n <= 1) continue;
    if (x.stride > kMost / x.n) return true;
    end += (x.n - 1) * x.stride;
  }
  if (end > kMost) return true;
  if (!output) return false;
  uint64_t inner = s.dim;  // the axes from the smallest stride on: each steps over the ones inside
  for (int k = 0; k < 3; ++k) {
    int least = -1;
    for (int i = 0; i < 3; ++i)
      if (ax[i].n > 1 && (least < 0 || ax[i].stride < ax[least].stride)) least = i;
    if (least < 0) break;
    if (ax[least].stride < inner) return true;
    inner = (ax[least].n - 1) * ax[least].stride + inner;
    ax[least].n = 1;
  }
  return false;
}

// The bytes of an argument as rows: its outermost axis, or the two outermost where they
// step alike; what lies inside counts as taken in full.
Bytes bytesOfSide(const void* p, size_t heads, const size_t* st, const Shape& s, int es) {
  if (!p) return {0, 0, 0, 0};
  struct Axis {
    uint64_t n, stride;
  } ax[3] = {{s.batch, st[0]}, {s.tokens, st[1]}, {heads, st[2]}};
  for (int i = 0; i < 3; ++i)  // outermost first, axes of one element last
    for (int j = i + 1; j < 3; ++j)
      if (ax[j].n > 1 && (ax[i].n <= 1 || ax[j].stride > ax[i].stride)) {
        const Axis t = ax[i];
        ax[i] = ax[j], ax[j] = t;
      }
  uint64_t rows = ax[0].n, stride = ax[0].stride, width = s.dim;
  int inside = 1;
  if (ax[1].n > 1 && stride == ax[1].n * ax[1].stride) {
    rows *= ax[1].n;
    stride = ax[1].stride;
    inside = 2;
  }
  for (int i = inside; i < 3; ++i) width += (ax[i].n - 1) * (ax[i].n > 1 ? ax[i].stride : 0);
  if (rows <= 1) stride = width;
  if (rows > 1 && stride < width) return bytesOf(p, ((rows - 1) * stride + width) * es);
  return bytesOf(p, rows, width, stride, es);
}

template <typename F>
vrResult_t dispatch(vrDataType_t t, vrDataType_t w, F f) {
  if (t == vrFloat32) return f(float{}, float{});
  if (t == vrFloat16) return w == t ? f(__half{}, __half{}) : f(__half{}, float{});
  return w == t ? f(__nv_bfloat16{}, __nv_bfloat16{}) : f(__nv_bfloat16{}, float{});
}

bool wholePacks(const Side& s, int es) {
  return !s.p || (((uintptr_t)s.p | s.batch * es | s.token * es | s.head * es) & 15) == 0;
}

// Lays a call out for the kernels of whole packs; false if it has parts of packs, or a
// head is wider than a warp's two packs a lane.
template <typename T>
bool layOut(QkArgs& a, bool backward) {
  constexpr int V = kV<T>, es = sizeof(T);
  if (a.dim % V || (!a.inter && a.rot / 2 % V)) return false;
  for (int k = 0; k < 2; ++k)
    if (!wholePacks(a.x[k], es) || !wholePacks(a.out[k], es) || (backward && !wholePacks(a.dy[k], es))) return false;
  const int packs = a.dim / V, half = a.inter ? 0 : a.rot / 2 / V;
  a.pairs = half + (packs - 2 * half + 1) / 2;
  if (a.pairs > 32) return false;
  a.lanes = 1;
  while (a.lanes < a.pairs) a.lanes *= 2;
  const uint32_t groups = 32 / a.lanes;
  for (int k = 0; k < 2; ++k) a.steps[k] = (a.heads[k] + groups - 1) / groups;
  const uint32_t steps = backward ? (a.steps[0] > a.steps[1] ? a.steps[0] : a.steps[1]) : a.steps[0] + a.steps[1];
  // A token is one warp's, which reads its angles once, but where few tokens would leave
  // SMs without work.
  const uint64_t warps = (uint64_t)kSMs * 16;
  uint64_t chunk = (uint64_t)steps * a.all / warps;
  chunk = chunk < 1 ? 1 : chunk > steps ? steps : chunk;
  a.chunk = (uint32_t)chunk;
  a.chunks = (uint32_t)((steps + chunk - 1) / chunk);
  return true;
}

struct Call {
  QkArgs a;
  Shape s;
  int es, ws;
  bool nothing;
};

// The checks that both passes share.
vrResult_t begin(Call& c, const void* q, size_t qHeads, const size_t* qStrides, const void* k, size_t kHeads,
                 const size_t* kStrides, const void* qWeight, const void* kWeight, const float* cosTable,
                 const float* sinTable, size_t tableRows, const void* positions, vrDataType_t positionType,
                 size_t positionStride, size_t batch, size_t tokens, size_t dim, size_t rotaryDim, int interleaved,
                 float eps, vrDataType_t dtype, vrDataType_t weightType) {
  if (!typesOk(dtype, weightType) || dim < 1 || dim > kMostDim || rotaryDim > dim || rotaryDim % 2 ||
      !(eps >= 0.f) || !(eps - eps == 0.f) || (interleaved != 0 && interleaved != 1))
    return vrInvalidArgument;
  constexpr uint64_t k31 = 1ull << 31;
  if (batch >= k31 || tokens >= k31 || batch * tokens >= k31 || qHeads > 65535 || kHeads > 65535 || qHeads == 0)
    return vrInvalidArgument;
  c.es = elemSizeOf(dtype), c.ws = elemSizeOf(weightType);
  c.s = {batch, tokens, dim};
  memset(&c.a, 0, sizeof(c.a));
  c.nothing = batch * tokens == 0;
  if (misaligned(qWeight, c.ws) || misaligned(kWeight, c.ws)) return vrInvalidArgument;
  if (c.nothing) return vrSuccess;
  if (badSide(q, qHeads, qStrides, c.s, c.es, false) || (kHeads && badSide(k, kHeads, kStrides, c.s, c.es, false)))
    return vrInvalidArgument;
  if (rotaryDim) {
    const bool wide = positionType == vrInt64;
    if ((!wide && positionType != vrInt32) || !positions || misaligned(positions, wide ? 8 : 4) || !cosTable ||
        !sinTable || misaligned(cosTable, 4) || misaligned(sinTable, 4) || tableRows > kMost ||
        (batch > 1 && positionStride > kMost / batch))
      return vrInvalidArgument;
    c.a.wide = wide;
  }
  QkArgs& a = c.a;
  const auto side = [](const void* p, const size_t* st) { return p ? Side{p, st[0], st[1], st[2]} : Side{}; };
  a.x[0] = side(q, qStrides);
  if (kHeads) a.x[1] = side(k, kStrides);
  a.w[0] = qWeight, a.w[1] = kWeight;
  a.heads[0] = (uint32_t)qHeads, a.heads[1] = (uint32_t)kHeads;
  a.cos = cosTable, a.sin = sinTable, a.tableRows = tableRows;
  a.positions = positions, a.positionStride = batch > 1 ? positionStride : 0;
  a.tokens = (uint32_t)tokens, a.all = (uint32_t)(batch * tokens);
  a.dim = (uint32_t)dim, a.rot = (uint32_t)rotaryDim, a.inter = interleaved, a.eps = eps;
  return vrSuccess;
}

// The arguments that no output may touch.
int inputs(const Call& c, Bytes* in) {
  const QkArgs& a = c.a;
  const size_t table = a.rot ? a.tableRows * (a.rot / 2) * 4 : 0;
  in[0] = bytesOf(a.w[0], c.s.dim * c.ws);
  in[1] = bytesOf(a.w[1], c.s.dim * c.ws);
  in[2] = bytesOf(a.cos, table);
  in[3] = bytesOf(a.sin, table);
  in[4] = bytesOf(a.positions, a.rot ? ((c.s.batch - 1) * a.positionStride + c.s.tokens) * (a.wide ? 8 : 4) : 0);
  return 5;
}

bool same(const size_t* p, const size_t* q) { return p[0] == q[0] && p[1] == q[1] && p[2] == q[2]; }

size_t workspaceOf(size_t dim) { return (size_t)kBackwardBlocks * 2 * dim * sizeof(float); }

}  // namespace

extern "C" VR_API vrResult_t vrQkNormRopeForward(
    const void* q, size_t qHeads, const size_t* qStrides, const void* k, size_t kHeads, const size_t* kStrides,
    const void* qWeight, const void* kWeight, void* qOut, const size_t* qOutStrides, void* kOut,
    const size_t* kOutStrides, const float* cosTable, const float* sinTable, size_t tableRows, const void* positions,
    vrDataType_t positionType, size_t positionStride, size_t batch, size_t tokens, size_t dim, size_t rotaryDim,
    int interleaved, float eps, vrDataType_t dtype, vrDataType_t weightType, void* stream) {
  NvtxRange range("vrQkNormRopeForward");
  Call c;
  const vrResult_t rc = begin(c, q, qHeads, qStrides, k, kHeads, kStrides, qWeight, kWeight, cosTable, sinTable,
                              tableRows, positions, positionType, positionStride, batch, tokens, dim, rotaryDim,
                              interleaved, eps, dtype, weightType);
  if (rc != vrSuccess || c.nothing) return rc;
  QkArgs& a = c.a;
  if (badSide(qOut, qHeads, qOutStrides, c.s, c.es, true) ||
      (kHeads && badSide(kOut, kHeads, kOutStrides, c.s, c.es, true)))
    return vrInvalidArgument;
  a.out[0] = {qOut, qOutStrides[0], qOutStrides[1], qOutStrides[2]};
  if (kHeads) a.out[1] = {kOut, kOutStrides[0], kOutStrides[1], kOutStrides[2]};
  // In place is allowed, each for itself.
  Bytes in[7];
  const int n = inputs(c, in);
  const Bytes qIn = bytesOfSide(q, qHeads, qStrides, c.s, c.es), qo = bytesOfSide(qOut, qHeads, qOutStrides, c.s, c.es);
  const Bytes none = {0, 0, 0, 0};
  const Bytes kIn = kHeads ? bytesOfSide(k, kHeads, kStrides, c.s, c.es) : none;
  const Bytes ko = kHeads ? bytesOfSide(kOut, kHeads, kOutStrides, c.s, c.es) : none;
  const Bytes outs[] = {qo, ko};
  if (anyOverlap(outs, 2, in, n) || overlap(qo, kIn) || overlap(ko, qIn) ||
      (!(q == qOut && same(qStrides, qOutStrides)) && overlap(qo, qIn)) ||
      (kHeads && !(k == kOut && same(kStrides, kOutStrides)) && overlap(ko, kIn)))
    return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    cudaStream_t st = (cudaStream_t)stream;
    if (layOut<T>(a, false)) {
      const uint64_t blocks = ((uint64_t)a.all * a.chunks + kWarps - 1) / kWarps;
      const void* f = a.inter ? (const void*)&vrQkForward<T, W, true, 4> : (const void*)&vrQkForward<T, W, false, 4>;
      if (blocks > 0x7fffffffu) return vrInvalidArgument;
      return launch(f, dim3((unsigned)blocks), dim3(kThreads), 0, st, a);
    }
    const uint64_t units = (uint64_t)a.all * (a.heads[0] + a.heads[1]);
    const uint64_t blocks = (units + kWarps - 1) / kWarps, most = (uint64_t)kSMs * 8;
    return launch((const void*)&vrQkForwardAny<T, W>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads),
                  0, st, a);
  });
}

extern "C" VR_API vrResult_t vrQkNormRopeBackwardWorkspace(size_t dim, size_t* bytes) {
  if (dim < 1 || dim > kMostDim || !bytes) return vrInvalidArgument;
  *bytes = workspaceOf(dim);
  return vrSuccess;
}

extern "C" VR_API vrResult_t vrQkNormRopeBackward(
    const void* dq, const size_t* dqStrides, const void* dk, const size_t* dkStrides, const void* q, size_t qHeads,
    const size_t* qStrides, const void* k, size_t kHeads, const size_t* kStrides, const void* qWeight,
    const void* kWeight, void* dqIn, const size_t* dqInStrides, void* dkIn, const size_t* dkInStrides, void* dqWeight,
    void* dkWeight, const float* cosTable, const float* sinTable, size_t tableRows, const void* positions,
    vrDataType_t positionType, size_t positionStride, size_t batch, size_t tokens, size_t dim, size_t rotaryDim,
    int interleaved, float eps, vrDataType_t dtype, vrDataType_t weightType, void* workspace, size_t workspaceBytes,
    void* stream) {
  NvtxRange range("vrQkNormRopeBackward");
  Call c;
  const vrResult_t rc = begin(c, q, qHeads, qStrides, k, kHeads, kStrides, qWeight, kWeight, cosTable, sinTable,
                              tableRows, positions, positionType, positionStride, batch, tokens, dim, rotaryDim,
                              interleaved, eps, dtype, weightType);
  if (rc != vrSuccess) return rc;
  if (misaligned(dqWeight, c.ws) || misaligned(dkWeight, c.ws) || (!kHeads && dkWeight)) return vrInvalidArgument;
  cudaStream_t st = (cudaStream_t)stream;
  if (c.nothing) {  // sums over no tokens
    for (void* p : {dqWeight, dkWeight})
      if (p && cudaMemsetAsync(p, 0, dim * c.ws, st) != cudaSuccess) {
        cudaGetLastError();
        return vrCudaError;
      }
    return vrSuccess;
  }
  QkArgs& a = c.a;
  const bool params = dqWeight || dkWeight;
  if (badSide(dq, qHeads, dqStrides, c.s, c.es, false) || badSide(dqIn, qHeads, dqInStrides, c.s, c.es, true) ||
      (kHeads && (badSide(dk, kHeads, dkStrides, c.s, c.es, false) ||
                  badSide(dkIn, kHeads, dkInStrides, c.s, c.es, true))) ||
      (params && (!workspace || misaligned(workspace, 16) || workspaceBytes < workspaceOf(dim))))
    return vrInvalidArgument;
  a.dy[0] = {dq, dqStrides[0], dqStrides[1], dqStrides[2]};
  a.out[0] = {dqIn, dqInStrides[0], dqInStrides[1], dqInStrides[2]};
  if (kHeads) {
    a.dy[1] = {dk, dkStrides[0], dkStrides[1], dkStrides[2]};
    a.out[1] = {dkIn, dkInStrides[0], dkInStrides[1], dkInStrides[2]};
  }
  a.dw[0] = dqWeight, a.dw[1] = dkWeight;
  a.partials = params ? (float*)workspace : nullptr;
  // dq and dk may be overwritten by what is computed from them, each for itself.
  Bytes in[9];
  int n = inputs(c, in);
  const Bytes none = {0, 0, 0, 0};
  in[n++] = bytesOfSide(q, qHeads, qStrides, c.s, c.es);
  in[n++] = kHeads ? bytesOfSide(k, kHeads, kStrides, c.s, c.es) : none;
  const bool overQ = dq == dqIn && same(dqStrides, dqInStrides);
  const bool overK = kHeads && dk == dkIn && same(dkStrides, dkInStrides);
  const Bytes dqb = bytesOfSide(dq, qHeads, dqStrides, c.s, c.es);
  const Bytes dkb = kHeads ? bytesOfSide(dk, kHeads, dkStrides, c.s, c.es) : none;
  const Bytes outs[] = {bytesOfSide(dqIn, qHeads, dqInStrides, c.s, c.es),
                        kHeads ? bytesOfSide(dkIn, kHeads, dkInStrides, c.s, c.es) : none,
                        bytesOf(dqWeight, dim * c.ws), bytesOf(dkWeight, dim * c.ws),
                        bytesOf(params ? workspace : nullptr, workspaceOf(dim))};
  if (anyOverlap(outs, 5, in, n)) return vrInvalidArgument;
  for (int i = 0; i < 5; ++i)
    if ((!(i == 0 && overQ) && overlap(outs[i], dqb)) || (!(i == 1 && overK) && overlap(outs[i], dkb)))
      return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    const size_t smem = params ? (size_t)kWarps * 2 * dim * sizeof(float) : 0;
    const bool whole = layOut<T>(a, true);
    const uint64_t units = whole ? (uint64_t)a.all * a.chunks : (uint64_t)a.all * (a.heads[0] + a.heads[1]);
    const uint64_t blocks = (units + kWarps - 1) / kWarps;
    a.blocks = (unsigned)(blocks < kBackwardBlocks ? blocks : kBackwardBlocks);
    const void* f = !whole    ? (const void*)&vrQkBackwardAny<T, W>
                    : a.inter ? (const void*)&vrQkBackward<T, W, true, 2>
                              : (const void*)&vrQkBackward<T, W, false, 2>;
    if (smem > 48 * 1024 && !setOnce(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024)) return vrCudaError;
    vrResult_t r = launch(f, dim3(a.blocks), dim3(kThreads), smem, st, a);
    if (r == vrSuccess && params)
      r = launch((const void*)&vrQkJoin<W>, dim3((unsigned)((dim + 31) / 32), 2), dim3(32 * kJoinWarps), 0, st, a);
    return r;
  });
}
