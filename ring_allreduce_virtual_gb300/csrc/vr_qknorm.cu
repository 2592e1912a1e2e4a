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
#include "vr_places.h"

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
  uint32_t steps[2];  // of a warp: a token's queries, all of its heads
  uint32_t warps, rounds;  // each warp has so many tokens in full
  uint32_t quota, extra;   // its steps of the other tokens; how many warps have one more
  bool wideTable;  // rows of the tables are whole 16 bytes
  float* partials;  // [blocks][2][dim]: sums of g u
  uint32_t blocks;
  void* dw[2];
};

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;

// A token's position as it was loaded (whoever waits for it does that later), and its row of
// the tables; tableRows where it is outside of them.
__device__ __forceinline__ int2 load_position(const QkArgs& a, uint32_t b, uint32_t t) {
  if (!a.rot) return make_int2(0, 0);
  const uint64_t at = b * a.positionStride + t;
  return a.wide ? static_cast<const int2*>(a.positions)[at]
                : make_int2(static_cast<const int32_t*>(a.positions)[at], 0);
}
__device__ __forceinline__ uint64_t table_row(const QkArgs& a, int2 v) {
  const int64_t p = a.wide ? (int64_t)((uint64_t)(uint32_t)v.y << 32 | (uint32_t)v.x) : (int64_t)v.x;
  return p >= 0 && (uint64_t)p < a.tableRows ? (uint64_t)p : a.tableRows;
}
__device__ __forceinline__ uint64_t table_row(const QkArgs& a, uint32_t b, uint32_t t) {
  return table_row(a, load_position(a, b, t));
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
};

// A lane's angles of a token, from the rows of the tables in shared memory: of halves one
// for each element of a pack, of neighbours one for both elements of a pair. Past the
// rotated part, no rotation. BACK: the opposite angles.
template <typename T, bool INTER, bool BACK>
struct Angles {
  static constexpr int V = kV<T>, N = INTER ? V : V / 2;
  F2 c[N], s[N];
  __device__ __forceinline__ void load(const Packs<T, INTER>& at, const float* cosRow, const float* sinRow, int half) {
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int pair = (i < V / 2 ? at.a : at.b) / 2 + i % (V / 2);
        const bool in = (i < V / 2 ? at.hasA : at.hasB) && pair < half;
        const float sn = in ? (BACK ? -sinRow[pair] : sinRow[pair]) : 0.f;
        c[i] = f2(in ? cosRow[pair] : 1.f);
        s[i] = f2(-sn, sn);
      }
    } else {
      const bool in = at.a < half;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float2 cs = in ? *reinterpret_cast<const float2*>(cosRow + at.a + 2 * i) : make_float2(1.f, 1.f);
        const float2 sn = in ? *reinterpret_cast<const float2*>(sinRow + at.a + 2 * i) : make_float2(0.f, 0.f);
        c[i] = f2(cs.x, cs.y);
        s[i] = BACK ? f2(-sn.x, -sn.y) : f2(sn.x, sn.y);
      }
    }
  }
  // Both packs turned.
  __device__ __forceinline__ void turn(F2 (&x)[V / 2], F2 (&y)[V / 2]) const {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      if constexpr (INTER) {
        float p, q;
        split(x[i], p, q);
        x[i] = fma2(f2(q, p), s[i], x[i] * c[i]);
        split(y[i], p, q);
        y[i] = fma2(f2(q, p), s[V / 2 + i], y[i] * c[V / 2 + i]);
      } else {
        const F2 p = x[i];
        x[i] = p * c[i] - y[i] * s[i];
        y[i] = fma2(p, s[i], y[i] * c[i]);
      }
    }
  }
};

// The same with a kind's weights and one factor for the whole head: three operations for two
// elements, where weights, factor and turn one after the other are nine for four.
template <typename T, bool INTER>
struct WeightedAngles {
  static constexpr int V = kV<T>, H = V / 2;
  F2 p[H], q[H], s[H], t[H];
  __device__ __forceinline__ void load(const Packs<T, INTER>& at, const float* cosRow, const float* sinRow, int half,
                                       const float* w) {
    const float one[2] = {1.f, 1.f};
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const float* wa = at.hasA ? w + at.a + 2 * i : one;
      const float* wb = at.hasB ? w + at.b + 2 * i : one;
      if constexpr (INTER) {
        const int k = at.a / 2 + i, l = at.b / 2 + i;
        const bool inA = at.hasA && k < half, inB = at.hasB && l < half;
        const float ca = inA ? cosRow[k] : 1.f, sn = inA ? sinRow[k] : 0.f;
        const float cb = inB ? cosRow[l] : 1.f, sm = inB ? sinRow[l] : 0.f;
        p[i] = f2(wa[0], wa[1]) * f2(ca);
        q[i] = f2(wa[1], wa[0]) * f2(-sn, sn);
        s[i] = f2(wb[0], wb[1]) * f2(cb);
        t[i] = f2(wb[1], wb[0]) * f2(-sm, sm);
      } else {
        const bool in = at.a < half;
        const F2 c = in ? f2(cosRow[at.a + 2 * i], cosRow[at.a + 2 * i + 1]) : f2(1.f);
        const F2 n = in ? f2(sinRow[at.a + 2 * i], sinRow[at.a + 2 * i + 1]) : f2(0.f);
        p[i] = f2(wa[0], wa[1]) * c;
        q[i] = f2(wb[0], wb[1]) * n;
        s[i] = f2(wb[0], wb[1]) * c;
        t[i] = f2(wa[0], wa[1]) * n;
      }
    }
  }
  __device__ __forceinline__ void turn(F2 (&x)[H], F2 (&y)[H], F2 r) const {
#pragma unroll
    for (int i = 0; i < H; ++i) {
      if constexpr (INTER) {
        float a, b;
        split(x[i], a, b);
        x[i] = fma2(f2(b, a), q[i], x[i] * p[i]) * r;
        split(y[i], a, b);
        y[i] = fma2(f2(b, a), t[i], y[i] * s[i]) * r;
      } else {
        const F2 a = x[i];
        x[i] = (a * p[i] - y[i] * q[i]) * r;
        y[i] = fma2(a, t[i], y[i] * s[i]) * r;
      }
    }
  }
};

// A warp's steps, token after token. First whole tokens, the warps' next to each other in
// memory; then what is left of the tokens shared out by steps, so that all warps end at
// the same time.
struct Walk {
  uint32_t token, step, end;  // the present token's steps; none: no token is left
  uint32_t rounds, left;      // whole tokens after this one, steps of the rest after this token's
  __device__ __forceinline__ void rest(const QkArgs& a, uint32_t warp) {
    left = a.quota + (warp < a.extra ? 1 : 0);
    const uint32_t first = warp * a.quota + min(warp, a.extra);
    token = first / a.steps[1];
    step = first - token * a.steps[1];
    token += a.rounds * a.warps;
    end = min(a.steps[1], step + left);
    left -= end - step;
    left |= 1u << 31;  // the rest has begun
  }
  __device__ __forceinline__ void start(const QkArgs& a, uint32_t warp) {
    rounds = a.rounds;
    left = 0;
    if (rounds) {
      --rounds;
      token = warp, step = 0, end = a.steps[1];
    } else {
      rest(a, warp);
    }
  }
  __device__ __forceinline__ bool done() const { return step == end; }
  __device__ __forceinline__ void next(const QkArgs& a, uint32_t warp) {
    step = 0, end = a.steps[1];
    if (rounds) {
      --rounds;
      token += a.warps;
    } else if (left >> 31) {
      ++token;
      end = min(end, left & 0x7fffffff);
      left -= end;
    } else {
      rest(a, warp);
    }
  }
};
struct Token {
  uint32_t b, t;
  __device__ __forceinline__ Token(const QkArgs& a, uint32_t token) : b(0), t(token) {
    if (a.all != a.tokens) {
      b = token / a.tokens;
      t = token - b * a.tokens;
    }
  }
};
template <typename T>
__device__ __forceinline__ T* place(const Side& s, const Token& k, uint32_t head) {
  return static_cast<T*>(const_cast<void*>(s.p)) + k.b * s.batch + k.t * s.token + head * s.head;
}

// Whole packs, forward or backward. A warp takes a token's queries, then its keys, U times
// 32 / lanes heads at a step: the chains of one head (its sums over lanes, its root) are
// long, and side by side they fill each other's gaps. Each lane copies its own packs
// to shared memory STAGES - 1 steps ahead, across tokens too, and a token's angles come with
// its first step: nothing is waited for but what was asked for long before, and what is on
// its way takes no registers. Backward, a warp's sums of g u stay in registers until its
// last token; a block leaves one set.
// Bound by HBM where heads fill the lanes: 4 x 4096 tokens of 32 + 8 heads of 128 bf16
// backward 84 us, 0.90 of the measured copy peak (with one chain in twice the warps 0.65, 12
// warps of 168 registers 0.49: they spill; float32 does not, 0.93 against 0.89), 64 + 8 forward
// 107 us, 0.85 (0.74 with one chain). Heads of 80 use 5 of 8 lanes: 4 x 4096 tokens of 16 + 16
// float16 neighbours 0.63 forward and 0.50 backward, bound by what a scheduler's two warps issue (0.44 instructions a cycle).
constexpr int kStages = 3, kAtOnce = 2;
template <bool BACK>
constexpr int kBlocks = BACK ? 1 : 2;  // on an SM: 255 (168) registers a thread, or 128
template <typename T, bool BACK>
constexpr int kHeadWarps = BACK && sizeof(T) == 4 ? 12 : 8;
template <typename T, typename W, bool INTER, bool BACK>
__global__ void __launch_bounds__(32 * kHeadWarps<T, BACK>, kBlocks<BACK>) vrQkHeads(const __grid_constant__ QkArgs a) {
  constexpr int V = kV<T>, NP = BACK ? 4 : 2, H = V / 2, U = kAtOnce, WARPS = kHeadWarps<T, BACK>;
  extern __shared__ uint4 shared[];  // rings, then the tables' rows, then the weights
  begin_kernel();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = lane / a.lanes, groups = 32 / a.lanes, half = a.rot / 2;
  const Packs<T, INTER> at(a, lane % a.lanes);
  uint4* const ring = shared + warp * (kStages * U * NP * 32) + lane;
  float* const rows = reinterpret_cast<float*>(shared + WARPS * kStages * U * NP * 32) + warp * (kStages * 2 * half);
  float* const w = reinterpret_cast<float*>(shared + WARPS * kStages * U * NP * 32) + WARPS * (kStages * 2 * half);
  for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += 32 * WARPS) {
    const W* p = static_cast<const W*>(a.w[i >= a.dim]);
    w[i] = p ? to_f32(p[i < a.dim ? i : i - a.dim]) : 1.f;
  }
#pragma unroll
  for (int i = 0; i < kStages * U * NP; ++i)
    if (i % 2 ? !at.hasB : !at.hasA) ring[i * 32] = make_uint4(0, 0, 0, 0);
  __syncthreads();

  const uint32_t me = blockIdx.x * WARPS + warp, keys = a.steps[0];
  Walk now;
  now.start(a, me);
  Walk ahead = now, after = now;  // of the copies; of the positions, which are loaded a token before
  int2 position = make_int2(0, 0);
  const auto look = [&]() {
    if (after.done()) return;
    const Token k(a, after.token);
    position = load_position(a, k.b, k.t);
  };
  look();
  bool fresh = true;
  uint32_t into = 0;  // a token's place among the tables' rows
  const T *xp = nullptr, *gp = nullptr;
  uint64_t xStep = 0, gStep = 0;
  uint32_t left = 0;  // heads from this lane's next one on
  const auto fetch = [&](int stage) {
    if (!ahead.done()) {
      if (fresh || ahead.step == keys) {
        const Token k(a, ahead.token);
        const int kind = ahead.step >= keys;
        const uint32_t head = (kind ? ahead.step - keys : ahead.step) * U * groups + group;
        left = a.heads[kind] - head;  // "negative" where there is none
        xp = place<const T>(a.x[kind], k, head);
        xStep = groups * a.x[kind].head;
        if (BACK) {
          gp = place<const T>(a.dy[kind], k, head);
          gStep = groups * a.dy[kind].head;
        }
      }
      if (fresh) {
        fresh = false;
        float* to = rows + into * 2 * half;
        into = into + 1 == kStages ? 0 : into + 1;
        const uint64_t row = half ? table_row(a, position) : 0;
        const bool none = row == a.tableRows;
        const float *cp = a.cos + row * half, *sp = a.sin + row * half;
        if (!none && a.wideTable) {  // 16 bytes a lane
          for (int i = lane * 4; i < 2 * half; i += 128)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(to + i)),
                         "l"(i < half ? cp + i : sp + (i - half))
                         : "memory");
        } else {
          for (int i = lane; i < 2 * half; i += 32) {
            if (none)
              to[i] = nan32();
            else
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(to + i)),
                           "l"(i < half ? cp + i : sp + (i - half))
                           : "memory");
          }
        }
        after.next(a, me);
        look();
      }
      const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + stage * (U * NP * 32));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((int)left > 0) {
          const auto copy = [&](int p, const T* from) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + (u * NP + p) * 512), "l"(from) : "memory");
          };
          if (at.hasA) copy(0, xp + at.a);
          if (at.hasB) copy(1, xp + at.b);
          if (BACK && at.hasA) copy(2, gp + at.a);
          if (BACK && at.hasB) copy(3, gp + at.b);
        }
        left -= groups;
        xp += xStep;
        if (BACK) gp += gStep;
      }
      if (++ahead.step == ahead.end) {
        ahead = after;
        fresh = true;
      }
    }
    copies_commit();
  };
#pragma unroll 1
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  F2 sa[2][BACK ? H : 1], sb[2][BACK ? H : 1];  // sums of g u
  if (BACK) {
#pragma unroll
    for (int i = 0; i < H; ++i) sa[0][i] = sb[0][i] = sa[1][i] = sb[1][i] = f2(0.f);
  }
  const float mean = 1.f / (float)a.dim;
  std::conditional_t<BACK, Angles<T, INTER, true>, WeightedAngles<T, INTER>> angles;
  int stage = 0;
  uint32_t from = 0;  // the next token's place among the tables' rows
  bool first;         // of the token's steps here
  // Steps [now.step, end) of the present token, which are of one kind.
  const auto run = [&](auto kindOf, uint32_t end) {
    constexpr int kind = decltype(kindOf)::value;
    uint32_t head = (now.step - (kind ? keys : 0)) * U * groups + group;
    T* op = place<T>(a.out[kind], Token(a, now.token), head);
    const uint64_t oStep = groups * a.out[kind].head;
    [[maybe_unused]] F2 wa[H], wb[H];
    if (BACK) {
#pragma unroll
      for (int i = 0; i < H; ++i) {
        const float* p = w + kind * a.dim;
        wa[i] = at.hasA ? f2(p[at.a + 2 * i], p[at.a + 2 * i + 1]) : f2(1.f);
        wb[i] = at.hasB ? f2(p[at.b + 2 * i], p[at.b + 2 * i + 1]) : f2(1.f);
      }
    }
    bool load = first || !BACK;  // the angles, forward each kind's with its weights
#pragma unroll 1
    for (; now.step < end; ++now.step) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      copies_wait<kStages - 1>();
      if (load) {
        load = false;
        if (first) {
          first = false;
          __syncwarp();  // the row was copied by all lanes
          from = from + 1 == kStages ? 0 : from + 1;
        }
        const float* r = rows + (from == 0 ? kStages - 1 : from - 1) * 2 * half;
        if constexpr (BACK) angles.load(at, r, r + half, half);
        else angles.load(at, r, r + half, half, w + kind * a.dim);
        // Before a copy for a later token takes this one's place (of tokens of one step the next fetch's):
        // where a head is one lane's, no shuffle holds the lanes together. In front of that fetch it
        // costs 1 % of the backward pass, here nothing.
        __syncwarp();
      }
      const uint4* in = ring + stage * (U * NP * 32);
      stage = stage + 1 == kStages ? 0 : stage + 1;
      F2 fa[U][H], fb[U][H];
      [[maybe_unused]] F2 ga[U][H], gb[U][H];
      [[maybe_unused]] float q[U], p[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        F2 q2 = f2(0.f), p2 = f2(0.f);
        unpack<T>(in[u * NP * 32], fa[u]);
        unpack<T>(in[u * NP * 32 + 32], fb[u]);
#pragma unroll
        for (int i = 0; i < H; ++i) q2 = fma2(fb[u][i], fb[u][i], fma2(fa[u][i], fa[u][i], q2));
        q[u] = both(q2);
        if constexpr (BACK) {
          unpack<T>(in[u * NP * 32 + 64], ga[u]);
          unpack<T>(in[u * NP * 32 + 96], gb[u]);
          angles.turn(ga[u], gb[u]);
#pragma unroll
          for (int i = 0; i < H; ++i)
            p2 = fma2(gb[u][i] * wb[i], fb[u][i], fma2(ga[u][i] * wa[i], fa[u][i], p2));
          p[u] = both(p2);
        }
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1)
        if (d < a.lanes) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            q[u] += __shfl_xor_sync(~0u, q[u], d);
            if (BACK) p[u] += __shfl_xor_sync(~0u, p[u], d);
          }
        }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool mine = head < a.heads[kind];
        head += groups;
        const float r = rsqrtf(q[u] * mean + a.eps);
        const F2 r2 = f2(r);
        if constexpr (BACK) {
          // never r^2, which leaves the range of a float before dx does
          const F2 k2 = f2(-(r * (r * (p[u] * mean))));
          if (mine) {
#pragma unroll
            for (int i = 0; i < H; ++i) {
              sa[kind][i] = fma2(ga[u][i], fa[u][i] * r2, sa[kind][i]);
              sb[kind][i] = fma2(gb[u][i], fb[u][i] * r2, sb[kind][i]);
              fa[u][i] = fma2(fa[u][i], k2, ga[u][i] * wa[i]) * r2;
              fb[u][i] = fma2(fb[u][i], k2, gb[u][i] * wb[i]) * r2;
            }
          }
        } else {
          angles.turn(fa[u], fb[u], r2);
        }
        if (mine) {
          if (at.hasA) *reinterpret_cast<uint4*>(op + at.a) = pack<T>(fa[u]);
          if (at.hasB) *reinterpret_cast<uint4*>(op + at.b) = pack<T>(fb[u]);
        }
        op += oStep;
      }
    }
  };
  for (; !now.done(); now.next(a, me)) {
    first = true;
    if (now.step < keys) run(std::integral_constant<int, 0>{}, min(keys, now.end));
    if (now.step < now.end) run(std::integral_constant<int, 1>{}, now.end);
  }
  if constexpr (BACK) {
    if (!a.partials) return;
    copies_wait<0>();
    __syncthreads();  // the sums take the rings' place
    float* const sums = reinterpret_cast<float*>(shared);  // [warps][2][dim]
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      float sum[2 * V];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        split(sa[kind][i], sum[2 * i], sum[2 * i + 1]);
        split(sb[kind][i], sum[V + 2 * i], sum[V + 2 * i + 1]);
      }
      // over the heads of a warp, then over the warps
      for (int d = a.lanes; d < 32; d <<= 1) {
#pragma unroll
        for (int i = 0; i < 2 * V; ++i) sum[i] += __shfl_xor_sync(~0u, sum[i], d);
      }
      if (group == 0) {
        float* mine = sums + (warp * 2 + kind) * a.dim;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (at.hasA) mine[at.a + i] = sum[i];
          if (at.hasB) mine[at.b + i] = sum[V + i];
        }
      }
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += 32 * WARPS) {
      float t = 0.f;
      for (int v = 0; v < WARPS; ++v) t += sums[v * 2 * a.dim + i];
      a.partials[(uint64_t)blockIdx.x * 2 * a.dim + i] = t;
    }
  }
}

// Heads of any width, strides and alignment, and those whose rotated half is no whole packs: a warp
// for each head walks over it in single elements, twice, and loads positions and angles for each
// head: bound by its instructions. 4 x 4096 tokens of 16 + 16 bf16 heads of 80, of which 40 are
// rotated, 251 us forward and 750 backward, 0.10 and 0.05 of the measured copy peak (with 32
// rotated, whole packs, 39 and 76); of 96 with 24 rotated 246 and 735. Pair i is elements (2 i, 2 i + 1) or (i, i + rot / 2); the elements
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

// The bytes of an argument.
Places placesOf(const void* p, size_t heads, const size_t* st, const Shape& s, int es) {
  Places b(p, s.dim * es);
  b.axis(s.batch, st[0] * es);
  b.axis(s.tokens, st[1] * es);
  b.axis(heads, st[2] * es);
  return b;
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
  a.wideTable = (((uintptr_t)a.cos | (uintptr_t)a.sin | a.rot * 2) & 15) == 0;
  // Batches whose tokens follow one another are one.
  bool one = a.all != a.tokens && (!a.rot || a.positionStride == a.tokens);
  for (int k = 0; k < 2; ++k)
    for (const Side* s : {&a.x[k], &a.dy[k], &a.out[k]}) one = one && (!s->p || s->batch == a.tokens * s->token);
  if (one) a.tokens = a.all;
  return true;
}

template <typename T, typename W, bool BACK>
vrResult_t wholeHeads(QkArgs& a, cudaStream_t st) {
  constexpr int WARPS = kHeadWarps<T, BACK>;
  const void* f = a.inter ? (const void*)&vrQkHeads<T, W, true, BACK> : (const void*)&vrQkHeads<T, W, false, BACK>;
  const uint32_t at = kAtOnce * (32 / a.lanes);
  a.steps[0] = (a.heads[0] + at - 1) / at;
  a.steps[1] = a.steps[0] + (a.heads[1] + at - 1) / at;
  // One round of blocks; of few steps, a warp for each.
  const uint64_t need = ((uint64_t)a.all * a.steps[1] + WARPS - 1) / WARPS, most = (uint64_t)kSMs * kBlocks<BACK>;
  a.blocks = (uint32_t)(need < most ? need : most);
  a.warps = a.blocks * WARPS;
  a.rounds = a.all / a.warps;
  const uint32_t rest = a.all % a.warps * a.steps[1];  // below 2^12 tokens of below 2^17 steps
  a.quota = rest / a.warps;
  a.extra = rest % a.warps;
  size_t smem = (size_t)WARPS * kStages * ((BACK ? 4 : 2) * 512 * kAtOnce + a.rot * sizeof(float)) +
                2 * a.dim * sizeof(float);
  if constexpr (BACK) {
    const size_t sums = (size_t)WARPS * 2 * a.dim * sizeof(float);
    if (smem < sums) smem = sums;
  }
  if (!setOnce(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024) ||
      !setOnce(f, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared))
    return vrCudaError;
  return launch(f, dim3(a.blocks), dim3(32 * WARPS), smem, st, a);
}

// An argument for the kernels; what the stride of an axis of one element is does not matter.
Side sideOf(const void* p, size_t heads, const size_t* st, const Shape& s) {
  return {p, s.batch > 1 ? st[0] : 0, s.tokens > 1 ? st[1] : 0, heads > 1 ? st[2] : 0};
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
  a.x[0] = sideOf(q, qHeads, qStrides, c.s);
  if (kHeads) a.x[1] = sideOf(k, kHeads, kStrides, c.s);
  a.w[0] = qWeight, a.w[1] = kWeight;
  a.heads[0] = (uint32_t)qHeads, a.heads[1] = (uint32_t)kHeads;
  a.cos = cosTable, a.sin = sinTable, a.tableRows = tableRows;
  a.positions = positions, a.positionStride = batch > 1 ? positionStride : 0;
  a.tokens = (uint32_t)tokens, a.all = (uint32_t)(batch * tokens);
  a.dim = (uint32_t)dim, a.rot = (uint32_t)rotaryDim, a.inter = interleaved, a.eps = eps;
  return vrSuccess;
}

// The arguments that no output may touch.
int inputs(const Call& c, Places* in) {
  const QkArgs& a = c.a;
  const size_t table = a.rot ? a.tableRows * (a.rot / 2) * 4 : 0;
  in[0] = Places(a.w[0], c.s.dim * c.ws);
  in[1] = Places(a.w[1], c.s.dim * c.ws);
  in[2] = Places(a.cos, table);
  in[3] = Places(a.sin, table);
  in[4] = Places(a.positions, a.rot ? ((c.s.batch - 1) * a.positionStride + c.s.tokens) * (a.wide ? 8 : 4) : 0);
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
  a.out[0] = sideOf(qOut, qHeads, qOutStrides, c.s);
  if (kHeads) a.out[1] = sideOf(kOut, kHeads, kOutStrides, c.s);
  // In place is allowed, each for itself.
  Places in[5];
  const int n = inputs(c, in);
  const Places qIn = placesOf(q, qHeads, qStrides, c.s, c.es), qo = placesOf(qOut, qHeads, qOutStrides, c.s, c.es);
  const Places kIn = kHeads ? placesOf(k, kHeads, kStrides, c.s, c.es) : Places();
  const Places ko = kHeads ? placesOf(kOut, kHeads, kOutStrides, c.s, c.es) : Places();
  const Places outs[] = {qo, ko};
  if (anyOverlap(outs, 2, in, n) || overlap(qo, kIn) || overlap(ko, qIn) ||
      (!(q == qOut && same(qStrides, qOutStrides)) && overlap(qo, qIn)) ||
      (kHeads && !(k == kOut && same(kStrides, kOutStrides)) && overlap(ko, kIn)))
    return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    cudaStream_t st = (cudaStream_t)stream;
    if (layOut<T>(a, false)) return wholeHeads<T, W, false>(a, st);
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
  if (misaligned(dqWeight, c.ws) || misaligned(dkWeight, c.ws)) return vrInvalidArgument;
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
  a.dy[0] = sideOf(dq, qHeads, dqStrides, c.s);
  a.out[0] = sideOf(dqIn, qHeads, dqInStrides, c.s);
  if (kHeads) {
    a.dy[1] = sideOf(dk, kHeads, dkStrides, c.s);
    a.out[1] = sideOf(dkIn, kHeads, dkInStrides, c.s);
  }
  a.dw[0] = dqWeight, a.dw[1] = dkWeight;
  a.partials = params ? (float*)workspace : nullptr;
  // dq and dk may be overwritten by what is computed from them, each for itself.
  Places in[7];
  int n = inputs(c, in);
  in[n++] = placesOf(q, qHeads, qStrides, c.s, c.es);
  in[n++] = kHeads ? placesOf(k, kHeads, kStrides, c.s, c.es) : Places();
  const bool overQ = dq == dqIn && same(dqStrides, dqInStrides);
  const bool overK = kHeads && dk == dkIn && same(dkStrides, dkInStrides);
  const Places dqb = placesOf(dq, qHeads, dqStrides, c.s, c.es);
  const Places dkb = kHeads ? placesOf(dk, kHeads, dkStrides, c.s, c.es) : Places();
  const Places outs[] = {placesOf(dqIn, qHeads, dqInStrides, c.s, c.es),
                         kHeads ? placesOf(dkIn, kHeads, dkInStrides, c.s, c.es) : Places(),
                         Places(dqWeight, dim * c.ws), Places(dkWeight, dim * c.ws),
                         Places(params ? workspace : nullptr, workspaceOf(dim))};
  if (anyOverlap(outs, 5, in, n)) return vrInvalidArgument;
  for (int i = 0; i < 5; ++i)
    if ((!(i == 0 && overQ) && overlap(outs[i], dqb)) || (!(i == 1 && overK) && overlap(outs[i], dkb)))
      return vrInvalidArgument;
  return dispatch(dtype, weightType, [&](auto t, auto w) {
    using T = decltype(t);
    using W = decltype(w);
    vrResult_t r;
    if (layOut<T>(a, true)) {
      r = wholeHeads<T, W, true>(a, st);
    } else {
      const size_t smem = params ? (size_t)kWarps * 2 * dim * sizeof(float) : 0;
      const uint64_t blocks = ((uint64_t)a.all * (a.heads[0] + a.heads[1]) + kWarps - 1) / kWarps;
      a.blocks = (unsigned)(blocks < kBackwardBlocks ? blocks : kBackwardBlocks);
      const void* f = (const void*)&vrQkBackwardAny<T, W>;
      if (smem > 48 * 1024 && !setOnce(f, cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024)) return vrCudaError;
      r = launch(f, dim3(a.blocks), dim3(kThreads), smem, st, a);
    }
    if (r == vrSuccess && params)
      r = launch((const void*)&vrQkJoin<W>, dim3((unsigned)((dim + 31) / 32), 2), dim3(32 * kJoinWarps), 0, st, a);
    return r;
  });
}
