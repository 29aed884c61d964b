// qknorm.hip -- a projection to queries, keys and values: the sum of N rank buffers, the
// norm of each head of the queries and keys, and their rotation by position, in one pass;
// and its gradient.
//
//   h    = round(x_0 + ... + x_{N-1})              summed in that order in f32
//   rs   = 1 / sqrt(mean(h^2) + eps), xhat = h rs  over a head
//   y    = R(xhat w), R turns the pair (a, b) to (a c - b s, b c + a s); values: v = h
//
//   u    = R^T dy, g = u w
//   dh   = rs (g - xhat mean(g xhat)), dw = sum over tokens and heads of u xhat; dv passes
//
// Both are HBM-bound: a few operations an element.  A head lies in the registers of LPH
// lanes, so every tensor is read once.  A lane holds two vectors of V elements, the two
// halves of the same pairs where halves rotate together, so that no pair crosses lanes;
// 64 / LPH heads of a token share a wave, an iteration.  Sums are f32; each output is rounded
// once.
//
// Rows need no alignment beyond their element's.  Where a part of a head (a half of the
// rotated elements, or the rest) ends inside a vector, the vector is moved back to end with
// it; its first `over` elements are then the neighbour's too: they are left out of sums,
// and both lanes, of one wave, store the same value after both have read.  Parts shorter
// than a vector go a pair a lane (V 1).
#include <type_traits>

#include "mrr_device.hpp"
#include "mrr_internal.hpp"
#include "mrr_ops.hpp"
#include "mrr_rows.hpp"

namespace mrr {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// ---- a lane's place in a head --------------------------------------------------------
struct Slot {
  uint32_t at, over;  // first element; elements that are the neighbour's too (V: all)
};

// Vector u of the part [from, from + len): whole, moved back, or past its end.
template <int V> __device__ __forceinline__ Slot part_slot(uint32_t from, uint32_t len, uint32_t u) {
  const uint32_t c = u * V, at = c + V <= len ? c : len - V, over = c - at;
  return {from + at, over < (uint32_t)V ? over : (uint32_t)V};
}

// Unit `u` of a head: its two vectors, which of them rotate, and its angles' place in a
// table row.  PAIRS: neighbours rotate together.  Past the head's units: nothing of its own.
// FULL: all of the head rotates and every lane has a whole unit, which leaves no element to
// mask (the kernels' arithmetic takes as long as their traffic otherwise).
template <int V, int LPH, bool PAIRS, bool FULL> struct Unit {
  Slot s[2];
  bool turn[2];
  uint32_t angle[2];  // PAIRS, V > 1: V / 2 angles for each vector; else V for both, the first
  __device__ __forceinline__ Unit(uint32_t dim, uint32_t rot, uint32_t u) {
    const uint32_t half = rot / 2, rest = dim - rot;
    if constexpr (FULL) {
      turn[0] = turn[1] = true;
      s[0].over = s[1].over = 0;
      s[0].at = u * V;
      s[1].at = u * V + dim / 2;
      angle[0] = PAIRS ? u * (V / 2) : u * V;
      angle[1] = angle[0] + dim / 4;
    } else if constexpr (PAIRS && V > 1) {
      const uint32_t nrot = (rot + V - 1) / V;
      auto vector = [&](uint32_t v, Slot& slot, bool& on, uint32_t& from) {
        on = v < nrot;
        slot = part_slot<V>(on ? 0 : rot, on ? rot : rest, on ? v : v - nrot);
        if (!on && rest == 0) slot.at = 0, slot.over = V;
        from = on ? slot.at / 2 : 0;
      };
      // (a load of the wave then takes what lies side by side)
      vector(u, s[0], turn[0], angle[0]);
      vector(u + LPH, s[1], turn[1], angle[1]);
    } else {
      const uint32_t nrot = (half + V - 1) / V, nrest = ((rest + V - 1) / V + 1) / 2;
      const bool on = u < nrot;
      // (a unit past the last has the first's vectors of the rest, all of them the neighbour's)
      const uint32_t v = on ? u : u < nrot + nrest ? u - nrot : 2 * nrest;
      Slot p = part_slot<V>(on ? 0 : rot, on ? half : rest, v);
      Slot q = part_slot<V>(rot, rest, u < nrot + nrest ? u - nrot + nrest : 2 * nrest);
      angle[0] = on ? p.at : 0;
      angle[1] = 0;
      turn[0] = turn[1] = on;
      if (on) {
        q.at = PAIRS ? 2 * p.at + 1 : p.at + half;
        q.over = p.over;
        if (PAIRS) p.at *= 2;
      } else if (rest == 0) {
        p.at = q.at = 0;
        p.over = q.over = V;
      }
      s[0] = p;
      s[1] = q;
    }
  }
};
// Units of a head.
template <int V> uint32_t head_units(uint32_t dim, uint32_t rot, bool pairs) {
  const uint32_t rest = (dim - rot + V - 1) / V;
  if (pairs && V > 1) return ((rot + V - 1) / V + rest + 1) / 2;
  return (rot / 2 + V - 1) / V + (rest + 1) / 2;
}

// ---- V elements ------------------------------------------------------------------------
template <int T, int V> struct Raw { u32x4 v; };
template <int T> struct Raw<T, 1> { float v; };
template <int T, int V> __device__ __forceinline__ Raw<T, V> load_v(const void* p, uint64_t i) {
  Raw<T, V> r;
  if constexpr (V == 1) r.v = load_elem<T>(p, i);
  else r.v = *reinterpret_cast<const u32x4_any*>(at<T>(p, i));
  return r;
}
template <int T, int V> __device__ __forceinline__ void get_v(const Raw<T, V>& r, float* x) {
  if constexpr (V == 1) x[0] = r.v;
  else decode16<T>(r.v, x);
}
template <int T, int V> __device__ __forceinline__ void round_v(float* x) {
  if constexpr (V == 1) x[0] = to_f32<T>(from_f32<T>(x[0]));
  else decode16<T>(encode16<T>(x), x);
}
template <int T, int V> __device__ __forceinline__ void put_v(void* p, uint64_t i, const float* x) {
  if constexpr (V == 1) store_elem<T>(p, i, x[0]);
  else *reinterpret_cast<u32x4_any*>(at<T>(p, i)) = encode16<T>(x);
}
// N floats that lie anywhere.
template <int N> __device__ __forceinline__ void load_f32(const float* p, float* x) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) decode16<kF32>(load_raw<kF32>(p + 4 * k, 4), x + 4 * k);
  } else if constexpr (N == 2) {
    typedef f32x2 any __attribute__((aligned(4)));
    const f32x2 v = *reinterpret_cast<const any*>(p);
    x[0] = v.x;
    x[1] = v.y;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) x[k] = p[k];
  }
}
// ---- rotation -----------------------------------------------------------------------------
template <int V> struct Angles {
  float c[V], s[V];
};
// The angles of a position; NaN for one past the table.
template <int V, int LPH, bool PAIRS, bool FULL> __device__ __forceinline__ void load_angles(const QkArgs& a, const Unit<V, LPH, PAIRS, FULL>& u, int64_t pos, Angles<V>& r) {
  constexpr bool two = PAIRS && V > 1;
  constexpr int N = two ? V / 2 : V;
  const bool have = (uint64_t)pos < a.table_rows;
  const float* row = a.table + (have ? (uint64_t)pos * a.rot : 0);
#pragma unroll
  for (int k = 0; k < (two ? 2 : 1); ++k) {
    float c[N], s[N];
    load_f32<N>(row + u.angle[k], c);
    load_f32<N>(row + a.rot / 2 + u.angle[k], s);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      r.c[k * N + j] = have ? c[j] : __builtin_nanf("");
      r.s[k * N + j] = have ? s[j] : __builtin_nanf("");
    }
  }
}
// x: a lane's 2 V elements.
template <int V, int LPH, bool PAIRS, bool FULL, bool BACK> __device__ __forceinline__ void rotate(const Unit<V, LPH, PAIRS, FULL>& u, const Angles<V>& r, float* x) {
  auto turn = [](float& p, float& q, float c, float s, bool on) {
    if (BACK) s = -s;
    const float y = __builtin_fmaf(p, c, -(q * s)), z = __builtin_fmaf(q, c, p * s);
    p = FULL || on ? y : p;
    q = FULL || on ? z : q;
  };
  if constexpr (PAIRS && V > 1) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int j = 0; j < V / 2; ++j)
        turn(x[k * V + 2 * j], x[k * V + 2 * j + 1], r.c[k * (V / 2) + j], r.s[k * (V / 2) + j], u.turn[k]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) turn(x[j], x[V + j], r.c[j], r.s[j], u.turn[0]);
  }
}

template <int LPH> __device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = LPH / 2; m > 0; m >>= 1) v += __shfl_xor(v, m);
  return v;
}

// Streams: past the caches, for calls that move more than they hold.
// `base` is the wave's, `i` the lane's.
template <int T, int V, bool NT> __device__ __forceinline__ Raw<T, V> load_s(const void* p, uint64_t base, uint64_t i) {
  p = at<T>(p, base);
  if constexpr (V > 1 && NT) {
    Raw<T, V> r;
    r.v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(at<T>(p, i)));
    return r;
  } else {
    return load_v<T, V>(p, i);
  }
}
template <int T, int V, bool NT> __device__ __forceinline__ void put_s(void* p, uint64_t base, uint64_t i, const float* x) {
  p = at<T>(p, base);
  if constexpr (V > 1 && NT) __builtin_nontemporal_store(encode16<T>(x), reinterpret_cast<u32x4_any*>(at<T>(p, i)));
  else put_v<T, V>(p, i, x);
}

template <class X> __device__ __forceinline__ X of_kind(X q, X k, X v, uint32_t kind) { return kind == 0 ? q : kind == 1 ? k : v; }

// A wave's walk over its tokens and, of each, its iterations [first, end): 64 / LPH heads of
// one kind each.
struct Walk {
  uint64_t t;
  uint32_t i;
  __device__ __forceinline__ void next(uint32_t first, uint32_t end, uint64_t step) {
    if (++i == end) i = first, t += step;
  }
};
template <int LPH> struct Head {
  uint32_t kind, head, mine;  // first head of the iteration, and which of its heads is the lane's
  bool live;
  __device__ __forceinline__ Head(const QkArgs& a, const Walk& w) {
    constexpr uint32_t per = 64 / LPH;
    const uint32_t sub = (threadIdx.x & 63) / LPH;
    kind = w.i < a.its[1] ? 0u : w.i < a.its[2] ? 1u : 2u;
    head = (w.i - of_kind(0u, a.its[1], a.its[2], kind)) * per;
    const uint32_t left = of_kind(a.heads[0], a.heads[1], a.heads[2], kind) - head;
    live = sub < left;
    mine = live ? sub : left - 1;  // (a lane without a head reads the last one)
  }
  // First element of the iteration (wave-uniform) in the inputs,
  __device__ __forceinline__ uint64_t in(const QkArgs& a, const Walk& w) const {
    return w.t * a.ld_in + (uint64_t)(of_kind(0u, a.first_head[1], a.first_head[2], kind) + head) * a.dim;
  }
  // and in the queries, keys or values.
  __device__ __forceinline__ uint64_t out(const QkArgs& a, const Walk& w) const {
    return w.t * of_kind(a.ld_out[0], a.ld_out[1], a.ld_out[2], kind) + head * stride(a);
  }
  __device__ __forceinline__ uint64_t stride(const QkArgs& a) const { return of_kind(a.hs_out[0], a.hs_out[1], a.hs_out[2], kind); }
};

// The weights of the queries and keys, widened, in LDS: [2][512].
constexpr int kMaxDim = 512;
template <int T> __device__ __forceinline__ void stage_weights(const QkArgs& a, float* lds) {
  for (uint32_t i = threadIdx.x; i < 2 * a.dim; i += kThreads) {
    const uint32_t kind = i >= a.dim, c = kind ? i - a.dim : i;
    const void* w = a.w[kind];
    lds[kind * kMaxDim + c] = !w ? 1.0f : a.wf32 ? load_elem<kF32>(w, c) : load_elem<T>(w, c);
  }
  __syncthreads();
}
template <int V> __device__ __forceinline__ void staged(const float* lds, uint32_t kind, const Slot& s, float* w) {
#pragma unroll
  for (int j = 0; j < V; ++j) w[j] = lds[kind * kMaxDim + s.at + j];
}

// ---- forward --------------------------------------------------------------------------------
// What becomes of a lane's elements of the iteration that begins at `w`, summed and rounded.
template <int T, int V, int LPH, int K, bool PAIRS, bool FULL, bool NT, class Weights>
__device__ __forceinline__ void finish(const QkArgs& a, const Walk& w, const Head<LPH>& h, float inv, float (&x)[K][2 * V],
                                       const Angles<V> (&angles)[K], Weights&& weights) {
  constexpr int E = 2 * V;
  const int at_lane = threadIdx.x & (LPH - 1);
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float v = FULL || (uint32_t)(e % V) >= u.s[e / V].over ? x[k][e] : 0.0f;
      ss = __builtin_fmaf(v, v, ss);
    }
  }
  float rs = 0.0f;
  if (h.kind < 2) rs = 1.0f / __builtin_sqrtf(head_sum<LPH>(ss) * inv + a.eps);
  if (!h.live) return;
  void* const out = of_kind(a.out[0], a.out[1], a.out[2], h.kind);
  const uint64_t from = h.in(a, w), to = h.out(a, w), mine = h.mine * h.stride(a);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, at_lane + k * LPH);
    if (a.sum) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (FULL || u.s[s].over < (uint32_t)V) put_s<T, V, NT>(a.sum, from, h.mine * a.dim + u.s[s].at, x[k] + s * V);
    }
    if (!out) continue;
    if (h.kind < 2) {
      float wt[E];
      weights(k, u, wt);
#pragma unroll
      for (int e = 0; e < E; ++e) x[k][e] = x[k][e] * rs * wt[e];
      if (FULL || a.rot) rotate<V, LPH, PAIRS, FULL, false>(u, angles[k], x[k]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
      if (FULL || u.s[s].over < (uint32_t)V) put_s<T, V, NT>(out, to, mine + u.s[s].at, x[k] + s * V);
  }
}

// One iteration a wave, which is a workgroup: the dispatcher hands them out in order, so that HBM
// sees a narrow window that moves along, and all that a wave reads is asked for at once,
// but for the angles, whose place the position gives.  For several ranks (8 ranks of 4096 tokens of
// 48 heads of 128 bf16 and their sum 85 us, 112 where waves walk over tokens), and for few tokens.  G
// ranks' loads in flight: 8, 4 of up to 4, 2 of 2, as fewer registers leave room for more waves (2047
// tokens of 9 heads of 80 f16, 4 ranks, 9.9 us with 4 and 11.1 with 8; 4096 tokens of 48 heads of 128
// bf16, 2 ranks and their sum, 32 us with 2 or 4, 37 with 8).  K units a lane (1 but for heads without vectors).
constexpr int kAtOnce = 8;

// A lane's 2 V weights as they lie in memory, and widened.  No branch chooses between f32 and
// the data type before the loads are under way: 16-bit ones are loaded twice.
template <int T, int V> struct RawWeights {
  static constexpr int N = T == kF32 || V == 1 ? 1 : 2;
  typedef Raw<kF32, V == 1 ? 1 : 4> R;
  R r[2][N];
  __device__ __forceinline__ void load(const void* w, int wf32, const Slot* s) {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (V == 1) {
        r[k][0].v = T == kF32 || wf32 ? load_elem<kF32>(w, s[k].at) : load_elem<T>(w, s[k].at);
      } else {
        const uint8_t* p = (const uint8_t*)w + s[k].at * (T == kF32 || wf32 ? 4u : 2u);
#pragma unroll
        for (int h = 0; h < N; ++h) r[k][h].v = *reinterpret_cast<const u32x4_any*>(p + (h && wf32 ? 16 : 0));
      }
    }
  }
  __device__ __forceinline__ void get(int wf32, float* x) const {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if constexpr (V == 1) {
        x[k] = r[k][0].v;
      } else if (T == kF32 || wf32) {
#pragma unroll
        for (int h = 0; h < N; ++h) decode16<kF32>(r[k][h].v, x + k * V + 4 * h);
      } else {
        decode16<T>(r[k][0].v, x + k * V);
      }
    }
  }
};

template <int T, int V, int LPH, int K, int G, bool PAIRS, bool FULL, bool NT>
__global__ void __launch_bounds__(64) qk_fwd_k(QkArgs a) {
  constexpr int E = 2 * V;
  const int at_lane = threadIdx.x & (LPH - 1);
  const float inv = 1.0f / (float)a.dim;
  const uint32_t per = a.its[3], it = blockIdx.x % per;
  for (uint64_t t = blockIdx.x / per; t < a.tokens; t += gridDim.x / per) {
    const int64_t pos = a.positions ? a.positions[t] : (int64_t)t;
    if (a.positions && pos < 0) continue;
    const Walk w{t, it};
    const Head<LPH> h(a, w);
    const uint64_t from = h.in(a, w);
    Raw<T, V> raw[K][G][2];
    RawWeights<T, V> rw[K];
    // (values, and a kind without weights, load the other's and do not use them)
    const bool weighted = h.kind < 2 && (h.kind ? a.w[1] : a.w[0]);
    const void* wp = h.kind == 1 ? a.w[1] : a.w[0];
    if (!wp) wp = h.kind == 1 ? a.w[0] : a.w[1];
    auto fetch = [&](int r0) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const void* in = a.in[r0 + g < a.nranks ? r0 + g : 0];  // (past the last rank: the first again, not added)
#pragma unroll
          for (int s = 0; s < 2; ++s) raw[k][g][s] = load_s<T, V, NT>(in, from, h.mine * a.dim + u.s[s].at);
        }
      }
    };
    fetch(0);
    if (wp) {
#pragma unroll
      for (int k = 0; k < K; ++k) rw[k].load(wp, a.wf32, Unit<V, LPH, PAIRS, FULL>(a.dim, a.rot, at_lane + k * LPH).s);
    }
    Angles<V> angles[K];
    if ((FULL || a.rot) && h.kind < 2) {
#pragma unroll
      for (int k = 0; k < K; ++k) load_angles<V, LPH, PAIRS, FULL>(a, Unit<V, LPH, PAIRS, FULL>(a.dim, a.rot, at_lane + k * LPH), pos, angles[k]);
    }
    float x[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      get_v<T, V>(raw[k][0][0], x[k]);
      get_v<T, V>(raw[k][0][1], x[k] + V);
    }
    if constexpr (G > 1) {
      for (int r0 = 0; r0 < a.nranks; r0 += G) {
        if (r0) fetch(r0);
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int g = 0; g < G; ++g) {
            if (r0 + g > 0 && r0 + g < a.nranks) {
              float d[E];
              get_v<T, V>(raw[k][g][0], d);
              get_v<T, V>(raw[k][g][1], d + V);
#pragma unroll
              for (int e = 0; e < E; ++e) x[k][e] += d[e];
            }
          }
      }
#pragma unroll
      for (int k = 0; k < K; ++k) round_v<T, V>(x[k]), round_v<T, V>(x[k] + V);
    }
    finish<T, V, LPH, K, PAIRS, FULL, NT>(a, w, h, inv, x, angles, [&](int k, const Unit<V, LPH, PAIRS, FULL>&, float* wt) {
      if (weighted) {
        rw[k].get(a.wf32, wt);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) wt[e] = 1.0f;
      }
    });
  }
}

// Many tokens of one rank: a wave takes all heads of a token in turn, its units, addresses and
// angles worked out once, and asks for the next iteration's elements before it works on the
// present one's.  16384 tokens of 48 heads of 128 bf16: 72 us, 5.6 TB/s; the above
// 84 (96 elements a head 82 and 86; where half of 128 rotate 92 and 87; 8192 tokens f32 77 and 71).
template <int T, int V, int LPH, bool PAIRS, bool FULL>
__global__ void __launch_bounds__(kThreads, 4) qk_walk_k(QkArgs a) {
  __shared__ float weights[2 * kMaxDim];
  const int at_lane = threadIdx.x & (LPH - 1);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float inv = 1.0f / (float)a.dim;
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, at_lane);
  Raw<T, V> now[2], next[2];
  auto fetch = [&](const Walk& w) __attribute__((always_inline)) {
    const Head<LPH> h(a, w);
    const uint64_t from = h.in(a, w);
#pragma unroll
    for (int s = 0; s < 2; ++s) next[s] = load_s<T, V, true>(a.in[0], from, h.mine * a.dim + u.s[s].at);
  };
  auto position = [&](uint64_t t) { return a.positions ? a.positions[t] : (int64_t)t; };
  Walk w{(uint64_t)blockIdx.x * kWaves + wave, 0};
  int64_t pos = 0;
  if (w.t < a.tokens) {
    pos = position(w.t);
    if (pos >= 0) fetch(w);
  }
  stage_weights<T>(a, weights);
  Angles<V> angles[1];
  for (bool fresh = true; w.t < a.tokens;) {
    now[0] = next[0];
    now[1] = next[1];
    if (fresh && (FULL || a.rot) && pos >= 0) load_angles<V, LPH, PAIRS, FULL>(a, u, pos, angles[0]);
    const Walk cur = w;
    const int64_t cur_pos = pos;
    w.next(0, a.its[3], step);
    fresh = w.t != cur.t;
    if (w.t < a.tokens) {
      if (fresh) pos = position(w.t);
      if (pos >= 0) fetch(w);
    }
    if (cur_pos < 0) continue;
    const Head<LPH> h(a, cur);
    float x[1][2 * V];
    get_v<T, V>(now[0], x[0]);
    get_v<T, V>(now[1], x[0] + V);
    finish<T, V, LPH, 1, PAIRS, FULL, true>(a, cur, h, inv, x, angles, [&](int, const Unit<V, LPH, PAIRS, FULL>& at, float* wt) {
      staged<V>(weights, h.kind, at.s[0], wt);
      staged<V>(weights, h.kind, at.s[1], wt + V);
    });
  }
}

// ---- backward -------------------------------------------------------------------------------
// The weights' gradients of a lane's elements stay in registers over all of its tokens and
// heads; a workgroup's are joined in a fixed order and written once.
template <int T, int V, int LPH, int K, bool PAIRS, bool FULL, bool NT>
__global__ void __launch_bounds__(kThreads) qk_bwd_k(QkArgs a) {
  constexpr int E = 2 * V;
  __shared__ float weights[2 * kMaxDim];
  __shared__ float lds[kWaves][2 * K * E][LPH];
  const int lane = threadIdx.x & 63, at_lane = lane & (LPH - 1);
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t first = blockIdx.y * a.chunk, end = first + a.chunk < a.its[3] ? first + a.chunk : a.its[3];
  const float inv = 1.0f / (float)a.dim;
  const uint64_t step = (uint64_t)gridDim.x * kWaves;
  typedef Raw<T, V> R;
  R now_d[K][2], now_h[K][2], next_d[K][2], next_h[K][2];
  auto position = [&](uint64_t t) { return a.positions ? a.positions[t] : (int64_t)t; };
  auto grads = [&](uint32_t kind) { return of_kind(a.out[0], a.out[1], a.out[2], kind); };
  auto fetch = [&](const Walk& w) __attribute__((always_inline)) {
    const Head<LPH> h(a, w);
    // (without a branch: where there is no gradient the row itself is loaded twice, of the
    // values the gradient, and one of the two is not used)
    const void* d = grads(h.kind);
    const uint64_t base = h.in(a, w), step = h.mine * a.dim;
    const uint64_t from = d ? h.out(a, w) : base, mine = d ? h.mine * h.stride(a) : step;
    if (!d) d = a.h;
    const void* row = h.kind < 2 ? a.h : d;
    const uint64_t in = h.kind < 2 ? base : from, at_in = h.kind < 2 ? step : mine;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        next_d[k][s] = load_s<T, V, NT>(d, from, mine + u.s[s].at);
        next_h[k][s] = load_s<T, V, NT>(row, in, at_in + u.s[s].at);
      }
    }
  };
  float dw[2][K][E];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) dw[kind][k][e] = 0.0f;
  Walk w{(uint64_t)blockIdx.x * kWaves + wave, first};
  if (end <= first) w.t = a.tokens;
  int64_t pos = 0;
  if (w.t < a.tokens) {
    pos = position(w.t);
    if (pos >= 0) fetch(w);
  }
  // (the first token's before the weights, whose barrier waits for both)
  Angles<V> angles[K];
  auto turn = [&]() __attribute__((always_inline)) {
    if (!(FULL || a.rot) || pos < 0 || first >= a.its[2]) return;
#pragma unroll
    for (int k = 0; k < K; ++k) load_angles<V, LPH, PAIRS, FULL>(a, Unit<V, LPH, PAIRS, FULL>(a.dim, a.rot, at_lane + k * LPH), pos, angles[k]);
  };
  if (w.t < a.tokens) turn();
  stage_weights<T>(a, weights);
  for (bool fresh = false; w.t < a.tokens;) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int s = 0; s < 2; ++s) now_d[k][s] = next_d[k][s], now_h[k][s] = next_h[k][s];
    if (fresh) turn();
    const Walk cur = w;
    const int64_t cur_pos = pos;
    w.next(first, end, step);
    fresh = w.t != cur.t;
    if (w.t < a.tokens) {
      if (fresh) pos = position(w.t);
      if (pos >= 0) fetch(w);
    }
    const Head<LPH> h(a, cur);
    const bool none = cur_pos < 0 || !grads(h.kind);
    float u[K][E], x[K][E], g[K][E];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (none) {
#pragma unroll
          for (int j = 0; j < V; ++j) u[k][s * V + j] = 0.0f;
        } else {
          get_v<T, V>(now_d[k][s], u[k] + s * V);
        }
      }
    if (h.kind < 2 && !none) {
      float ss = 0.0f, sg = 0.0f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const Unit<V, LPH, PAIRS, FULL> at(a.dim, a.rot, at_lane + k * LPH);
        get_v<T, V>(now_h[k][0], x[k]);
        get_v<T, V>(now_h[k][1], x[k] + V);
        if (FULL || a.rot) rotate<V, LPH, PAIRS, FULL, true>(at, angles[k], u[k]);
        float wt[E];
        staged<V>(weights, h.kind, at.s[0], wt);
        staged<V>(weights, h.kind, at.s[1], wt + V);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float xe = FULL || (uint32_t)j >= at.s[h].over ? x[k][h * V + j] : 0.0f;
            ss = __builtin_fmaf(xe, xe, ss);
            g[k][h * V + j] = u[k][h * V + j] * wt[h * V + j];
            sg = __builtin_fmaf(FULL || (uint32_t)j >= at.s[h].over ? g[k][h * V + j] : 0.0f, xe, sg);
          }
      }
      const float rs = 1.0f / __builtin_sqrtf(head_sum<LPH>(ss) * inv + a.eps);
      const float c = head_sum<LPH>(sg) * inv * rs * rs;
      auto add = [&](float (&to)[K][E]) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < E; ++e) to[k][e] = __builtin_fmaf(u[k][e], x[k][e] * rs, to[k][e]);
      };
      // (a lane without a head adds nothing, not even zero times the last head's elements, which
      // it holds: they may be infinite)
      if (h.live) {
        if (h.kind == 0) add(dw[0]);
        else add(dw[1]);
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) u[k][e] = __builtin_fmaf(x[k][e], -c, g[k][e]) * rs;
    }
    if (!h.live || !a.dsum) continue;
    const uint64_t to = h.in(a, cur);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const Unit<V, LPH, PAIRS, FULL> at(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        if (FULL || at.s[s].over < (uint32_t)V) put_s<T, V, NT>(a.dsum, to, h.mine * a.dim + at.s[s].at, u[k] + s * V);
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float v = dw[kind][k][e];
#pragma unroll
        for (int m = LPH; m < 64; m <<= 1) v += __shfl_xor(v, m);
        if (lane < LPH) lds[wave][(kind * K + k) * E + e][at_lane] = v;
      }
  __syncthreads();
  const uint64_t group = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < 2 * K * E * LPH; i += kThreads) {
    const int l = i % LPH, row = i / LPH, e = row % E, k = row / E % K, kind = row / (E * K);
    const Unit<V, LPH, PAIRS, FULL> u(a.dim, a.rot, l + k * LPH);
    const Slot s = e < V ? u.s[0] : u.s[1];
    if ((uint32_t)(e % V) < s.over) continue;
    float v = lds[0][row][l];
#pragma unroll
    for (int m = 1; m < kWaves; ++m) v += lds[m][row][l];
    a.partial[(group * 2 + kind) * a.dim + s.at + e % V] = v;
  }
}

// The workgroups' sums of the weights' gradients, in order (64 strided chains, then those
// in order), rounded once.  16 columns a workgroup; blockIdx.y 0 is the queries', 1 the keys'.
constexpr int kJoinCols = 16, kJoinChains = 64;
template <int T> __global__ void __launch_bounds__(kJoinCols * kJoinChains) qk_join_k(QkArgs a, uint32_t groups) {
  __shared__ float lds[kJoinChains][kJoinCols];
  void* to = a.dw[blockIdx.y];
  if (!to) return;
  const uint32_t x = threadIdx.x % kJoinCols, chain = threadIdx.x / kJoinCols, c = blockIdx.x * kJoinCols + x;
  float s = 0.0f;
  if (c < a.dim) {
    const float* p = a.partial + (uint64_t)blockIdx.y * a.dim + c;
#pragma unroll 4
    for (uint32_t g = chain; g < groups; g += kJoinChains) s += p[(uint64_t)g * 2 * a.dim];
  }
  lds[chain][x] = s;
  __syncthreads();
  if (chain || c >= a.dim) return;
#pragma unroll
  for (int k = 1; k < kJoinChains; ++k) s += lds[k][x];
  if (a.wf32) store_elem<kF32>(to, c, s);
  else store_elem<T>(to, c, s);
}

// ---- launches -------------------------------------------------------------------------------
// A backward's grid: as many workgroups as the card holds at once (3 a CU, of which
// every wave then has as many tokens as the others: 16384 tokens of 48 heads of 128 bf16
// 111 us, 128 with 1024 and 143 with 256; heads of 80 that rotate 32 in pairs 101, 115 and 166; 12 heads of
// 512 f32 204, 210 and 264), few tokens' heads dealt out over more of them.
struct Shape {
  uint32_t x, y, chunk;
};
constexpr uint32_t kFill = 768;
Shape shape_of(uint64_t tokens, uint32_t its) {
  const uint64_t blocks = (tokens + kWaves - 1) / kWaves;
  uint64_t x = blocks < kFill ? blocks : kFill;
  if (x < 1) x = 1;
  uint64_t y = kFill / x;
  if (y < 1) y = 1;
  if (y > its) y = its;
  const uint32_t chunk = (uint32_t)((its + y - 1) / y);
  return {(uint32_t)x, (its + chunk - 1) / chunk, chunk};
}

// Calls that move more than the 256 MiB of the Infinity Cache go past the caches (48 heads of 128
// bf16, one rank: 384 MiB forward 72 us, 84 through them, backward 79 and 86; 192 MiB that the cache still
// holds forward 38 us, 35 through it, backward 46 and 42; 2 and 8 ranks alike).
constexpr uint64_t kCacheBytes = 256ull << 20;
// Elements of a token that a call moves: `reads` times its heads, and those of what it has of
// the queries, keys and values.
uint64_t token_moves(const QkArgs& a, uint64_t reads) {
  uint64_t heads = reads * (a.heads[0] + a.heads[1] + (uint64_t)(a.skip_values ? 0 : a.heads[2]));
  for (int k = 0; k < 3; ++k) heads += a.out[k] && !(k == 2 && a.skip_values) ? a.heads[k] : 0;
  return heads * a.dim;
}
constexpr uint64_t kMaxWaves = 1u << 24, kMaxBlocks = 4096;  // tokens past them are walked in strides

// Lanes a head, units a lane and elements a vector.
struct Layout {
  int v, lph, k;
};
template <int T> Layout layout_of(uint32_t dim, uint32_t rot, bool pairs) {
  constexpr uint32_t V = Vec<T>::VW;
  const uint32_t turn = pairs ? rot : rot / 2, rest = dim - rot;
  if ((rot == 0 || turn >= V) && (rest == 0 || rest >= V)) {
    const uint32_t n = head_units<V>(dim, rot, pairs);
    for (int lph = 4; lph <= 64; lph *= 2)
      if (n <= (uint32_t)lph) return {(int)V, lph, 1};
  }
  const uint32_t n = head_units<1>(dim, rot, pairs);
  return n <= 16 ? Layout{1, 16, 1} : n <= 64 ? Layout{1, 64, 1} : Layout{1, 64, 4};
}
int lanes_of(const QkArgs& a, int t) {
  const bool p = a.pairs;
  return (t == kF32 ? layout_of<kF32>(a.dim, a.rot, p) : layout_of<kF16>(a.dim, a.rot, p)).lph;
}

// Fills in what depends on the lanes a head takes.
void prepare(QkArgs& a, int t) {
  const uint32_t per = 64 / lanes_of(a, t);
  a.its[0] = a.first_head[0] = 0;
  for (int k = 0; k < 3; ++k) {
    a.its[k + 1] = a.its[k] + (a.heads[k] + per - 1) / per;
    if (k < 2) a.first_head[k + 1] = a.first_head[k] + a.heads[k];
  }
  if (a.skip_values) a.its[3] = a.its[2];
}

template <int T, bool PAIRS, class Go> void typed(const Layout& l, Go&& go) {
  constexpr int V = Vec<T>::VW;
  auto v = [&](auto vv, auto lph, auto k) { go(vv, lph, k, std::bool_constant<PAIRS>()); };
#define MRR_LANES(vv, lph, kk) v(std::integral_constant<int, vv>(), std::integral_constant<int, lph>(), std::integral_constant<int, kk>())
  if (l.v == 1) {
    if (l.lph == 16) MRR_LANES(1, 16, 1);
    else if (l.k == 1) MRR_LANES(1, 64, 1);
    else MRR_LANES(1, 64, 4);
  } else if (l.lph == 4) {
    MRR_LANES(V, 4, 1);
  } else if (l.lph == 8) {
    MRR_LANES(V, 8, 1);
  } else if (l.lph == 16) {
    MRR_LANES(V, 16, 1);
  } else if (l.lph == 32) {
    MRR_LANES(V, 32, 1);
  } else {
    MRR_LANES(V, 64, 1);
  }
#undef MRR_LANES
}

// Whether a head is FULL, and the call one that goes past the caches.
template <class V, class L, class Go> void shaped(V, L, const QkArgs& a, bool stream, Go&& go) {
  constexpr std::true_type yes;
  constexpr std::false_type no;
  if constexpr (V::value > 1) {
    if (a.rot == a.dim && a.dim == 2u * V::value * L::value) stream ? go(yes, yes) : go(yes, no);
    else stream ? go(no, yes) : go(no, no);
  } else {
    go(no, no);
  }
}

template <int T> void fwd(const QkArgs& a, hipStream_t s) {
  const uint64_t bytes = a.tokens * token_moves(a, a.nranks + (a.sum ? 1 : 0)) * Ty<T>::size;
  auto go = [&](auto v, auto lph, auto k, auto pairs) {
    auto full = [&](auto f, auto nt) {
      if constexpr (nt) {
        if (a.nranks == 1) {
          const uint64_t blocks = (a.tokens + kWaves - 1) / kWaves;
          hipLaunchKernelGGL((qk_walk_k<T, v, lph, pairs, f>), dim3((uint32_t)(blocks < kMaxBlocks ? blocks : kMaxBlocks)), dim3(kThreads), 0, s, a);
          return;
        }
      }
      const uint64_t rows = a.tokens < kMaxWaves / a.its[3] ? a.tokens : kMaxWaves / a.its[3];
      const dim3 grid((uint32_t)(a.its[3] * rows));
      if (a.nranks > kAtOnce / 2) hipLaunchKernelGGL((qk_fwd_k<T, v, lph, k, kAtOnce, pairs, f, nt>), grid, dim3(64), 0, s, a);
      else if (a.nranks > 2) hipLaunchKernelGGL((qk_fwd_k<T, v, lph, k, kAtOnce / 2, pairs, f, nt>), grid, dim3(64), 0, s, a);
      else if (a.nranks > 1) hipLaunchKernelGGL((qk_fwd_k<T, v, lph, k, 2, pairs, f, nt>), grid, dim3(64), 0, s, a);
      else if constexpr (!nt) hipLaunchKernelGGL((qk_fwd_k<T, v, lph, k, 1, pairs, f, false>), grid, dim3(64), 0, s, a);
    };
    shaped(v, lph, a, bytes > kCacheBytes, full);
  };
  const Layout l = layout_of<T>(a.dim, a.rot, a.pairs);
  if (a.pairs) typed<T, true>(l, go);
  else typed<T, false>(l, go);
}

template <int T> void bwd(const QkArgs& a, const Shape& g, hipStream_t s) {
  // (the sum, of the queries and keys alone, its gradient, and the outputs')
  const uint64_t sums = (a.heads[0] + (uint64_t)a.heads[1]) * a.dim;
  const uint64_t bytes = a.tokens * (sums + token_moves(a, a.dsum ? 1 : 0)) * Ty<T>::size;
  auto go = [&](auto v, auto lph, auto k, auto pairs) {
    auto full = [&](auto f, auto nt) {
      hipLaunchKernelGGL((qk_bwd_k<T, v, lph, k, pairs, f, nt>), dim3(g.x, g.y), dim3(kThreads), 0, s, a);
    };
    shaped(v, lph, a, bytes > kCacheBytes, full);
  };
  const Layout l = layout_of<T>(a.dim, a.rot, a.pairs);
  if (a.pairs) typed<T, true>(l, go);
  else typed<T, false>(l, go);
  if (a.partial)
    hipLaunchKernelGGL(qk_join_k<T>, dim3((a.dim + kJoinCols - 1) / kJoinCols, 2), dim3(kJoinCols * kJoinChains), 0, s, a, g.x * g.y);
}

}  // namespace

uint64_t qk_bwd_groups() { return kFill; }

hipError_t launch_qk_fwd(QkArgs a, int t, hipStream_t s) {
  prepare(a, t);
  if (a.its[3] == 0) return hipSuccess;
  if (t == kF32) fwd<kF32>(a, s);
  else if (t == kF16) fwd<kF16>(a, s);
  else fwd<kBF16>(a, s);
  return hipGetLastError();
}

hipError_t launch_qk_bwd(QkArgs a, int t, hipStream_t s) {
  prepare(a, t);
  const Shape g = shape_of(a.tokens, a.its[3] ? a.its[3] : 1);
  a.chunk = g.chunk;
  if (t == kF32) bwd<kF32>(a, g, s);
  else if (t == kF16) bwd<kF16>(a, g, s);
  else bwd<kBF16>(a, g, s);
  return hipGetLastError();
}

}  // namespace mrr
