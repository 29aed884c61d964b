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
// halves of the same pairs where halves rotate together and neighbours where neighbours do,
// so that no pair crosses lanes; 64 / LPH heads of a token share a wave.  A wave takes all
// heads of a token in turn, with the token's cosines and sines and the weights in
// registers; few tokens are dealt out by heads as well.  Sums are f32; each output is rounded
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
template <int V, bool PAIRS> struct Unit {
  Slot s[2];
  bool turn[2];
  uint32_t angle[2];  // PAIRS, V > 1: V / 2 angles for each vector; else V for both, the first
  __device__ __forceinline__ Unit(uint32_t dim, uint32_t rot, uint32_t u) {
    const uint32_t half = rot / 2, rest = dim - rot;
    if constexpr (PAIRS && V > 1) {
      const uint32_t nrot = (rot + V - 1) / V;
      auto vector = [&](uint32_t v, Slot& slot, bool& on, uint32_t& from) {
        on = v < nrot;
        slot = part_slot<V>(on ? 0 : rot, on ? rot : rest, on ? v : v - nrot);
        if (!on && rest == 0) slot.at = 0, slot.over = V;
        from = on ? slot.at / 2 : 0;
      };
      vector(2 * u, s[0], turn[0], angle[0]);
      vector(2 * u + 1, s[1], turn[1], angle[1]);
    } else {
      const uint32_t nrot = (half + V - 1) / V;
      const bool on = u < nrot;
      Slot p = part_slot<V>(on ? 0 : rot, on ? half : rest, on ? u : 2 * (u - nrot));
      Slot q = part_slot<V>(rot, rest, 2 * (u - nrot) + 1);
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
// A lane's 2 V weights, f32 or of the data type; 1 without.
template <int T, int V> __device__ __forceinline__ void load_weights(const void* w, int wf32, const Slot* s, float* x) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (!w) {
#pragma unroll
      for (int j = 0; j < V; ++j) x[k * V + j] = 1.0f;
    } else if (T == kF32 || wf32) {
      load_f32<V>((const float*)w + s[k].at, x + k * V);
    } else {
      get_v<T, V>(load_v<T, V>(w, s[k].at), x + k * V);
    }
  }
}

// ---- rotation -----------------------------------------------------------------------------
template <int V> struct Angles {
  float c[V], s[V];
};
// The angles of a position; NaN for one past the table.
template <int V, bool PAIRS> __device__ __forceinline__ void load_angles(const QkArgs& a, const Unit<V, PAIRS>& u, int64_t pos, Angles<V>& r) {
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
template <int V, bool PAIRS, bool BACK> __device__ __forceinline__ void rotate(const Unit<V, PAIRS>& u, const Angles<V>& r, float* x) {
  auto turn = [](float& p, float& q, float c, float s, bool on) {
    if (BACK) s = -s;
    const float y = __builtin_fmaf(p, c, -(q * s)), z = __builtin_fmaf(q, c, p * s);
    p = on ? y : p;
    q = on ? z : q;
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

// ---- forward --------------------------------------------------------------------------------
// K units a lane (1 but for heads without vectors).  A wave takes `chunk` of a token's
// iterations, each of 64 / LPH heads of one kind.
template <int T, int V, int LPH, int K, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_fwd_k(QkArgs a) {
  constexpr int HPW = 64 / LPH, E = 2 * V;
  const int lane = threadIdx.x & 63, sub = lane / LPH;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t first = blockIdx.y * a.chunk, end = first + a.chunk < a.its[3] ? first + a.chunk : a.its[3];
  const float inv = 1.0f / (float)a.dim;
  for (uint64_t t = (uint64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (uint64_t)gridDim.x * kWaves) {
    const int64_t pos = a.positions ? a.positions[t] : (int64_t)t;
    if (pos < 0) continue;
    Angles<V> angles[K];
    if (a.rot && first < a.its[2]) {
#pragma unroll
      for (int k = 0; k < K; ++k) load_angles<V, PAIRS>(a, Unit<V, PAIRS>(a.dim, a.rot, (lane % LPH) + k * LPH), pos, angles[k]);
    }
#pragma unroll
    for (int kind = 0; kind < 3; ++kind) {
      const uint32_t i0 = first > a.its[kind] ? first : a.its[kind], i1 = end < a.its[kind + 1] ? end : a.its[kind + 1];
      if (i0 >= i1) continue;
      float w[K][E];
      if (kind < 2) {
#pragma unroll
        for (int k = 0; k < K; ++k)
          load_weights<T, V>(a.w[kind], a.wf32, Unit<V, PAIRS>(a.dim, a.rot, (lane % LPH) + k * LPH).s, w[k]);
      }
      for (uint32_t i = i0; i < i1; ++i) {
        const uint32_t mine = (i - a.its[kind]) * HPW + sub;
        const bool live = mine < a.heads[kind];
        const uint32_t head = live ? mine : a.heads[kind] - 1;
        const uint64_t from = t * a.ld_in + (uint64_t)(a.first_head[kind] + head) * a.dim;
        float x[K][E];
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Unit<V, PAIRS> u(a.dim, a.rot, (lane % LPH) + k * LPH);
#pragma unroll
          for (int e = 0; e < E; ++e) x[k][e] = -0.0f;  // (the first sum is then exactly x_0)
#pragma unroll 4
          for (int r = 0; r < a.nranks; ++r) {
            float d[E];
            const Raw<T, V> p = load_v<T, V>(a.in[r], from + u.s[0].at), q = load_v<T, V>(a.in[r], from + u.s[1].at);
            get_v<T, V>(p, d);
            get_v<T, V>(q, d + V);
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] += d[e];
          }
          round_v<T, V>(x[k]);
          round_v<T, V>(x[k] + V);
#pragma unroll
          for (int e = 0; e < E; ++e) ss += (uint32_t)(e % V) >= u.s[e / V].over ? x[k][e] * x[k][e] : 0.0f;
        }
        float rs = 0.0f;
        if (kind < 2) rs = 1.0f / __builtin_sqrtf(head_sum<LPH>(ss) * inv + a.eps);
        if (!live) continue;
        const uint64_t to = t * a.ld_out[kind] + head * a.hs_out[kind];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Unit<V, PAIRS> u(a.dim, a.rot, (lane % LPH) + k * LPH);
          if (a.sum) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (u.s[h].over < (uint32_t)V) put_v<T, V>(a.sum, from + u.s[h].at, x[k] + h * V);
          }
          if (kind < 2) {
#pragma unroll
            for (int e = 0; e < E; ++e) x[k][e] = x[k][e] * rs * w[k][e];
            if (a.rot) rotate<V, PAIRS, false>(u, angles[k], x[k]);
          }
          if (a.out[kind]) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (u.s[h].over < (uint32_t)V) put_v<T, V>(a.out[kind], to + u.s[h].at, x[k] + h * V);
          }
        }
      }
    }
  }
}

// ---- backward -------------------------------------------------------------------------------
// The weights' gradients of a lane's elements stay in registers over all of its tokens and
// heads; a workgroup's are joined in a fixed order and written once.
template <int T, int V, int LPH, int K, bool PAIRS>
__global__ void __launch_bounds__(kThreads) qk_bwd_k(QkArgs a) {
  constexpr int HPW = 64 / LPH, E = 2 * V;
  __shared__ float lds[kWaves][2 * K * E][LPH];
  const int lane = threadIdx.x & 63, sub = lane / LPH, at_lane = lane % LPH;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t first = blockIdx.y * a.chunk, end = first + a.chunk < a.its[3] ? first + a.chunk : a.its[3];
  const float inv = 1.0f / (float)a.dim;
  float dw[2][K][E];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < E; ++e) dw[kind][k][e] = 0.0f;
  for (uint64_t t = (uint64_t)blockIdx.x * kWaves + wave; t < a.tokens; t += (uint64_t)gridDim.x * kWaves) {
    const int64_t pos = a.positions ? a.positions[t] : (int64_t)t;
    Angles<V> angles[K];
    if (a.rot && pos >= 0 && first < a.its[2]) {
#pragma unroll
      for (int k = 0; k < K; ++k) load_angles<V, PAIRS>(a, Unit<V, PAIRS>(a.dim, a.rot, at_lane + k * LPH), pos, angles[k]);
    }
#pragma unroll
    for (int kind = 0; kind < 3; ++kind) {
      const uint32_t i0 = first > a.its[kind] ? first : a.its[kind], i1 = end < a.its[kind + 1] ? end : a.its[kind + 1];
      if (i0 >= i1) continue;
      float w[K][E];
      if (kind < 2 && a.dsum) {
#pragma unroll
        for (int k = 0; k < K; ++k) load_weights<T, V>(a.w[kind], a.wf32, Unit<V, PAIRS>(a.dim, a.rot, at_lane + k * LPH).s, w[k]);
      }
      for (uint32_t i = i0; i < i1; ++i) {
        const uint32_t mine = (i - a.its[kind]) * HPW + sub;
        const bool live = mine < a.heads[kind];
        const uint32_t head = live ? mine : a.heads[kind] - 1;
        const uint64_t in = t * a.ld_in + (uint64_t)(a.first_head[kind] + head) * a.dim;
        const uint64_t from = t * a.ld_out[kind] + head * a.hs_out[kind];
        float u[K][E], x[K][E], ss = 0.0f, sg = 0.0f;
        const bool none = pos < 0 || !a.out[kind];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Unit<V, PAIRS> at(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (none) {
#pragma unroll
              for (int j = 0; j < V; ++j) u[k][h * V + j] = 0.0f;
            } else {
              get_v<T, V>(load_v<T, V>(a.out[kind], from + at.s[h].at), u[k] + h * V);
            }
          }
          if (kind < 2 && !none) {
#pragma unroll
            for (int h = 0; h < 2; ++h) get_v<T, V>(load_v<T, V>(a.h, in + at.s[h].at), x[k] + h * V);
            if (a.rot) rotate<V, PAIRS, true>(at, angles[k], u[k]);
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const bool counts = (uint32_t)(e % V) >= at.s[e / V].over;
              ss += counts ? x[k][e] * x[k][e] : 0.0f;
              if (a.dsum) sg += counts ? u[k][e] * w[k][e] * x[k][e] : 0.0f;
            }
          }
        }
        if (kind < 2 && !none) {
          const float rs = 1.0f / __builtin_sqrtf(head_sum<LPH>(ss) * inv + a.eps);
          if (live) {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int e = 0; e < E; ++e) dw[kind < 2 ? kind : 0][k][e] = __builtin_fmaf(u[k][e], x[k][e] * rs, dw[kind < 2 ? kind : 0][k][e]);
          }
          if (a.dsum) {
            const float c = head_sum<LPH>(sg) * inv * rs * rs;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
              for (int e = 0; e < E; ++e) u[k][e] = (u[k][e] * w[k][e] - x[k][e] * c) * rs;
          }
        }
        if (!live || !a.dsum) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const Unit<V, PAIRS> at(a.dim, a.rot, at_lane + k * LPH);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (at.s[h].over < (uint32_t)V) put_v<T, V>(a.dsum, in + at.s[h].at, u[k] + h * V);
        }
      }
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
        if (sub == 0) lds[wave][(kind * K + k) * E + e][at_lane] = v;
      }
  __syncthreads();
  const uint64_t group = (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = threadIdx.x; i < 2 * K * E * LPH; i += kThreads) {
    const int l = i % LPH, row = i / LPH, e = row % E, k = row / E % K, kind = row / (E * K);
    const Unit<V, PAIRS> u(a.dim, a.rot, l + k * LPH);
    const Slot s = e < V ? u.s[0] : u.s[1];
    if ((uint32_t)(e % V) < s.over) continue;
    float v = lds[0][row][l];
#pragma unroll
    for (int m = 1; m < kWaves; ++m) v += lds[m][row][l];
    a.partial[(group * 2 + kind) * a.dim + s.at + e % V] = v;
  }
}

// The workgroups' sums of the weights' gradients, in order (16 strided chains, then those
// in order), rounded once.  64 columns a workgroup; blockIdx.y 0 is the queries', 1 the keys'.
constexpr int kJoinCols = 64, kJoinChains = 16;
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
// A call's grid: waves for every token as long as the card has room, few tokens' heads dealt
// out over more of them.
struct Shape {
  uint32_t x, y, chunk;
};
constexpr uint32_t kFill = 1024;        // workgroups that give every SIMD some waves
constexpr uint32_t kBwdGroups = kFill;  // most of a backward, whose sums are joined
Shape shape_of(uint64_t tokens, uint32_t its, uint64_t most) {
  const uint64_t blocks = (tokens + kWaves - 1) / kWaves;
  uint64_t x = blocks < most ? blocks : most;
  if (x < 1) x = 1;
  uint64_t y = kFill / x;
  if (y < 1) y = 1;
  if (y > its) y = its;
  const uint32_t chunk = (uint32_t)((its + y - 1) / y);
  return {(uint32_t)x, (its + chunk - 1) / chunk, chunk};
}

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
Shape prepare(QkArgs& a, int t, uint64_t most) {
  const uint32_t per = 64 / lanes_of(a, t);
  a.its[0] = a.first_head[0] = 0;
  for (int k = 0; k < 3; ++k) {
    a.its[k + 1] = a.its[k] + (a.heads[k] + per - 1) / per;
    if (k < 2) a.first_head[k + 1] = a.first_head[k] + a.heads[k];
  }
  if (a.skip_values) a.its[3] = a.its[2];
  const Shape s = shape_of(a.tokens, a.its[3] ? a.its[3] : 1, most);
  a.chunk = s.chunk;
  return s;
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

template <int T> void fwd(const QkArgs& a, const Shape& g, hipStream_t s) {
  auto go = [&](auto v, auto lph, auto k, auto pairs) {
    hipLaunchKernelGGL((qk_fwd_k<T, v, lph, k, pairs>), dim3(g.x, g.y), dim3(kThreads), 0, s, a);
  };
  const Layout l = layout_of<T>(a.dim, a.rot, a.pairs);
  if (a.pairs) typed<T, true>(l, go);
  else typed<T, false>(l, go);
}

template <int T> void bwd(const QkArgs& a, const Shape& g, hipStream_t s) {
  auto go = [&](auto v, auto lph, auto k, auto pairs) {
    hipLaunchKernelGGL((qk_bwd_k<T, v, lph, k, pairs>), dim3(g.x, g.y), dim3(kThreads), 0, s, a);
  };
  const Layout l = layout_of<T>(a.dim, a.rot, a.pairs);
  if (a.pairs) typed<T, true>(l, go);
  else typed<T, false>(l, go);
  if (a.partial)
    hipLaunchKernelGGL(qk_join_k<T>, dim3((a.dim + kJoinCols - 1) / kJoinCols, 2), dim3(kJoinCols * kJoinChains), 0, s, a, g.x * g.y);
}

}  // namespace

uint64_t qk_bwd_groups() { return kBwdGroups; }

hipError_t launch_qk_fwd(QkArgs a, int t, hipStream_t s) {
  const Shape g = prepare(a, t, 1u << 20);
  if (a.its[3] == 0) return hipSuccess;
  if (t == kF32) fwd<kF32>(a, g, s);
  else if (t == kF16) fwd<kF16>(a, g, s);
  else fwd<kBF16>(a, g, s);
  return hipGetLastError();
}

hipError_t launch_qk_bwd(QkArgs a, int t, hipStream_t s) {
  const Shape g = prepare(a, t, kBwdGroups);
  if (t == kF32) bwd<kF32>(a, g, s);
  else if (t == kF16) bwd<kF16>(a, g, s);
  else bwd<kBF16>(a, g, s);
  return hipGetLastError();
}

}  // namespace mrr
