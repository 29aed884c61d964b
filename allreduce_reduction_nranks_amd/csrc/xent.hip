// xent.hip -- cross entropy of a linear layer whose vocabulary lies in N rank
// shards, without the logits in memory, and its gradient.
//
//   z[t][v] = sum over c of h[t][c] w[v][c]
//   lse[t]  = log(sum over v of exp(z[t][v])),  loss[t] = lse[t] - z[t][target[t]]
//
//   dz[t][v] = (exp(z[t][v] - lse[t]) - [v = target[t]]) dloss[t]
//   dh[t][c] = sum over v of dz[t][v] w[v][c],  dw[v][c] = sum over t of dz[t][v] h[t][c]
//
// The forward is one product whose tile epilogue reduces 128 logits of each token
// to (max, sum of exponentials); a join over those pairs gives lse.  Logits stay
// f32 in accumulators.  The backward computes the logits again, a piece of the
// vocabulary at a time, keeps that piece's dz in 16 bits and multiplies it with
// the piece's weights and with the hidden states: 3 products of 2 T V C
// operations, bound by the matrix units.
//
// Tokens without a loss are left out of the backward altogether: the others'
// hidden states are gathered first, so nothing in an ignored token's row (not
// even a NaN) reaches a gradient, and a batch pays for its counted tokens only.
//
// f32 operands are split into three bf16 parts, x = x1 + x2 + x3 exactly (8 bits each, with
// the signs; from 2^-102 on), and a product is the sum of the 6 products x_i y_j with i + j <= 4 in f32,
// smallest first.  What is left out is at most 2^-26 of |x y|, a quarter of an f32
// product's rounding.  bf16 has f32's exponents: no operand is scaled, so that no row's
// error depends on another row, nor on how a call is multiplied.  (Two f16 parts take three
// products and three quarters of the laid-out bytes, but hold 22 bits and need one scale for all
// of a tensor: with one row 10^8 times the others, those are off by 3e-4 of themselves.  1024 x
// 32000 x 1024 forward: 394 us, 170 TFLOP/s; an f32 product's rate is 75.)  An infinite x stays
// whole in x1, and the five smaller products read a copy of x1 that has 0 in its place (else
// infinity would meet the zeros and the signs of the other operand's smaller parts and give
// NaN): a row of -inf weights keeps its probability 0.
#include "mrr_gemm.hpp"
#include "mrr_internal.hpp"
#include "mrr_ops.hpp"
#include "mrr_rows.hpp"

namespace mrr {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kPlanes = 4, kSegs = 6;  // x1, x2, x3, x1 without infinities

// Plane of A and of B in segment s of an f32 product.
__device__ __forceinline__ uint32_t seg_a(uint32_t s) { return (0x031132u >> (4 * s)) & 3u; }
__device__ __forceinline__ uint32_t seg_b(uint32_t s) { return (0x013123u >> (4 * s)) & 3u; }

// ---- layouts of operands ---------------------------------------------------------
// A product reads rows of a multiple of 64 elements, 16-byte aligned, zeros past
// the last column.  What does not lie so, and all f32, is laid out first.
struct LayoutArgs {
  XentVocab v;            // weights: padded row r is row r % 256 of tile tile0 + r / 256
  const void* hidden;     // [tokens], rows ld_hidden elements apart
  const int32_t* idx;     // source row of each row, -1: zeros; null: row r itself
  uint64_t ld_weight, ld_hidden, hidden_plane, weight_plane;  // bytes between planes
  uint64_t hidden_rows, weight_rows;
  uint8_t *hidden_dst, *weight_dst;
  uint32_t tokens, cols, kpad, tile0, units_log2;
  uint32_t hidden_blocks, weight_blocks;  // workgroups of each
};

__device__ __forceinline__ void split(float x, uint32_t* p) {
  const bool finite = (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u;
  p[0] = f32_to_bf16(x);
  // the largest values round to infinity: cut those off instead
  if (finite && (p[0] & 0x7F80u) == 0x7F80u) p[0] = __float_as_uint(x) >> 16;
  const float rest = finite ? x - bf16_to_f32(p[0]) : 0.0f;
  p[1] = f32_to_bf16(rest);
  p[2] = f32_to_bf16(rest - bf16_to_f32(p[1]));
  p[3] = finite ? p[0] : 0u;
}

// The power of two that brings the largest of values with these bits (of |x|, finite)
// to at most 2^14, kept where it and its inverse are normal.
__device__ __forceinline__ float scale_to(uint32_t most) {
  uint32_t e = (most >> 23) + ((most & 0x7FFFFFu) ? 1u : 0u);
  e = e < 32u ? 32u : e > 254u ? 254u : e;
  return most == 0 ? 1.0f : __uint_as_float((254u + 14u - e) << 23);
}

__device__ __forceinline__ uint32_t block_max(uint32_t m, uint32_t* lds) {
#pragma unroll
  for (int x = 32; x > 0; x >>= 1) {
    const uint32_t o = __shfl_xor(m, x);
    m = o > m ? o : m;
  }
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
  __syncthreads();
  for (uint32_t w = 0; w < blockDim.x / 64; ++w) m = lds[w] > m ? lds[w] : m;
  return m;
}

__device__ __forceinline__ bool is_counted(int64_t target, int64_t ignore, int64_t vocab) {
  return target != ignore && target >= 0 && target < vocab;
}

// ---- tokens of a backward call ---------------------------------------------------
// Counted tokens in order, what their gradient needs, and for each token its place.
// One workgroup.  Gradients of logits held in f16 are scaled so that the largest dloss is
// 2^14: p dloss goes far below f16's smallest normal otherwise.  The scale is a
// power of two and is taken out of the f32 sums of both gradients.
struct TokensArgs {
  const int64_t* targets;
  const float* lse;
  const float* dloss;
  uint64_t dloss_stride;
  int64_t ignore, vocab;
  XentToken* token;  // [tpad], and again from lo on if that is not 0
  int32_t* idx;      // [tpad]: source row, -1 where there is none; likewise
  int32_t* place;    // [tokens]: place among the counted ones, -1: ignored
  XentScalars* scalars;
  uint32_t tokens, tpad, lo;
  int scaled;
};

constexpr int kTokensThreads = 1024;

__global__ void __launch_bounds__(kTokensThreads) tokens_k(TokensArgs a) {
  __shared__ uint32_t sums[kTokensThreads / 64];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  float scale = 1.0f;
  if (a.scaled) {
    uint32_t most = 0;  // bits of |dloss| order as the values do
    for (uint32_t t = tid; t < a.tokens; t += kTokensThreads) {
      const int64_t target = a.targets[t];
      const uint32_t u = __float_as_uint(a.dloss[t * a.dloss_stride]) & 0x7FFFFFFFu;
      if (is_counted(target, a.ignore, a.vocab) && u < 0x7F800000u && u > most) most = u;
    }
    scale = scale_to(block_max(most, sums));
    __syncthreads();
  }
  uint32_t before = 0;
  for (uint32_t t0 = 0; t0 < a.tokens; t0 += kTokensThreads) {
    const uint32_t t = t0 + tid;
    int64_t target = -1;
    if (t < a.tokens) target = a.targets[t];
    const bool counted = t < a.tokens && is_counted(target, a.ignore, a.vocab);
    const uint64_t mask = __ballot(counted);
    if (lane == 0) sums[wave] = (uint32_t)__popcll(mask);
    __syncthreads();
    uint32_t at = before, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < kTokensThreads / 64; ++w) {
      if (w < wave) at += sums[w];
      all += sums[w];
    }
    at += (uint32_t)__popcll(mask & ((1ull << lane) - 1));
    if (counted) {
      const XentToken tk = {a.lse[t], a.dloss[t * a.dloss_stride] * scale, (int32_t)target, 0};
      a.token[at] = tk;
      a.idx[at] = (int32_t)t;
      if (a.lo) {
        a.token[a.lo + at] = tk;
        a.idx[a.lo + at] = (int32_t)t;
      }
    }
    if (t < a.tokens) a.place[t] = counted ? (int32_t)at : -1;
    before += all;
    __syncthreads();
  }
  for (uint32_t t = before + tid; t < a.tpad; t += kTokensThreads) {
    if (a.lo && t - a.lo < before) continue;
    a.token[t] = {0.0f, 0.0f, -1, 0};
    a.idx[t] = -1;
  }
  if (tid == 0) {
    a.scalars->count = before;
    a.scalars->unscale_dz = 1.0f / scale;
  }
}

// Counted tokens in the order of their targets' 256-row tiles, tokens of a tile in
// order: a workgroup a tile finds its own and counts those of the tiles before.
struct HitsArgs {
  XentVocab v;
  const XentToken* token;
  const XentScalars* scalars;
  uint32_t *hits, *first;
  uint32_t tiles;  // 0: not wanted
};
__device__ __forceinline__ void sort_hits(const HitsArgs& a, uint32_t tile, uint32_t* before, uint32_t* mine) {
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int sh = 0;
  while (tile >= a.v.first_tile[sh + 1]) ++sh;
  const uint32_t row0 = (tile - a.v.first_tile[sh]) * kTileV, first = a.v.first_row[sh] + row0;
  const uint32_t rows = a.v.rows[sh] - row0 < (uint32_t)kTileV ? a.v.rows[sh] - row0 : (uint32_t)kTileV;
  const uint32_t count = a.scalars->count;
  uint32_t less = 0;
  for (uint32_t t = tid; t < count; t += 256) less += (uint32_t)a.token[t].target < first;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) less += __shfl_xor(less, m);
  if (lane == 0) before[wave] = less;
  __syncthreads();
  uint32_t at = before[0] + before[1] + before[2] + before[3];
  if (tid == 0) {
    a.first[tile] = at;
    if (tile + 1 == a.tiles) a.first[tile + 1] = count;
  }
  for (uint32_t t0 = 0; t0 < count; t0 += 256) {
    const uint32_t t = t0 + tid;
    const bool in = t < count && (uint32_t)a.token[t].target - first < rows;
    const uint64_t mask = __ballot(in);
    if (lane == 0) mine[wave] = (uint32_t)__popcll(mask);
    __syncthreads();
    uint32_t to = at + (uint32_t)__popcll(mask & ((1ull << lane) - 1));
    for (uint32_t w = 0; w < 4; ++w) {
      if (w < wave) to += mine[w];
      at += mine[w];
    }
    if (in) a.hits[to] = t;
    __syncthreads();
  }
}

template <int T> __device__ __forceinline__ void lay_row(const LayoutArgs& a, const uint8_t* src, uint8_t* dst, uint64_t plane, uint32_t u0) {
  const uint32_t lanes = 1u << a.units_log2, units = a.kpad / 8;
  for (uint32_t u = u0; u < units; u += lanes) {
    uint8_t* d = dst + 16 * (uint64_t)u;
    if constexpr (T == kF32) {
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
      if (src) {
        decode16<kF32>(load_cols<kF32>(src, 8 * u, a.cols), x);
        decode16<kF32>(load_cols<kF32>(src, 8 * u + 4, a.cols), x + 4);
      }
      uint32_t p[kPlanes][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t q[kPlanes];
        split(x[j], q);
#pragma unroll
        for (int k = 0; k < kPlanes; ++k) p[k][j] = q[k];
      }
#pragma unroll
      for (int k = 0; k < kPlanes; ++k)
        *reinterpret_cast<u32x4*>(d + k * plane) =
            u32x4{p[k][0] | p[k][1] << 16, p[k][2] | p[k][3] << 16, p[k][4] | p[k][5] << 16, p[k][6] | p[k][7] << 16};
    } else {
      *reinterpret_cast<u32x4*>(d) = src ? load_cols<T>(src, 8 * u, a.cols) : u32x4{0u, 0u, 0u, 0u};
    }
  }
}

// What the products need laid out, in one launch: hidden states, weights of a piece, and
// the tokens by their targets.  Bound by memory: 32003 x 1023 f16, whose rows start at any
// even address, 30 us, 4.4 TB/s.
template <int T> __global__ void __launch_bounds__(256) layout_k(LayoutArgs a, HitsArgs h) {
  __shared__ uint32_t lds[8];
  uint32_t id = blockIdx.x;
  const bool hidden = id < a.hidden_blocks;
  if (!hidden) id -= a.hidden_blocks;
  if (!hidden && id >= a.weight_blocks) return sort_hits(h, id - a.weight_blocks, lds, lds + 4);
  const uint32_t per = 256u >> a.units_log2, sub = threadIdx.x >> a.units_log2, u0 = threadIdx.x & ((1u << a.units_log2) - 1);
  if (hidden) {
    for (uint64_t row = (uint64_t)id * per + sub; row < a.hidden_rows; row += (uint64_t)a.hidden_blocks * per) {
      const int64_t r = a.idx ? (int64_t)a.idx[row] : row < a.tokens ? (int64_t)row : -1;
      lay_row<T>(a, r >= 0 ? at<T>(a.hidden, (uint64_t)r * a.ld_hidden) : nullptr, a.hidden_dst + row * a.kpad * 2, a.hidden_plane, u0);
    }
  } else {
    for (uint64_t row = (uint64_t)id * per + sub; row < a.weight_rows; row += (uint64_t)a.weight_blocks * per) {
      const uint32_t tile = a.tile0 + (uint32_t)(row / kTileV);
      int sh = 0;
      while (tile >= a.v.first_tile[sh + 1]) ++sh;
      const uint32_t r = (tile - a.v.first_tile[sh]) * kTileV + (uint32_t)(row % kTileV);
      lay_row<T>(a, r < a.v.rows[sh] ? at<T>(a.v.w[sh], (uint64_t)r * a.ld_weight) : nullptr, a.weight_dst + row * a.kpad * 2, a.weight_plane, u0);
    }
  }
}

// ---- tiles -------------------------------------------------------------------------
// Workgroup id to tile (m, n) of mt x nt, and to one of `splits` parts of k.  Workgroups
// go to the 8 XCDs in turn; each XCD gets one contiguous run of the order, which walks 8
// m tiles by all n tiles of a split, so that the tiles an XCD works on together share
// operands in its L2.  (Splits dealt out over the XCDs instead: 231 us against 134 for
// the hidden states' gradient of 700 x 50257 x 1600 f16.)
__device__ __forceinline__ bool tile_of(uint32_t id, uint32_t mt, uint32_t nt, uint32_t splits, uint32_t& m, uint32_t& n,
                                        uint32_t& split) {
  const uint32_t tiles = mt * nt, total = tiles * splits, per = total / 8, extra = total % 8, x = id & 7, j = id >> 3;
  if (j >= per + (x < extra ? 1u : 0u)) return false;
  uint32_t t = x * per + (x < extra ? x : extra) + j;
  split = t / tiles;
  t -= split * tiles;
  constexpr uint32_t G = 8;
  const uint32_t g = t / (G * nt), rem = t - g * (G * nt), gm = mt - g * G < G ? mt - g * G : G;
  m = g * G + rem % gm;
  n = rem / gm;
  return true;
}
uint32_t tile_grid(uint64_t tiles) { return (uint32_t)((tiles + 7) / 8 * 8); }

// A pair of a forward: the largest logit z of some rows, and the sum of exp(z' - z) over
// them.  The terms are exp2(fma(z', log2 e, -base)), base = z log2 e as rounded; what that
// rounding takes is given back to the sum, so that the pair is as exact as its parts.
// Rows without a finite logit add nothing (or, with +inf, NaN).
__device__ __forceinline__ float base_of(float mx) { return mx == -__builtin_inff() ? 0.0f : mx * kLog2e; }
__device__ __forceinline__ float2 part_of(float mx, float s, float base) {
  const float lost = mx == -__builtin_inff() ? 0.0f : __builtin_fmaf(mx, kLog2e, -base);
  return make_float2(mx, s * __builtin_amdgcn_exp2f(-lost));
}

// dz of a logit.
template <bool F32> __device__ __forceinline__ float dz_of(float z, const XentToken& tk, bool hit) {
  const float x = z - tk.lse;
  return ((F32 ? __builtin_expf(x) : __builtin_amdgcn_exp2f(x * kLog2e)) - (hit ? 1.0f : 0.0f)) * tk.dl;
}

// What 16 bits lose of a dz.  Up to 64 tokens it is a second 16-bit part, in a row of its own:
// a tile of 128 tokens has the place, and past 32 tokens the weights' gradient takes 64 more k
// (64 x 32000 x 4096 bf16: 176 to 195 us).  Of more tokens only the target's is kept, nearly all of most rows'
// gradient, in f32, and added to the sums of both gradients.  The others' one rounding is as
// that of the gradient itself, but takes part in sums over tokens and rows: 4096 x 128256 x
// 4096 bf16 gradients are 0.00166 off, which is their own rounding; rows that are no token's
// target 0.0023.  (Two parts there would be five products for three.  An f32 call's dz keeps
// its 24 bits.)
template <int T> __device__ __forceinline__ float residue_of(float d) {
  const float r = d - to_f32<T>(from_f32<T>(d));
  return (__float_as_uint(r) & 0x7F800000u) != 0x7F800000u ? r : 0.0f;
}

// N values of dz stored in T (f32: as planes).
template <int T, int N> __device__ __forceinline__ void store_dz(uint8_t* to, uint64_t plane, const float* d) {
  constexpr int P = T == kF32 ? kPlanes : 1;
  uint32_t w[P][N / 2] = {};
#pragma unroll
  for (int e = 0; e < N; ++e) {
    uint32_t part[kPlanes];
    if constexpr (T == kF32) split(d[e], part);
    else part[0] = from_f32<T>(d[e]);
#pragma unroll
    for (int b = 0; b < P; ++b) w[b][e >> 1] |= part[b] << (16 * (e & 1));
  }
#pragma unroll
  for (int b = 0; b < P; ++b) {
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(to + b * plane) = u32x4{w[b][0], w[b][1], w[b][2], w[b][3]};
    else *reinterpret_cast<u32x2*>(to + b * plane) = u32x2{w[b][0], w[b][1]};
  }
}

// What becomes of a tile's logits.  FULL: all its rows and tokens exist.  The rare
// lanes whose target lies in the wave's rows are looked for once for 32 tokens, not at
// each logit: what is left is an fma, an exponential (a quarter of the rate) and an
// add or two.
template <int T, int S, bool BWD, int SEG, bool FULL, class Prod>
__device__ __forceinline__ void logits_out(const XentArgs& a, Prod& p, lds8* lds, int wm, int wn, int lane,
                                           uint32_t mt, uint32_t part, uint32_t t0, uint32_t tokens, uint32_t first,
                                           uint32_t left) {
  const uint32_t m0 = wm * Prod::FM * 32;
  const uint32_t lo = BWD && S == 128 && SEG == 1 ? a.lo : 0u;  // up to 64 tokens: one tile of 128
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j) {
    const uint32_t t = t0 + (wn * Prod::FN + j) * 32 + (lane & 31);
    const bool low = !FULL && lo && t >= lo;
    const bool live = FULL || (low ? t - lo : t) < tokens;
    // the target's row of the wave's, if it is there
    uint32_t hit = ~0u;
    XentToken tk;
    if constexpr (BWD) {
      tk = a.token[t];
      if (live && (uint32_t)tk.target - first < left) hit = (uint32_t)tk.target - first - m0;
    } else {
      const int64_t target = live ? a.targets[t] : -1;
      if (target >= first && target < (int64_t)first + left) hit = (uint32_t)(target - first) - m0;
    }
    const bool hits = __any(hit < Prod::FM * 32u);
    if constexpr (!BWD) {
      if (hits) {
        float z = 0.0f;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool is = (uint32_t)(32 * i + acc_row(lane, e)) == hit;
            z = is ? p.acc[i][j][e] : z;
            mine |= is;
          }
        if (mine) a.zt[t] = z;
      }
      float mx = -__builtin_inff();
#pragma unroll
      for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          if (!FULL && m0 + 32 * i + acc_row(lane, e) >= left) p.acc[i][j][e] = -__builtin_inff();
          mx = __builtin_fmaxf(mx, p.acc[i][j][e]);
        }
      mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
      const float base = base_of(mx);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(p.acc[i][j][e], kLog2e, -base));
      s += __shfl_xor(s, 32);
      if (lane < 32 && live) a.part[(a.part0 + (uint64_t)part * Prod::WM + wm) * a.tokens + t] = part_of(mx, s, base);
    } else {
#pragma unroll
      for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float d = dz_of<(SEG > 1)>(p.acc[i][j][e], tk, false);
          p.acc[i][j][e] = FULL || (live && m0 + 32 * i + acc_row(lane, e) < left) ? d : 0.0f;
        }
      if (hits) {
        float d = 0.0f;
        bool mine = false;
#pragma unroll
        for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const bool is = (uint32_t)(32 * i + acc_row(lane, e)) == hit;
            p.acc[i][j][e] -= is ? tk.dl : 0.0f;
            d = is ? p.acc[i][j][e] : d;
            mine |= is;
          }
        if (SEG == 1 && mine && !lo) a.residue[t] = residue_of<T>(d);
      }
      if (SEG == 1 && low) {
#pragma unroll
        for (int i = 0; i < Prod::FM; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) p.acc[i][j][e] = residue_of<T>(p.acc[i][j][e]);
      }
      if (j == 0) __syncthreads();
      p.template rows_out<8>(lds, j, [](auto) {}, [&](int n, int m, const float (&d)[8]) {
        store_dz<SEG == 1 ? T : (int)kF32, 8>(a.dz + (uint64_t)(t0 + n) * a.lddz + ((uint64_t)mt * S + m) * 2, a.dz_plane, d);
      });
    }
  }
}

// Logits of one tile of S vocabulary rows by S tokens.  Forward: reduced to a
// (max, sum) pair for each wave's rows, and the target's logit.
// Backward: dz, vocabulary contiguous.  4096 x 128256 x 4096 bf16 forward: 3.2 ms, 1.34
// PFLOP/s (a library product of that size 2.96 ms); backward, a quarter of it for the 3690
// tokens that count: 0.83 ms, 1.17.  What a tile does besides its products is not hidden (one
// workgroup of 256 x 256 fills a CU's LDS): the matrix units multiply in 0.81 of the forward's
// time at 64 stages a tile, in 0.67 at 25.
template <int T, int S, int NS, bool BWD, int SEG>
__global__ void __launch_bounds__(tile_threads(S)) logits_k(XentArgs a) {
  typedef Tile<T, false, false, S, NS> Prod;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Prod::kLds];
  uint32_t mt, nt, split;
  constexpr uint32_t per = kTileV / S;  // of a vocabulary tile
  if (!tile_of(blockIdx.x, a.sub * per, a.tpad / S, 1, mt, nt, split)) return;
  const uint32_t part = mt;
  mt += a.sub0 * per;
  const uint32_t tokens = BWD ? a.scalars->count : a.tokens;
  const uint32_t t0 = nt * S, tile = a.tile0 + mt / per;
  if (t0 >= tokens) return;
  int sh = 0;
  while (tile >= a.v.first_tile[sh + 1]) ++sh;
  const uint32_t row0 = (tile - a.v.first_tile[sh]) * kTileV + mt % per * S, rows = a.v.rows[sh];  // of the shard
  const uint32_t left = row0 < rows ? (rows - row0 < (uint32_t)S ? rows - row0 : (uint32_t)S) : 0u;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // rows past the shard: any that exists
  const uint32_t at0 = row0 < rows ? row0 : rows - 1, have = a.laid ? (uint32_t)S : left ? left : 1u;
  const uint8_t* wa = a.laid ? a.laid + (uint64_t)mt * S * a.ldw : (const uint8_t*)a.v.w[sh] + (uint64_t)at0 * a.ldw;
  const uint8_t* hb = a.h + (uint64_t)t0 * a.ldh;
  const uint32_t t_have = tokens - t0;  // of a forward: hidden states may be read in place
  uint32_t k = 0, seg = 0;
  const uint32_t kend = a.kpad * 2;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
      const uint32_t c = row_src_chunk(tid) * 16;
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) {
        const uint32_t r = row_src_row<S>(tid, i);
        oa[i] = (r < have ? r : have - 1) * a.ldw + c;
        ob[i] = (BWD || r < t_have ? r : t_have - 1) * a.ldh + c;
      }
    }
    pa = wa + k;
    pb = hb + k;
    if constexpr (SEG > 1) {
      pa += seg_a(seg) * a.laid_plane;
      pb += seg_b(seg) * a.h_plane;
    }
    k += kTileK * 2;
    if (SEG > 1 && k == kend) k = 0, ++seg;
  };
  Prod p;
  p.run((int)(a.kpad / kTileK) * SEG, (lds8*)lds, src);

  const int wm = wave / Prod::WN, wn = wave % Prod::WN;
  const uint32_t first = a.v.first_row[sh] + row0;  // of the whole vocabulary
  if (left == (uint32_t)S && t0 + S <= tokens) logits_out<T, S, BWD, SEG, true>(a, p, (lds8*)lds, wm, wn, lane, mt, part, t0, tokens, first, left);
  else logits_out<T, S, BWD, SEG, false>(a, p, (lds8*)lds, wm, wn, lane, mt, part, t0, tokens, first, left);
}

// ---- logits of few tokens ----------------------------------------------------------
// The same without LDS tiles, for calls that are bound by reading the weights: a
// workgroup takes 16 R vocabulary rows by 16 NT tokens, its 4 waves every fourth 128
// bytes of the rows, and operands go from memory to the matrix instructions as they
// are loaded (any address, no layout pass; f32 multiplies as f32).  A lane loads 32
// bytes of its row, two loads that use up a line together; which k of the block a
// lane's elements are is the same for both operands, so their order does not matter.
// 1 token x 32000 x 4096 bf16: 43.5 us, 6.0 TB/s.
typedef float f32x4v __attribute__((ext_vector_type(4)));
template <int T> __device__ __forceinline__ f32x4v mfma16(u32x4 a, u32x4 b, f32x4v c) {
  if constexpr (T == kF32) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  } else if constexpr (T == kF16) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  } else {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  }
}

template <int T, int NT, int R, bool BWD> __global__ void __launch_bounds__(256) few_k(XentArgs a) {
  constexpr int V = Vec<T>::VW, B = 8 * V;  // elements of a load, and of a 128-byte block
  constexpr int U = R * NT >= 8 ? 2 : 4;    // blocks in flight
  __shared__ f32x4v red[4][R * NT][64];
  const uint32_t tokens = BWD ? a.scalars->count : a.tokens;
  const uint32_t t0 = blockIdx.y * (16 * NT);
  // dz of the last 64 tokens' places past the counted ones is zero, of those before the low parts too
  if (t0 >= (!BWD ? tokens : a.lo ? a.lo : (tokens + kTileK - 1) / kTileK * kTileK)) return;
  constexpr uint32_t per = kTileV / (16 * R);
  const uint32_t mt = blockIdx.x / per, tile = a.tile0 + mt, sub = blockIdx.x % per * (16 * R);
  int sh = 0;
  while (tile >= a.v.first_tile[sh + 1]) ++sh;
  const uint32_t row0 = (tile - a.v.first_tile[sh]) * kTileV + sub, rows = a.v.rows[sh];
  const uint32_t left = row0 < rows ? (rows - row0 < 16u * R ? rows - row0 : 16u * R) : 0u;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  f32x4v acc[R][NT];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f32x4v{0.0f, 0.0f, 0.0f, 0.0f};
  if (left && t0 < tokens) {
    const uint32_t lane0 = (lane >> 4) * 2 * V;  // a lane's first element of a block
    const uint8_t *pw[R], *ph[NT];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t m = 16 * r + (lane & 15);
      pw[r] = at<T>(a.v.w[sh], (uint64_t)(row0 + (m < left ? m : left - 1)) * a.ld_w + lane0);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t t = t0 + 16 * n + (lane & 15);
      uint32_t from = t < tokens ? t : tokens - 1;
      if constexpr (BWD) from = (uint32_t)a.idx[from];
      ph[n] = at<T>(a.hidden, (uint64_t)from * a.ld_h + lane0);
    }
    const uint32_t blocks = a.cols / B;
    uint32_t b = wave;
    for (; b + 4 * (U - 1) < blocks; b += 4 * U) {
      u32x4 vw[U][R][2], vh[U][NT][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int x = 0; x < 2; ++x) vw[u][r][x] = load_raw<T>(pw[r] + (uint64_t)(b + 4 * u) * 128 + 16 * x, V);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int x = 0; x < 2; ++x) vh[u][n][x] = load_raw<T>(ph[n] + (uint64_t)(b + 4 * u) * 128 + 16 * x, V);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int n = 0; n < NT; ++n) acc[r][n] = mfma16<T>(vw[u][r][x], vh[u][n][x], acc[r][n]);
    }
    for (; b * B < a.cols; b += 4) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t c = b * B + lane0 + x * V;
        u32x4 vw[R], vh[NT];
#pragma unroll
        for (int r = 0; r < R; ++r) vw[r] = load_cols<T>(pw[r] - (uint64_t)lane0 * Ty<T>::size, c, a.cols);
#pragma unroll
        for (int n = 0; n < NT; ++n) vh[n] = load_cols<T>(ph[n] - (uint64_t)lane0 * Ty<T>::size, c, a.cols);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int n = 0; n < NT; ++n) acc[r][n] = mfma16<T>(vw[r], vh[n], acc[r][n]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) red[wave][r * NT + n][lane] = acc[r][n];
  __syncthreads();
  if (wave >= NT) return;
  // wave n joins the four parts of the n-th 16 tokens; a lane has token lane % 16
  const uint32_t t = t0 + 16 * wave + (lane & 15), first = a.v.first_row[sh] + row0;
  f32x4v z[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    z[r] = red[0][r * NT + wave][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) z[r] += red[w][r * NT + wave][lane];
  }
  if constexpr (!BWD) {
    const int64_t target = t < tokens ? a.targets[t] : -1;
    const uint32_t hit = target >= first && target < (int64_t)first + left ? (uint32_t)(target - first) : ~0u;
    float mx = -__builtin_inff();
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = 16 * r + 4 * (lane >> 4) + e;
        if (m == hit) a.zt[t] = z[r][e];
        if (m >= left) z[r][e] = -__builtin_inff();
        mx = __builtin_fmaxf(mx, z[r][e]);
      }
    mx = __builtin_fmaxf(mx, __shfl_xor(mx, 16));
    mx = __builtin_fmaxf(mx, __shfl_xor(mx, 32));
    const float base = base_of(mx);
    float s = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e) s += __builtin_amdgcn_exp2f(__builtin_fmaf(z[r][e], kLog2e, -base));
    s += __shfl_xor(s, 16);
    s += __shfl_xor(s, 32);
    if (lane < 16 && t < tokens) a.part[(uint64_t)t * a.parts + (uint64_t)a.tile0 * per + blockIdx.x] = part_of(mx, s, base);
  } else {
    const XentToken tk = a.token[t];
    const bool live = t < tokens;
    const uint32_t hit = live && (uint32_t)tk.target - first < left ? (uint32_t)tk.target - first : ~0u;
    uint8_t* row = a.dz + (uint64_t)t * a.lddz + ((uint64_t)mt * kTileV + sub) * 2;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float d[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = 16 * r + 4 * (lane >> 4) + e;
        d[e] = live && m < left ? dz_of<T == kF32>(z[r][e], tk, m == hit) : 0.0f;
      }
      store_dz<T, 4>(row + (16 * r + 4 * (lane >> 4)) * 2, a.dz_plane, d);
      if constexpr (T != kF32) {  // up to 64 tokens: lo is not 0
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = residue_of<T>(d[e]);
        store_dz<T, 4>(row + (uint64_t)a.lo * a.lddz + (16 * r + 4 * (lane >> 4)) * 2, 0, d);
      }
    }
  }
}

// Gradient of the hidden states from one piece of the vocabulary: a tile of S columns
// by S tokens over the split's share of the piece's rows, into (or, after the first
// piece, added to) the split's f32 sums.
template <int T, int S, int NS, int SEG> __device__ __forceinline__ void dhidden_tile(const XentArgs& a, uint32_t id, lds8* lds) {
  typedef Tile<T, true, false, S, NS> Prod;
  uint32_t mt, nt, split;
  if (!tile_of(id, (a.kpad + S - 1) / S, a.tpad / S, a.splits, mt, nt, split)) return;
  const uint32_t t0 = nt * S, c0 = mt * S;
  if (t0 >= a.scalars->count) return;
  const int tid = threadIdx.x;
  const uint32_t blocks = a.ntiles * (kTileV / kTileK);  // of 64 rows
  const uint32_t k0 = (uint32_t)((uint64_t)blocks * split / a.splits), k1 = (uint32_t)((uint64_t)blocks * (split + 1) / a.splits);
  uint32_t k = k0, seg = 0;
  int sh = 0;
  // a lane's column chunk; past the last column any that exists
  uint32_t col = c0 + col_src_chunk<S>(tid) * 8;
  col = (col < a.kpad ? col : a.kpad - 8) * 2;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
      const uint32_t c = row_src_chunk(tid) * 16;
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) ob[i] = row_src_row<S>(tid, i) * a.lddz + c;
    }
    uint32_t have = kTileK;
    if (SEG > 1 || a.laid) {
      pa = a.laid + (uint64_t)k * kTileK * a.ldw;
    } else {
      const uint32_t tile = a.tile0 + k / (kTileV / kTileK);
      while (tile >= a.v.first_tile[sh + 1]) ++sh;
      // rows past the shard meet zeros of dz: any that exists
      const uint32_t row = (tile - a.v.first_tile[sh]) * kTileV + k % (kTileV / kTileK) * kTileK, rows = a.v.rows[sh];
      const uint32_t at = row < rows ? row : rows - 1;
      have = rows - at < (uint32_t)kTileK ? rows - at : (uint32_t)kTileK;
      pa = (const uint8_t*)a.v.w[sh] + (uint64_t)at * a.ldw;
    }
    pb = a.dz + (uint64_t)t0 * a.lddz + (uint64_t)k * kTileK * 2;
    if constexpr (SEG > 1) {
      pa += seg_a(seg) * a.laid_plane;
      pb += seg_b(seg) * a.dz_plane;
    }
#pragma unroll
    for (int i = 0; i < Prod::L; ++i) {
      const uint32_t r = col_src_k<S>(tid, i);
      oa[i] = (r < have ? r : have - 1) * a.ldw + col;
    }
    if (++k == k1) k = k0, ++seg;
  };
  Prod p;
  p.run((int)(k1 - k0) * SEG, lds, src);

  float* sum = a.sum + (uint64_t)split * a.tpad * a.kpad;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template rows_out<4>(lds, j, [](auto) {}, [&](int n, int m, const float (&x)[4]) {
      if (c0 + m >= a.kpad) return;
      f32x4* to = reinterpret_cast<f32x4*>(sum + (uint64_t)(t0 + n) * a.kpad + c0 + m);
      f32x4 y = {x[0], x[1], x[2], x[3]};
      if (a.add) {
        const f32x4 o = *to;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = o[e] + y[e];
      }
      *to = y;
    });
}

// Weight gradients of one piece: a tile of S columns by S vocabulary rows over the
// counted tokens, rounded once.
template <int T, int OUT, int S, int NS, int SEG> __device__ __forceinline__ void dweight_tile(const XentArgs& a, uint32_t id, lds8* lds) {
  typedef Tile<T, true, true, S, NS> Prod;
  uint32_t mt, nt, split;
  constexpr uint32_t per = kTileV / S;  // of a vocabulary tile
  if (!tile_of(id, (a.kpad + S - 1) / S, a.sub * per, 1, mt, nt, split)) return;
  nt += a.sub0 * per;
  const uint32_t c0 = mt * S, tile = a.tile0 + nt / per;
  int sh = 0;
  while (tile >= a.v.first_tile[sh + 1]) ++sh;
  const uint32_t row0 = (tile - a.v.first_tile[sh]) * kTileV + nt % per * S, rows = a.v.rows[sh];
  if (!a.dw[sh] || row0 >= rows) return;
  const uint32_t left = rows - row0 < (uint32_t)S ? rows - row0 : (uint32_t)S;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  uint32_t col = c0 + col_src_chunk<S>(tid) * 8;
  col = (col < a.kpad ? col : a.kpad - 8) * 2;
  // of 64 tokens; those past the last have dz 0
  const uint32_t count = a.scalars->count, blocks = count ? (a.lo + count + kTileK - 1) / kTileK : 0u;
  uint32_t k = 0, seg = 0;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) {
        oa[i] = col_src_k<S>(tid, i) * a.ldh + col;
        ob[i] = col_src_k<S>(tid, i) * a.lddz + col_src_chunk<S>(tid) * 16;
      }
    }
    pa = a.h + (uint64_t)k * kTileK * a.ldh;
    pb = a.dz + (uint64_t)k * kTileK * a.lddz + (uint64_t)nt * S * 2;
    if constexpr (SEG > 1) {
      pa += seg_a(seg) * a.h_plane;
      pb += seg_b(seg) * a.dz_plane;
    }
    if (++k == blocks) k = 0, ++seg;
  };
  Prod p;
  p.run((int)blocks * SEG, lds, src);

  const float unscale = a.scalars->unscale_dz;
  constexpr int W = OUT == kF32 ? 4 : 8;
  const uint32_t first = a.v.first_row[sh] + row0;
  // the list of tokens whose target lies in this tile
  uint32_t h0 = 0, h1 = 0;
  if (SEG == 1 && !a.lo) h0 = a.hits_first[tile], h1 = a.hits_first[tile + 1];
  // a lane's token of the list's k-th 64, and its target's row in the tile
  auto entry = [&](uint32_t k, uint32_t& t) {
    t = k < h1 ? a.hits[k] : 0u;
    return k < h1 ? (uint32_t)a.token[t].target - first : ~0u;
  };
  uint32_t t0 = 0, r0 = ~0u;
  if (h0 < h1) r0 = entry(h0 + lane, t0);
  const int wm0 = wave / Prod::WN * (Prod::FM * 32);  // the wave's first column of the tile
  const uint32_t hc = c0 + wm0 + 4 * lane;
  __syncthreads();
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j) {
    const uint32_t n0 = (wave % Prod::WN * Prod::FN + j) * 32;
    auto residues = [&](auto add) {
      for (uint32_t k = h0; k < h1; k += 64) {
        uint32_t t = t0, r = r0;
        if (k != h0) r = entry(k + lane, t);
        uint64_t mask = __ballot(r - n0 < 32u);
        while (mask) {
          const int l = __builtin_ctzll(mask);
          mask &= mask - 1;
          const uint32_t token = __builtin_amdgcn_readlane(t, l), row = __builtin_amdgcn_readlane(r, l) - n0;
          if (lane < Prod::FM * 8 && hc < a.kpad) {
            const u32x2 raw = *reinterpret_cast<const u32x2*>(a.h + (uint64_t)token * a.ldh + (uint64_t)hc * 2);
            const float e = a.residue[token];
            const float x[4] = {e * to_f32<T>(raw.x & 0xFFFFu), e * to_f32<T>(raw.x >> 16), e * to_f32<T>(raw.y & 0xFFFFu),
                                e * to_f32<T>(raw.y >> 16)};
            add((int)row, 4 * lane, x);
          }
        }
      }
    };
    p.template rows_out<W>(
        lds, j,
        [&](auto add) {
          if constexpr (SEG == 1) residues(add);
        },
        [&](int n, int m, float (&x)[W]) {
          const uint32_t c = c0 + m;
          if ((uint32_t)n >= left || c >= a.cols) return;
#pragma unroll
          for (int i = 0; i < W; ++i) x[i] *= unscale;
          // past the caches: the weights' next reader finds them there (1 token x 32000 x 4096: 212 to 177 us)
          void* to = at<OUT>(a.dw[sh], (uint64_t)(row0 + n) * a.ld_dw + c);
          if (a.cols - c >= W) __builtin_nontemporal_store(encode16<OUT>(x), reinterpret_cast<u32x4_any*>(to));
          else store_raw<OUT>(to, (int)(a.cols - c), encode16<OUT>(x));
        });
  }
}

// Both gradients of a piece: the first `dh_grid` workgroups (none: 0) take tiles of the
// hidden states', the others of the weights'.  3690 counted tokens of 4096 x 32256 x 4096
// bf16: 0.89 and 0.82 ms, 1.10 and 1.19 PFLOP/s (the matrix units multiply in 0.63 and 0.72 of
// the time); 901 of 1001 x 32003 x 1023 f16, both: 135 us.
template <int T, int OUT, int S, int NS, int SEG> __global__ void __launch_bounds__(tile_threads(S)) grads_k(XentArgs a, uint32_t dh_grid) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Tile<T, true, true, S, NS>::kLds];
  if (blockIdx.x < dh_grid) dhidden_tile<T, S, NS, SEG>(a, blockIdx.x, (lds8*)lds);
  else dweight_tile<T, OUT, S, NS, SEG>(a, blockIdx.x - dh_grid, (lds8*)lds);
}

// ---- joins -------------------------------------------------------------------------
// lse and loss of JT tokens a workgroup (the loss as the largest logit less the target's, 0
// where they are one, and the log of the sum: a sure token's small loss keeps its digits): 1024 / JT chains of pairs, then those in order
// (halves first, so that the last steps are few).
constexpr int kJoinThreads = 1024;

__device__ __forceinline__ float2 join2(float2 a, float2 b) {
  const float top = __builtin_fmaxf(a.x, b.x);
  if (top == -__builtin_inff()) return make_float2(top, a.y + b.y);
  return make_float2(top, a.y * __builtin_amdgcn_exp2f((a.x - top) * kLog2e) + b.y * __builtin_amdgcn_exp2f((b.x - top) * kLog2e));
}

template <int JT> __global__ void __launch_bounds__(kJoinThreads) join_k(XentJoinArgs a) {
  constexpr uint32_t chains = kJoinThreads / JT;
  __shared__ float2 lds[kJoinThreads];
  const uint32_t x = threadIdx.x % JT, chain = threadIdx.x / JT;
  const uint32_t t = blockIdx.x * JT + x;
  float2 s = make_float2(-__builtin_inff(), 0.0f);
  if (t < a.tokens) {
    const float2* part = a.part + t * a.token_stride;
#pragma unroll 4
    for (uint32_t p = chain; p < a.parts; p += chains) s = join2(s, part[p * a.part_stride]);
  }
  lds[threadIdx.x] = s;
#pragma unroll
  for (uint32_t n = chains / 2; n > 0; n /= 2) {
    __syncthreads();
    if (chain < n) lds[threadIdx.x] = join2(lds[threadIdx.x], lds[threadIdx.x + n * JT]);
  }
  if (chain || t >= a.tokens) return;
  s = lds[threadIdx.x];
  const float rest = __builtin_log2f(s.y) * kLn2;
  if (a.lse) a.lse[t] = s.x + rest;
  if (a.loss) {
    const int64_t target = a.targets[t];
    a.loss[t] = target == a.ignore ? 0.0f : target >= 0 && target < a.vocab ? (s.x - a.zt[t]) + rest : __builtin_nanf("");
  }
}

// Gradient rows of the hidden states: the splits' sums in order, rounded once; zeros
// for a token that has no loss.
template <int T> __global__ void __launch_bounds__(256) dhidden_join_k(XentArgs a) {
  const float unscale = a.scalars->unscale_dz;
  for (uint32_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int32_t from = a.place[t];
    const uint8_t* w = nullptr;  // the target's row
    float residue = 0.0f;
    if constexpr (T != kF32) {
      if (from >= 0 && !a.lo) {
        const uint32_t target = (uint32_t)a.token[from].target;
        int sh = 0;
        while (target - a.v.first_row[sh] >= a.v.rows[sh]) ++sh;
        w = at<T>(a.v.w[sh], (uint64_t)(target - a.v.first_row[sh]) * a.ld_w);
        residue = a.residue[from];
      }
    }
    for (uint32_t c = 4 * (blockIdx.y * 256 + threadIdx.x); c < a.cols; c += 1024 * gridDim.y) {
      float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (from >= 0) {
        const float* p = a.sum + (uint64_t)from * a.kpad + c;
        const uint32_t parts = a.lo ? 2 * a.splits : a.splits;  // the low rows' sums after the others
#pragma unroll 8
        for (uint32_t s = 0; s < parts; ++s) {
          const uint32_t row = s < a.splits ? s * a.tpad : (s - a.splits) * a.tpad + a.lo;
          const f32x4 y = *reinterpret_cast<const f32x4*>(p + (uint64_t)row * a.kpad);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] += y[e];
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (T != kF32 && w && c + e < a.cols) x[e] = __builtin_fmaf(residue, load_elem<T>(w, c + e), x[e]);
          x[e] *= unscale;
        }
      }
      store4<T>(at<T>(a.dhidden, (uint64_t)t * a.ld_dh + c), (int)(a.cols - c), x);
    }
  }
}

// Weight gradients of a call without tokens.
__global__ void __launch_bounds__(256) zero_rows_k(uint8_t* p, uint64_t rows, uint64_t pitch, uint32_t halves) {
  for (uint64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (uint32_t i = threadIdx.x; i < halves; i += 256) reinterpret_cast<uint16_t*>(p + r * pitch)[i] = 0;
}

// ---- plan --------------------------------------------------------------------------
constexpr uint64_t kPieceBytes = 256ull << 20;  // of dz, and of weights laid out
constexpr uint64_t kMaxTiles = 1ull << 22;       // workgroups of 512 threads in a launch
uint64_t up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

uint64_t tiles_of(uint64_t m, uint64_t n, uint64_t s) { return (m + s - 1) / s * ((n + s - 1) / s); }

// A product of `rows` 256-row tiles by q256 tiles of 256 (q128 of 128): how many of the
// rows go in 256 x 256 tiles, the rest in 128 x 128.  Large tiles are the faster ones,
// but the last of their rounds over the 256 CUs may be nearly empty: then the rows past
// the full rounds go in small ones.  Times in 10 ns, measured: a round of large tiles
// 1.43 us for each 64 k and 9 us; of small ones, two a CU, 0.85 and 6, one a CU 0.75 and
// 6.  (700 tokens x 50257 x 1600, 25 stages: 138 us in large tiles, 136 in small ones,
// 119 in both.)
uint32_t large_rows(uint32_t rows, uint64_t q256, uint64_t q128, uint64_t stages) {
  const uint64_t large = 143 * stages + 900;
  auto small = [&](uint64_t n) {
    return n == 0 ? 0 : n <= 256 ? 75 * stages + 600 : (n + 511) / 512 * (85 * stages + 600);
  };
  if (q128 == 1) return 0;
  uint64_t best = small(2 * rows * q128);
  uint32_t r = 0;
  if (const uint64_t c = (rows * q256 + 255) / 256 * large; c < best) best = c, r = rows;
  const uint64_t full = rows * q256 / 256, most = full * 256 / q256;
  if (most && most < rows && full * large + small(2 * (rows - most) * q128) + 200 < best) r = (uint32_t)most;
  return r;
}

}  // namespace

XentPlan xent_plan(uint32_t tokens, uint32_t cols, const size_t* rows, int nranks, int t, bool backward) {
  XentPlan p{};
  const uint64_t planes = t == kF32 ? kPlanes : 1;
  p.tpad = (uint32_t)up(tokens, tokens <= 128 ? 128 : 256);
  p.kpad = (uint32_t)up(cols, kTileK);
  uint64_t tiles = 0;
  for (int r = 0; r < nranks; ++r) tiles += up(rows[r], kTileV) / kTileV;
  p.tiles = (uint32_t)tiles;
  // tiles of a piece: dz of all tokens, and the weights, each within kPieceBytes
  uint64_t most = kPieceBytes / ((uint64_t)kTileV * p.kpad * 2 * planes);
  if (backward) {
    const uint64_t d = kPieceBytes / ((uint64_t)kTileV * p.tpad * 2 * planes);
    if (d < most) most = d;
  }
  // at least two rounds of small tiles over the CUs, however many bytes that is up to 1 GiB
  const uint64_t fill = 4 * kPieceBytes / ((uint64_t)kTileV * p.kpad * 2 * planes), want = (1024 + p.tpad / 64) / (p.tpad / 64);
  if (most < want) most = want < fill ? want : fill;
  const uint64_t grid = kMaxTiles / (p.tpad / 128 * 2);
  if (grid < most) most = grid;
  if (most < 1) most = 1;
  const uint64_t pieces = tiles ? (tiles + most - 1) / most : 1;
  p.piece = (uint32_t)((tiles + pieces - 1) / pieces);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t o = at;
    at += up(bytes, 1024);
    return o;
  };
  p.h_plane = (uint64_t)p.tpad * p.kpad * 2;
  p.laid_plane = (uint64_t)p.piece * kTileV * p.kpad * 2;
  if (backward) {
    p.dz_plane = (uint64_t)p.tpad * p.piece * kTileV * 2;
    p.dz = take(p.dz_plane * planes);
    // enough splits of a piece's rows that every CU has a tile of 256 (small calls: two of 128)
    const uint64_t big = tiles_of(p.kpad, p.tpad, 256);
    p.dh_tile = p.tpad > 128 && big >= 8 ? 256 : 128;
    uint64_t s = p.dh_tile == 256 ? 256 / big : 512 / tiles_of(p.kpad, p.tpad, 128);
    if (s > p.piece) s = p.piece;
    p.splits = s < 1 ? 1 : (uint32_t)s;
    p.sum = take((uint64_t)p.splits * p.tpad * p.kpad * 4);
    p.token = take((uint64_t)p.tpad * sizeof(XentToken));
    p.idx = take((uint64_t)p.tpad * 4);
    p.place = take((uint64_t)tokens * 4);
    p.residue = take((uint64_t)p.tpad * 4);
    p.hits = take((uint64_t)p.tpad * 4);
    p.hits_first = take((tiles + 1) * 4);
  } else {
    // pairs of a tile and token: at most few_k's, else those of 128 x 128 tiles
    p.part = take(tiles * (tokens <= 64 ? 16 : t == kF32 ? 8 : 4) * tokens * sizeof(float2));
    p.zt = take((uint64_t)tokens * 4);
  }
  p.scalars = take(sizeof(XentScalars));
  // last what a call that reads its operands in place does without
  if (backward) p.h = take(p.h_plane * planes);
  p.bytes_in_place = at;
  if (!backward) p.h = take(p.h_plane * planes);
  p.laid = take(p.laid_plane * planes);
  p.bytes = at;
  return p;
}

namespace {

// h.tiles workgroups past those of the rows sort tokens by their targets.
template <int T> void layout(LayoutArgs l, const HitsArgs& h, hipStream_t s) {
  uint32_t log2 = 0;
  while (log2 < 8 && (1u << log2) < l.kpad / 8) ++log2;
  l.units_log2 = log2;
  auto blocks = [&](uint64_t rows) {
    const uint64_t per = 256u >> log2, n = (rows + per - 1) / per;
    return (uint32_t)(n < 65536 ? n : 65536);
  };
  l.hidden_blocks = blocks(l.hidden_rows);
  l.weight_blocks = blocks(l.weight_rows);
  if (const uint32_t grid = l.hidden_blocks + l.weight_blocks + h.tiles)
    hipLaunchKernelGGL(layout_k<T>, dim3(grid), dim3(256), 0, s, l, h);
}

// 16-token groups of a few_k workgroup, 0: logits_k.  Up to 64 tokens (f32: 4096), where it
// takes less than the other way (times in us):
// - the other way: the stages' time in large_rows(), and for a forward that lays the
//   weights out first (f32) 12 bytes of each moved at 5 TB/s;
// - 16 bits: 5 and all that its workgroups load, 32 rows each, at 9 TB/s, as each 16 tokens
//   read the weights again from the L2s.  (32000 x 4096, 1 / 4 / 8 / 16 tokens: 49 / 50 /
//   55 / 63 against 51; 35 x 512 x 2560: 8 against 24.)  Rows that are not aligned take
//   longer, so that there it is left to up to 4 tokens (50257 x 1023: 60 for 1 and 98 for
//   16 against 68), which it takes in any case;
// - f32: 5 and, for each weight, what its 4 bytes take at 4.4 TB/s or the products of 64
//   tokens at 75 TFLOP/s (64 x 32000 x 4096: 222 against 596; 128: 424 against 602; 600 x
//   3000 x 2048: 98 against 110).
uint32_t few_groups(int t, uint32_t tokens, uint32_t rows, uint32_t tpad, uint32_t kpad, bool backward, bool direct) {
  if (t != kF32 && tokens <= 4) return 1;
  if (t != kF32 ? tokens > 64 || !direct : tokens > 4096) return 0;
  const uint64_t wg16 = (uint64_t)rows * (kTileV / 16) * ((tokens + 15) / 16);
  // (f32: 4 groups load less, 2 fill the CUs: 130 x 3003 x 520)
  const uint32_t groups = t != kF32 || tokens <= 16 ? 1 : tokens <= 32 || wg16 < 16 * 256 ? 2 : 4;
  const double weights = (double)rows * kTileV * kpad * 1e-6;  // millions
  const double flops = 2.0 * (double)up(tokens, 16 * groups) / 75.0;
  const double few = t == kF32 ? 5 + weights * (flops > 4 / 4.4 ? flops : 4 / 4.4) : 5 + wg16 * (64.0 * kpad) / 9e6;
  const uint64_t stages = kpad / kTileK * (t == kF32 ? kSegs : 1), big = rows * (uint64_t)((tpad + 255) / 256), small = 2 * rows * (uint64_t)(tpad / 128);
  const uint64_t c256 = (big + 255) / 256 * (143 * stages + 900);
  const uint64_t c128 = small <= 256 ? 75 * stages + 600 : (small + 511) / 512 * (85 * stages + 600);
  const double other = 0.01 * (double)(c256 < c128 ? c256 : c128) + (backward || t != kF32 ? 0 : 8 + weights * 12 / 5);
  return few < other ? groups : 0;
}

}  // namespace

XentWays xent_ways(const XentCall& c, const XentPlan& p, int t, bool backward) {
  XentWays w;
  auto rows16 = [&](size_t ld) { return t != kF32 && c.cols % kTileK == 0 && ld % 8 == 0 && ld <= (1u << 22); };
  w.direct = rows16(c.ld_weight);
  for (int r = 0; r < c.nranks; ++r)
    if (c.rows[r] && (uintptr_t)c.weights[r] % 16) w.direct = false;
  w.hidden_direct = rows16(c.ld_hidden) && (uintptr_t)c.hidden % 16 == 0;
  w.groups = few_groups(t, c.tokens, p.tiles, p.tpad, p.kpad, backward, w.direct && w.hidden_direct);
  // few_k reads its operands where they are, a backward's gradients the weights alone
  w.bytes = (backward ? w.direct : w.groups || (w.direct && w.hidden_direct)) ? p.bytes_in_place : p.bytes;
  return w;
}

uint64_t xent_bytes(uint32_t tokens, uint32_t cols, const size_t* rows, int nranks, int t, bool backward, bool in_place) {
  const XentPlan p = xent_plan(tokens, cols, rows, nranks, t, backward);
  const bool can = in_place && t != kF32 && cols % kTileK == 0;
  return can || (!backward && few_groups(t, tokens, p.tiles, p.tpad, p.kpad, backward, false)) ? p.bytes_in_place : p.bytes;
}

namespace {

template <int T, bool BWD> void few(const XentArgs& a, uint32_t few, hipStream_t s) {
  const uint32_t tokens = !BWD ? a.tokens : a.lo ? a.lo : (uint32_t)up(a.tokens, kTileK);
  const dim3 grid(a.ntiles * (kTileV / (16 * few)), (tokens + 16 * few - 1) / (16 * few));
  if (few == 1) hipLaunchKernelGGL((few_k<T, 1, 1, BWD>), grid, dim3(256), 0, s, a);
  if constexpr (T == kF32) {
    if (few == 2) hipLaunchKernelGGL((few_k<T, 2, 2, BWD>), grid, dim3(256), 0, s, a);
    if (few == 4) hipLaunchKernelGGL((few_k<T, 4, 4, BWD>), grid, dim3(256), 0, s, a);
  }
}

// 128 x 128 tiles go two a CU with 2 stages, or with 4 when there is one a CU anyway.
template <int M, int S, int NS, bool BWD, int SEG> void logits_of(const XentArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((logits_k<M, S, NS, BWD, SEG>), dim3(tile_grid(tiles_of(a.sub * kTileV, a.tpad, S))),
                     dim3(tile_threads(S)), 0, s, a);
}
// Of a forward, part0 moves past the pairs it writes.
template <int M, bool BWD, int SEG> void logits(XentArgs& a, hipStream_t s) {
  const uint32_t large = large_rows(a.ntiles, (a.tpad + 255) / 256, a.tpad / 128, a.kpad / kTileK * SEG);
  a.sub0 = 0;
  a.sub = large;
  if (a.sub) logits_of<M, 256, 2, BWD, SEG>(a, s);
  a.part0 += 2 * a.sub;
  a.sub0 = large;
  a.sub = a.ntiles - large;
  if (a.sub && tiles_of(a.sub * kTileV, a.tpad, 128) > 256) logits_of<M, 128, 2, BWD, SEG>(a, s);
  else if (a.sub) logits_of<M, 128, 4, BWD, SEG>(a, s);
  a.part0 += 4 * a.sub;
}
template <int M, int T, int S, int SEG> void grads_of(const XentArgs& a, bool dh, bool dw, hipStream_t s) {
  const uint64_t h = dh ? tiles_of(a.kpad, a.tpad, S) * a.splits : 0, w = dw ? tiles_of(a.kpad, a.sub * kTileV, S) : 0;
  const uint32_t hg = tile_grid(h), grid = hg + tile_grid(w);
  if (S == 256) hipLaunchKernelGGL((grads_k<M, T, 256, 2, SEG>), dim3(grid), dim3(512), 0, s, a, hg);
  else if (h + w > 256) hipLaunchKernelGGL((grads_k<M, T, 128, 2, SEG>), dim3(grid), dim3(256), 0, s, a, hg);
  else hipLaunchKernelGGL((grads_k<M, T, 128, 4, SEG>), dim3(grid), dim3(256), 0, s, a, hg);
}
// The hidden states' tiles go with the weights' of their size where both together are few
// rounds over the CUs (1001 x 32003 x 1023 f16: 252 to 235 us; 4096 x 128256 x 4096, 9
// rounds, 9.90 to 9.97 ms), or alone.
template <int M, int T, int SEG> void grads(XentArgs& a, int dh_tile, bool dh, bool dw, hipStream_t s) {
  const uint32_t large = dw ? large_rows(a.ntiles, (a.kpad + 255) / 256, (a.kpad + 127) / 128, a.tpad / kTileK * SEG) : 0u;
  const bool dh256 = dh && dh_tile == 256, dh128 = dh && !dh256;
  a.sub0 = 0;
  a.sub = large;
  const bool apart = dh256 && a.sub && tiles_of(a.kpad, a.tpad, 256) * a.splits + tiles_of(a.kpad, a.sub * kTileV, 256) > 4 * 256;
  if (apart) grads_of<M, T, 256, SEG>(a, true, false, s);
  if (dh256 || a.sub) grads_of<M, T, 256, SEG>(a, dh256 && !apart, a.sub != 0, s);
  a.sub0 = large;
  a.sub = dw ? a.ntiles - large : 0;
  if (dh128 || a.sub) grads_of<M, T, 128, SEG>(a, dh128, a.sub != 0, s);
}

// T: type of the caller's tensors.  M: type that multiplies.
template <int T, bool BWD> hipError_t run(const XentCall& c, const XentPlan& p, hipStream_t s) {
  constexpr int M = T == kF32 ? kBF16 : T, SEG = T == kF32 ? kSegs : 1;
  uint8_t* ws = (uint8_t*)c.workspace;
  XentArgs a{};
  uint64_t vocab = 0;
  const XentWays ways = xent_ways(c, p, T, BWD);
  const bool direct = ways.direct, hidden_direct = ways.hidden_direct;
  const uint32_t groups = ways.groups;
  a.v.n = c.nranks;
  for (int r = 0; r < c.nranks; ++r) {
    a.v.w[r] = c.weights[r];
    a.v.rows[r] = (uint32_t)c.rows[r];
    a.v.first_row[r] = (uint32_t)vocab;
    a.v.first_tile[r + 1] = a.v.first_tile[r] + (uint32_t)(up(c.rows[r], kTileV) / kTileV);
    vocab += c.rows[r];
    if (c.dweights) a.dw[r] = c.dweights[r];
  }
  a.ldw = direct ? (uint32_t)c.ld_weight * 2 : p.kpad * 2;
  a.laid_plane = p.laid_plane;
  a.h = ws + p.h;
  a.h_plane = p.h_plane;
  a.ldh = p.kpad * 2;
  a.tokens = c.tokens;
  a.tpad = p.tpad;
  a.cols = c.cols;
  a.kpad = p.kpad;
  a.targets = c.targets;
  a.ignore = c.ignore;
  // few_k reads the operands where they are
  a.hidden = c.hidden;
  a.ld_h = c.ld_hidden;
  a.ld_w = c.ld_weight;
  XentScalars* scalars = (XentScalars*)(ws + p.scalars);
  a.scalars = scalars;
  HitsArgs hits{};
  TokensArgs tk{};
  if constexpr (BWD) {
    a.dz = ws + p.dz;
    a.dz_plane = p.dz_plane;
    a.lddz = p.piece * kTileV * 2;
    a.sum = (float*)(ws + p.sum);
    a.splits = p.splits;
    a.token = (XentToken*)(ws + p.token);
    a.place = (int32_t*)(ws + p.place);
    a.idx = (const int32_t*)(ws + p.idx);
    a.residue = (float*)(ws + p.residue);
    a.lo = T == kF32 || c.tokens > 64 ? 0 : c.tokens > 32 ? 64 : 32;
    a.dhidden = c.dhidden;
    a.ld_dh = c.ld_hidden;
    a.ld_dw = c.ld_weight;
    tk = TokensArgs{c.targets, c.lse, c.dloss, c.dloss_stride, c.ignore, (int64_t)vocab, (XentToken*)(ws + p.token),
                    (int32_t*)(ws + p.idx), (int32_t*)(ws + p.place), scalars, c.tokens, p.tpad, a.lo, T == kF16};
    if (T != kF32 && c.dweights && !a.lo) {
      a.hits = (uint32_t*)(ws + p.hits);
      a.hits_first = (uint32_t*)(ws + p.hits_first);
      hits = HitsArgs{a.v, a.token, scalars, a.hits, a.hits_first, p.tiles};
    }
  } else {
    a.part = (float2*)(ws + p.part);
    a.zt = (float*)(ws + p.zt);
  }
  const bool lay = BWD || !groups;  // few_k reads the operands where they are
  LayoutArgs l{};
  if (BWD) hipLaunchKernelGGL(tokens_k, dim3(1), dim3(kTokensThreads), 0, s, tk);
  l.v = a.v;
  l.hidden = c.hidden;
  l.idx = a.idx;
  l.tokens = c.tokens;
  l.cols = c.cols;
  l.kpad = p.kpad;
  l.ld_hidden = c.ld_hidden;
  l.ld_weight = c.ld_weight;
  l.hidden_dst = ws + p.h;
  l.weight_dst = ws + p.laid;
  l.hidden_plane = p.h_plane;
  l.weight_plane = p.laid_plane;
  // a forward reads hidden states in place where it can
  if (!BWD && hidden_direct) {
    a.h = (const uint8_t*)c.hidden;
    a.ldh = (uint32_t)c.ld_hidden * 2;
  } else if (lay) {
    l.hidden_rows = p.tpad;
  }
  const uint32_t nt = p.tpad / 128 * 2;  // of the smaller tiles, in halves of a vocabulary tile
  // a forward that reads the weights in place has nothing to divide but the grid
  uint32_t piece = p.piece;
  if (!BWD && groups) piece = p.tiles < kMaxTiles / 8 ? p.tiles : (uint32_t)(kMaxTiles / 8);
  else if (!BWD && direct) piece = nt <= kMaxTiles / p.tiles ? p.tiles : kMaxTiles / nt ? (uint32_t)(kMaxTiles / nt) : 1;
  if (groups) a.parts = p.tiles * (kTileV / (16 * groups));
  for (a.tile0 = 0; a.tile0 < p.tiles; a.tile0 += piece) {
    a.ntiles = p.tiles - a.tile0 < piece ? p.tiles - a.tile0 : piece;
    if (!direct && lay) {
      l.tile0 = a.tile0;
      l.weight_rows = (uint64_t)a.ntiles * kTileV;
      a.laid = ws + p.laid;
    }
    layout<T>(l, hits, s);
    // once for the call
    l.hidden_rows = hits.tiles = 0;
    if (groups) few<T, BWD>(a, groups, s);
    else logits<M, BWD, SEG>(a, s);
    if constexpr (BWD) {
      grads<M, T, SEG>(a, p.dh_tile, c.dhidden != nullptr, c.dweights != nullptr, s);
      a.add = 1;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if constexpr (BWD) {
    if (c.dhidden) {
      const uint32_t y = (c.cols + 1023) / 1024;
      hipLaunchKernelGGL(dhidden_join_k<T>, dim3(c.tokens < 65536 ? c.tokens : 65536, y < 1024 ? y : 1024), dim3(256), 0, s, a);
    }
  } else {
    const uint64_t parts = groups ? a.parts : a.part0;
    const XentJoinArgs j{a.part, a.zt, c.targets, c.ignore, (int64_t)vocab, c.loss, c.lse_out,
                         groups ? 1u : c.tokens, groups ? parts : 1u, (uint32_t)parts, c.tokens};
    // as many chains as leave every CU a workgroup
    const uint32_t jt = groups ? 1 : c.tokens <= 1024 ? 4 : 16;
    const dim3 grid((c.tokens + jt - 1) / jt), block(kJoinThreads);
    if (jt == 1) hipLaunchKernelGGL(join_k<1>, grid, block, 0, s, j);
    else if (jt == 4) hipLaunchKernelGGL(join_k<4>, grid, block, 0, s, j);
    else hipLaunchKernelGGL(join_k<16>, grid, block, 0, s, j);
  }
  return hipGetLastError();
}

template <bool BWD> hipError_t typed(const XentCall& c, int t, hipStream_t s) {
  if (c.tokens == 0) {
    const uint32_t e = t == kF32 ? 4 : 2;
    for (int r = 0; c.dweights && r < c.nranks; ++r) {
      if (!c.dweights[r] || !c.rows[r]) continue;
      hipLaunchKernelGGL(zero_rows_k, dim3((uint32_t)(c.rows[r] < 65536 ? c.rows[r] : 65536)), dim3(256), 0, s,
                         (uint8_t*)c.dweights[r], c.rows[r], c.ld_weight * e, c.cols * (e / 2));
      const hipError_t err = hipGetLastError();
      if (err != hipSuccess) return err;
    }
    return hipSuccess;
  }
  const XentPlan p = xent_plan(c.tokens, c.cols, c.rows, c.nranks, t, BWD);
  if (t == kF32) return run<kF32, BWD>(c, p, s);
  if (t == kF16) return run<kF16, BWD>(c, p, s);
  return run<kBF16, BWD>(c, p, s);
}

}  // namespace

hipError_t launch_xent_fwd(const XentCall& c, int t, hipStream_t stream) { return typed<false>(c, t, stream); }
hipError_t launch_xent_bwd(const XentCall& c, int t, hipStream_t stream) { return typed<true>(c, t, stream); }

}  // namespace mrr
