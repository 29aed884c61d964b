// muon.hip -- matrices made orthogonal by Newton-Schulz products, alone and as the
// weights' update of a training step.
//
//   X_0 = G / (|G|_F + eps)                     G^T where it has more rows than columns
//   A = X X^T, B = b A + c A^2, X <- a X + B X  `steps` times, coefficients of each step
//
// takes every singular value s of X through the odd polynomial a s + b s^3 + c s^5.
//
// Bound by the matrix units: with m <= n the sides, a step is m^2 n + m^3 + 2 m^2 n
// operations, since A and B are symmetric and only the tiles on and below the diagonal are
// computed, and stored twice.
//
// Precision.  X is held in two f16 parts (22 bits), scaled so that neither loses bits: it is
// what passes from step to step, and a small singular value, which grows a-fold a step, must
// not carry the rounding of the large ones.  O and B have two parts as well (TWO) and a product
// is three of the parts', which leaves 2^-22 of each term.  The diagonals of A and B, which are
// far larger than what lies beside them, stay in f32 and out of the products:  with A = D + O,
//   A^2 = O O + D O + O D + D^2,   a X + B X = (a + diag B) X + off(B) X.
// Callers that ask for F16 get products of the upper parts alone (TWO false), 11 bits: they reach X
// only as a correction B X beside a X, which is added in f32 from both parts.  Such results are off
// by some 1e-3 of their norm for noise (1.5e-2 with X in one part and diagonals in f16), but rows
// that repeat round alike and their errors add: 3e-3 for two equal ones, up to 3e-2 for blocks of
// equal values.
#include <math.h>

#include "mrr_device.hpp"
#include "mrr_gemm.hpp"
#include "mrr_internal.hpp"
#include "mrr_ops.hpp"
#include "mrr_rows.hpp"

namespace mrr {
namespace {

// Scales of the f16 parts, powers of two.  ns_bounds() keeps singular values below 7.5 and
// B below 1000, so nothing overflows; what lies under 2^-24 of a scale's unit is 2^-37 of
// X's, 2^-33 of A's and 2^-30 of B's norm.
constexpr float kScaleX = 8192.0f, kScaleA = 512.0f, kScaleB = 64.0f;

// ---- parts -------------------------------------------------------------------------
// A matrix of `cols` columns (a multiple of 64) whose products take upper parts (TWO false):
// rows of f16, and the lower parts, of X alone, in a plane of their own.  In two parts:
// blocks of 32 columns, 64 bytes of upper parts and 64 of lower ones, which is what a
// stage of the products takes of a row.
template <bool TWO> __device__ __forceinline__ uint64_t place(uint32_t row, uint32_t col, uint32_t cols) {
  return TWO ? (uint64_t)row * cols * 4 + (col >> 5) * 128 + (col & 31) * 2 : ((uint64_t)row * cols + col) * 2;
}
struct Raw8 {
  u32x4 hi, lo;
};
// 8 values to an upper f16 part and what it leaves.
__device__ __forceinline__ Raw8 split8(const float* x) {
  Raw8 r;
  float h[8], l[8];
  r.hi = encode16<kF16>(x);
  decode16<kF16>(r.hi, h);
#pragma unroll
  for (int e = 0; e < 8; ++e) l[e] = x[e] - h[e];
  r.lo = encode16<kF16>(l);
  return r;
}
__device__ __forceinline__ void join8(const Raw8& r, float* x) {
  float l[8];
  decode16<kF16>(r.hi, x);
  decode16<kF16>(r.lo, l);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] += l[e];
}
// X, in two parts in any case: `plane` from the upper to the lower ones.
__device__ __forceinline__ Raw8 load_parts(const uint8_t* p, uint64_t plane) {
  return {*reinterpret_cast<const u32x4*>(p), *reinterpret_cast<const u32x4*>(p + plane)};
}
__device__ __forceinline__ void store_parts(uint8_t* p, uint64_t plane, const float* x) {
  const Raw8 r = split8(x);
  *reinterpret_cast<u32x4*>(p) = r.hi;
  *reinterpret_cast<u32x4*>(p + plane) = r.lo;
}
// O and B, in one part or two.
template <bool TWO> __device__ __forceinline__ Raw8 load_operand(const uint8_t* p) {
  if constexpr (TWO) return load_parts(p, 64);
  return {*reinterpret_cast<const u32x4*>(p), u32x4{0u, 0u, 0u, 0u}};
}
template <bool TWO> __device__ __forceinline__ void store_operand(uint8_t* p, const float* x) {
  if constexpr (TWO) store_parts(p, 64, x);
  else *reinterpret_cast<u32x4*>(p) = encode16<kF16>(x);
}

// 8 values of type T, of which the first n exist.
template <int T> __device__ __forceinline__ void load8(const void* p, int n, float* x) {
  if constexpr (T == kF32) {
    decode16<kF32>(load_raw<kF32>(p, n), x);
    decode16<kF32>(load_raw<kF32>((const float*)p + 4, n - 4), x + 4);
  } else {
    decode16<T>(load_raw<T>(p, n), x);
  }
}
template <int T> __device__ __forceinline__ void store8(void* p, int n, const float* x) {
  if constexpr (T == kF32) {
    store_raw<kF32>(p, n, encode16<kF32>(x));
    store_raw<kF32>((float*)p + 4, n - 4, encode16<kF32>(x + 4));
  } else {
    store_raw<T>(p, n, encode16<T>(x));
  }
}

// ---- what comes before the products ----------------------------------------------------
// Sums of squares are f64: f32 would overflow on large gradients and vanish on small ones.
constexpr int kSumThreads = 256;
constexpr uint32_t kMaxParts = 1024;  // workgroups that sum a matrix's squares

__device__ __forceinline__ void block_sum(double s, double* to) {
  __shared__ double lds[kSumThreads / 64];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kSumThreads / 64; ++k) s += lds[k];
    *to = s;
  }
}

// Squares of a matrix; rows side by side come as one row.
template <int T> __global__ void __launch_bounds__(kSumThreads) squares_k(NsSource src, double* partial) {
  const uint64_t units = (src.cols + 7) / 8, total = units * src.rows;
  const uint8_t* base = (const uint8_t*)src.p + blockIdx.y * src.stride * Ty<T>::size;
  double s = 0.0;
  for (uint64_t u = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x; u < total; u += (uint64_t)gridDim.x * kSumThreads) {
    const uint64_t row = src.rows == 1 ? 0 : u / units, c = (u - row * units) * 8;
    const uint64_t left = src.cols - c;
    float x[8];
    load8<T>(base + (row * src.ld + c) * Ty<T>::size, left < 8 ? (int)left : 8, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)x[e], (double)x[e], s);
  }
  block_sum(s, partial + (uint64_t)blockIdx.y * gridDim.x + blockIdx.x);
}

// g = scale sum of the ranks' gradients (rank order, f32), m' = mu m + g, and the squares of
// u = g + mu m' or m'.  u has a buffer of its own with `nesterov` only.
constexpr int kAtOnce = 4;  // ranks whose loads are in flight together
template <int T> __global__ void __launch_bounds__(kSumThreads) momentum_k(MuonArgs a, double* partial) {
  const uint64_t units = (a.cols + 7) / 8, total = units * a.rows, y = blockIdx.y;
  double s = 0.0;
  for (uint64_t i = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x; i < total; i += (uint64_t)gridDim.x * kSumThreads) {
    const uint64_t row = a.rows == 1 ? 0 : i / units, c = (i - row * units) * 8;
    const int n = a.cols - c < 8 ? (int)(a.cols - c) : 8;
    const uint64_t from = y * a.stride_grad + row * a.ld_grad + c, to = y * a.stride_weight + row * a.ld_weight + c;
    float g[8], m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] = -0.0f, m[e] = 0.0f;  // (the first sum is then exactly the first gradient)
    if (a.momentum) load8<kF32>(a.momentum + to, n, m);
    for (int r0 = 0; r0 < a.nranks; r0 += kAtOnce) {
      float x[kAtOnce][8];
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r)
        if (r0 + r < a.nranks) load8<T>(at<T>(a.grads[r0 + r], from), n, x[r]);
#pragma unroll
      for (int r = 0; r < kAtOnce; ++r) {
        if (r0 + r < a.nranks) {
#pragma unroll
          for (int e = 0; e < 8; ++e) g[e] += x[r][e];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= a.grad_scale;
#pragma unroll
    for (int e = 0; e < 8; ++e) m[e] = __builtin_fmaf(a.mu, m[e], g[e]);
    store8<kF32>(a.momentum_out + to, n, m);
    if (a.u) {
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = __builtin_fmaf(a.mu, m[e], g[e]);
      store8<kF32>(a.u + (y * a.rows + row) * a.cols + c, n, m);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)m[e], (double)m[e], s);
  }
  block_sum(s, partial + y * gridDim.x + blockIdx.x);
}

// X's scale over (norm + eps) for a sum of squares, as a power of two and the rest: norms at
// both ends of f32's range have inverses past the other.
struct Factor {
  float power, rest;
  __device__ __forceinline__ Factor(double squares, float eps) {
    const double norm = __builtin_sqrt(squares) + (double)eps, f = (double)kScaleX / norm;
    power = f > 0x1p100 ? 0x1p100f : f < 0x1p-100 ? 0x1p-100f : 1.0f;
    rest = norm == 0.0 ? 0.0f : (float)(f / (double)power);  // (a matrix of zeros, without eps, stays one)
  }
  __device__ __forceinline__ float operator()(float x) const { return x * power * rest; }
};

// The same in every thread of the workgroup.
__device__ __forceinline__ Factor inverse_norm(const double* partial, uint32_t parts, float eps) {
  __shared__ double lds[kSumThreads / 64];
  double s = 0.0;
#pragma unroll
  for (uint32_t i = 0; i < kMaxParts; i += kSumThreads)
    if (i + threadIdx.x < parts) s += partial[(uint64_t)blockIdx.y * parts + i + threadIdx.x];
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = lds[0];
#pragma unroll
  for (int k = 1; k < kSumThreads / 64; ++k) s += lds[k];
  return Factor(s, eps);
}

// The counters of the products' splits, of this matrix, set to zero by its first workgroup.
__device__ __forceinline__ void clear_counters(const NsArgs& a) {
  if (blockIdx.x) return;
  for (uint32_t i = threadIdx.x; i < a.counters; i += kSumThreads) a.counter[blockIdx.y * a.counters + i] = 0;
}

// X_0 in two parts, padded with zeros to whole tiles.
template <int T, bool TWO> __global__ void __launch_bounds__(kSumThreads) spread_k(NsSource src, NsArgs a, const double* partial, uint32_t parts, float eps) {
  clear_counters(a);
  const Factor scale = inverse_norm(partial, parts, eps);
  const uint8_t* base = (const uint8_t*)src.p + blockIdx.y * src.stride * Ty<T>::size;
  uint8_t* to = a.y + blockIdx.y * a.x_batch;
  const uint32_t units = a.np / 8;
  const uint64_t total = (uint64_t)units * a.mp;
  for (uint64_t u = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x; u < total; u += (uint64_t)gridDim.x * kSumThreads) {
    const uint32_t row = (uint32_t)(u / units), c = (uint32_t)(u - (uint64_t)row * units) * 8;
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (row < src.rows && c < src.cols) {
      const uint64_t left = src.cols - c;
      load8<T>(base + (row * src.ld + c) * Ty<T>::size, left < 8 ? (int)left : 8, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = scale(x[e]);
    }
    store_parts(to + place<TWO>(row, c, a.np), a.x_plane, x);
  }
}

// The same of the transpose: 64 x 64 through LDS.
template <int T, bool TWO> __global__ void __launch_bounds__(kSumThreads) turn_k(NsSource src, NsArgs a, const double* partial, uint32_t parts, float eps) {
  __shared__ float lds[64][65];
  clear_counters(a);
  const Factor scale = inverse_norm(partial, parts, eps);
  const uint8_t* base = (const uint8_t*)src.p + blockIdx.y * src.stride * Ty<T>::size;
  uint8_t* to = a.y + blockIdx.y * a.x_batch;
  const uint32_t across = a.mp / 64, r0 = blockIdx.x / across * 64, c0 = blockIdx.x % across * 64;  // of the source
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t r = k * 32 + threadIdx.x / 8, c = threadIdx.x % 8 * 8;
    float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (r0 + r < src.rows && c0 + c < src.cols) {
      const uint64_t left = src.cols - c0 - c;
      load8<T>(base + ((r0 + r) * src.ld + c0 + c) * Ty<T>::size, left < 8 ? (int)left : 8, x);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) lds[c + e][r] = x[e];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t r = k * 32 + threadIdx.x / 8, c = threadIdx.x % 8 * 8;  // of X
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = scale(lds[r][c + e]);
    store_parts(to + place<TWO>(c0 + r, r0 + c, a.np), a.x_plane, x);
  }
}

// Both passes over a matrix of few elements, by one workgroup: a launch less (50 x 50 f32: 47 us
// a call, 49 with two; 64 x 768 76, 74 with two, and 768 x 64 115 and 75).  TURN: the transpose,
// read element by element.
constexpr int kFewThreads = 1024;
constexpr uint64_t kFewElements = 16384;

template <int T, bool TWO, bool TURN> __global__ void __launch_bounds__(kFewThreads) few_k(NsSource src, NsArgs a, float eps) {
  __shared__ double lds[kFewThreads / 64];
  const uint8_t* base = (const uint8_t*)src.p + blockIdx.y * src.stride * Ty<T>::size;
  uint8_t* to = a.y + blockIdx.y * a.x_batch;
  for (uint32_t i = threadIdx.x; i < a.counters; i += kFewThreads) a.counter[blockIdx.y * a.counters + i] = 0;
  const uint32_t rows = (uint32_t)(TURN ? src.cols : src.rows), cols = (uint32_t)(TURN ? src.rows : src.cols);  // of X
  const uint32_t units = a.np / 8, total = units * a.mp;
  auto load = [&](uint32_t row, uint32_t c, float* x) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.0f;
    if (row >= rows || c >= cols) return;
    const int n = cols - c < 8 ? (int)(cols - c) : 8;
    if constexpr (TURN) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < n) x[e] = load_elem<T>(base, (c + e) * src.ld + row);
    } else {
      load8<T>(base + (row * src.ld + c) * Ty<T>::size, n, x);
    }
  };
  double s = 0.0;
  for (uint32_t u = threadIdx.x; u < total; u += kFewThreads) {
    float x[8];
    load(u / units, u % units * 8, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) s = __builtin_fma((double)x[e], (double)x[e], s);
  }
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = lds[0];
#pragma unroll
  for (int k = 1; k < kFewThreads / 64; ++k) s += lds[k];
  const Factor scale(s, eps);
  for (uint32_t u = threadIdx.x; u < total; u += kFewThreads) {
    float x[8];
    load(u / units, u % units * 8, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = scale(x[e]);
    store_parts(to + place<TWO>(u / units, u % units * 8, a.np), a.x_plane, x);
  }
}

// ---- the products -------------------------------------------------------------------
// Of a workgroup: its matrix, its tile, and one of `splits` parts of k.  An XCD gets whole matrices, or as
// much of one, where there are several: 4 matrices of 1024 x 4096 in 11 bits 525 us, 561 with
// each of them spread over all XCDs.
struct Part {
  uint32_t mat, split, tile;
};
__device__ __forceinline__ bool part_of(const NsArgs& a, uint32_t tiles, uint32_t splits, Part& p) {
  uint32_t t;
  if (!place_of(blockIdx.x, tiles * splits * a.batch, t)) return false;
  p.mat = __builtin_amdgcn_readfirstlane(t / (tiles * splits));
  t -= p.mat * (tiles * splits);
  p.split = __builtin_amdgcn_readfirstlane(t / tiles);
  p.tile = t - p.split * tiles;
  return true;
}

// Place t of an order of the tiles (row, column <= row) on and below the diagonal, `side` tiles a
// side, that walks 6 rows at a time, column by column.
__device__ __forceinline__ void lower_tile(uint32_t t, uint32_t side, uint32_t& r, uint32_t& c) {
  constexpr uint32_t G = 6;
  uint32_t r0 = 0, rows = side < G ? side : G;
  // a group of rows: r0 whole columns, then its triangle
  while (t >= r0 * rows + rows * (rows + 1) / 2) {
    t -= r0 * rows + rows * (rows + 1) / 2;
    r0 += rows;
    rows = side - r0 < G ? side - r0 : G;
  }
  if (t < r0 * rows) {
    c = t / rows;
    r = r0 + t % rows;
  } else {
    t -= r0 * rows;
    c = r0;
    for (uint32_t n = rows; t >= n; --n) t -= n, ++c;
    r = c + t;
  }
  r = __builtin_amdgcn_readfirstlane(r);
  c = __builtin_amdgcn_readfirstlane(c);
}

// The sums of `tile`'s splits, in the workgroup that comes last: true there.
// (Calls for tiles of 192 or more have enough of them.)
template <int S, class Prod> __device__ __forceinline__ bool whole(Prod& p, const NsArgs& a, uint32_t mat, uint32_t tile, uint32_t tiles,
                                                                   uint32_t split, uint32_t splits, lds8* lds) {
  __syncthreads();
  if (S >= 192 || splits == 1) return true;
  const uint64_t of = (uint64_t)mat * tiles + tile;
  return p.join(lds, a.part + of * splits * S * S, a.counter + mat * a.counters + tile, split, splits);
}

// A tile of P P^T for P = X (A = X X^T) or O (O O): both operands are rows of P, ld bytes
// apart, of `stages` 128 bytes.
template <class Prod, int S> __device__ __forceinline__ void square_tile(Prod& p, const uint8_t* base, uint64_t ld, uint32_t stages, uint32_t rows,
                                                                         uint32_t m0, uint32_t n0, uint32_t split, uint32_t splits, lds8* lds) {
  const int tid = threadIdx.x;
  uint32_t k = stages * split / splits;
  const uint32_t k1 = stages * (split + 1) / splits;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) {
        const uint32_t r = row_src_row<S>(tid, i);
        oa[i] = ob[i] = r * (uint32_t)ld + row_src_chunk(tid) * 16;
        if (S == 192) {  // (of sides that 192 does not divide: rows past the last are the last)
          oa[i] = (m0 + r < rows ? r : rows - 1 - m0) * (uint32_t)ld + row_src_chunk(tid) * 16;
          ob[i] = (n0 + r < rows ? r : rows - 1 - n0) * (uint32_t)ld + row_src_chunk(tid) * 16;
        }
      }
    }
    const uint8_t* at = base + (uint64_t)k * 128;
    pa = at + m0 * ld;
    pb = at + n0 * ld;
    ++k;
  };
  p.run((int)(k1 - k), lds, src);
}

// A = X X^T, tile (r, c): what lies beside the diagonal to O, the diagonal to d.  False in a
// workgroup whose split is not the last.
template <int S, int NS, bool TWO> __device__ __forceinline__ bool gram_tile(const NsArgs& a, uint32_t mat, uint32_t r, uint32_t c, uint32_t split,
                                                                             uint32_t splits, lds8* lds) {
  typedef Tile<kF16, false, false, S, NS, TWO> Prod;
  const uint32_t m0 = r * S, n0 = c * S, side = (a.mp + S - 1) / S;
  Prod p;
  square_tile<Prod, S>(p, a.x + mat * a.x_batch, (uint64_t)a.np * (TWO ? 4 : 2), a.n_stages, a.mp, m0, n0, split, splits, lds);
  if (!whole<S>(p, a, mat, r * (r + 1) / 2 + c, side * (side + 1) / 2, split, splits, lds)) return false;
  uint8_t* o = a.o + mat * a.o_batch;
  float* d = a.d + mat * a.mp;
  constexpr float unscale = 1.0f / (kScaleX * kScaleX);
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, true>(lds, j, [](int, int) { return 0; }, [&](int n, int m, float (&x)[8], int) {
      if (S == 192 && (n0 + n >= a.mp || m0 + m >= a.mp)) return;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= unscale;
        if (n0 + n == m0 + m + e) d[n0 + n] = x[e], x[e] = 0.0f;
        x[e] *= kScaleA;
      }
      store_operand<TWO>(o + place<TWO>(n0 + n, m0 + m, a.mp), x);
    }, [&](int m, int n, const float (&x)[8]) {
      if (r != c && (S != 192 || m0 + m < a.mp)) store_operand<TWO>(o + place<TWO>(m0 + m, n0 + n, a.mp), x);
    });
  return true;
}

// B = b A + c A^2, tile (r, c): what lies beside the diagonal to B, a + its diagonal to beta.
template <int S, int NS, bool TWO> __device__ __forceinline__ void poly_tile(const NsArgs& a, uint32_t mat, uint32_t r, uint32_t c, lds8* lds) {
  typedef Tile<kF16, false, false, S, NS, TWO> Prod;
  const uint32_t m0 = r * S, n0 = c * S;
  const uint8_t* o = a.o + mat * a.o_batch;
  uint8_t* b = a.b + mat * a.o_batch;
  const float* d = a.d + mat * a.mp;
  float* beta = a.beta + mat * a.mp;
  Prod p;
  square_tile<Prod, S>(p, o, (uint64_t)a.mp * (TWO ? 4 : 2), a.m_stages, a.mp, m0, n0, 0, 1, lds);
  __syncthreads();
  constexpr float unscale = 1.0f / (kScaleA * kScaleA);
  struct In {
    Raw8 o;
    f32x4 dm[2];
    float dn;
  };
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, true>(lds, j, [&](int n, int m) {
      const bool in = S != 192 || (n0 + n < a.mp && m0 + m < a.mp);
      const uint32_t row = in ? n0 + n : n0, col = in ? m0 + m : m0;
      const f32x4* dm = reinterpret_cast<const f32x4*>(d + col);
      return In{load_operand<TWO>(o + place<TWO>(row, col, a.mp)), {dm[0], dm[1]}, d[row]};
    }, [&](int n, int m, float (&x)[8], const In& in) {
      if (S == 192 && (n0 + n >= a.mp || m0 + m >= a.mp)) return;
      float y[8];
      if constexpr (TWO) join8(in.o, y);
      else decode16<kF16>(in.o.hi, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dm = in.dm[e / 4][e % 4], off = y[e] * (1.0f / kScaleA), sq = x[e] * unscale;
        x[e] = (a.cb * off + a.cc * (sq + (in.dn + dm) * off)) * kScaleB;
        if (n0 + n == m0 + m + e) beta[n0 + n] = a.ca + (a.cb * in.dn + a.cc * (sq + in.dn * in.dn)), x[e] = 0.0f;
      }
      store_operand<TWO>(b + place<TWO>(n0 + n, m0 + m, a.mp), x);
    }, [&](int m, int n, const float (&x)[8]) {
      if (r != c && (S != 192 || m0 + m < a.mp)) store_operand<TWO>(b + place<TWO>(m0 + m, n0 + n, a.mp), x);
    });
}

template <int S, int NS, bool TWO> constexpr int square_lds() { return Tile<kF16, false, false, S, NS, TWO>::kLds; }

template <int S, int NS, bool TWO> __global__ void __launch_bounds__(tile_threads(S)) gram_k(NsArgs a, uint32_t splits) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[square_lds<S, NS, TWO>()];
  const uint32_t side = (a.mp + S - 1) / S;
  uint32_t r, c;
  Part p;
  if (!part_of(a, side * (side + 1) / 2, splits, p)) return;
  lower_tile(p.tile, side, r, c);
  gram_tile<S, NS, TWO>(a, p.mat, r, c, p.split, splits, (lds8*)lds);
}

template <int S, int NS, bool TWO> __global__ void __launch_bounds__(tile_threads(S)) square_k(NsArgs a) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[square_lds<S, NS, TWO>()];
  const uint32_t side = (a.mp + S - 1) / S;
  uint32_t r, c;
  Part p;
  if (!part_of(a, side * (side + 1) / 2, 1, p)) return;
  lower_tile(p.tile, side, r, c);
  poly_tile<S, NS, TWO>(a, p.mat, r, c, (lds8*)lds);
}

// Both, of matrices that are one tile high: the workgroup that has A goes on to B (what it has
// stored it reads back past a barrier).  12 matrices of 64 x 768 f32: 88 us with two
// launches a step, 80 with one.
template <int NS, bool TWO> __global__ void __launch_bounds__(tile_threads(64)) short_k(NsArgs a, uint32_t splits) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[square_lds<64, NS, TWO>()];
  Part p;
  if (!part_of(a, 1, splits, p) || !gram_tile<64, NS, TWO>(a, p.mat, 0, 0, p.split, splits, (lds8*)lds)) return;
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  poly_tile<64, NS, TWO>(a, p.mat, 0, 0, (lds8*)lds);
}

// Results of the last step: X, or the weights' update by it, of 8 values of a row of the
// result, n of them in it.
template <int T> __device__ __forceinline__ void put_typed(const NsLast& z, uint64_t i, int n, float* x) {
  if (z.weight) {
    float w[8];
    load8<T>(at<T>(z.weight, i), n, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(-z.rate, x[e], z.keep * w[e]);
  }
  for (int r = 0; r < z.nranks; ++r) store8<T>(at<T>(z.out[r], i), n, x);
}
__device__ __forceinline__ void put_result(const NsLast& z, uint32_t mat, uint32_t row, uint32_t col, float* x) {
  if (row >= z.rows || col >= z.cols) return;
  const uint64_t i = mat * z.stride + (uint64_t)row * z.ld + col;
  const int n = z.cols - col < 8 ? (int)(z.cols - col) : 8;
  if (z.type == kF32) put_typed<kF32>(z, i, n, x);
  else if (z.type == kF16) put_typed<kF16>(z, i, n, x);
  else put_typed<kBF16>(z, i, n, x);
}

// X <- (a + diag B) X + off(B) X, in parts (LAST false) or as the result, TURN: transposed.
template <int S, int NS, bool TWO, bool LAST, bool TURN>
__global__ void __launch_bounds__(tile_threads(S)) apply_k(NsArgs a, NsLast z) {
  typedef Tile<kF16, true, false, S, NS, TWO> Prod;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Prod::kLds];
  uint32_t mt, nt;
  Part at;
  if (!part_of(a, a.np / S * (a.mp / S), 1, at)) return;
  tile_at(at.tile, a.np / S, a.mp / S, mt, nt);
  const uint32_t mat = at.mat;
  const uint32_t j0 = mt * S, i0 = nt * S;  // column and row of X
  const uint8_t* x = a.x + mat * a.x_batch;
  const uint8_t* b = a.b + mat * a.o_batch;
  const float* beta = a.beta + mat * a.mp;
  const int tid = threadIdx.x;
  const uint32_t ldx = a.np * (TWO ? 4 : 2), ldb = a.mp * (TWO ? 4 : 2);
  uint32_t k = 0;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) {
        const uint32_t kk = col_src_k<S>(tid, i), col = col_src_chunk<S>(tid) * 8;
        oa[i] = TWO ? (kk & 31) * ldx + (kk >> 5) * 64 + (col >> 5) * 128 + (col & 31) * 2 : kk * ldx + col * 2;
        ob[i] = row_src_row<S>(tid, i) * ldb + row_src_chunk(tid) * 16;
      }
    }
    pa = x + (uint64_t)k * (TWO ? 32 : 64) * ldx + j0 * (TWO ? 4 : 2);
    pb = b + (uint64_t)i0 * ldb + (uint64_t)k * 128;
    ++k;
  };
  Prod p;
  p.run((int)a.m_stages, (lds8*)lds, src);
  __syncthreads();
  struct In {
    Raw8 x;
    float beta;
  };
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, LAST && TURN>((lds8*)lds, j, [&](int n, int m) {
      return In{load_parts(x + place<TWO>(i0 + n, j0 + m, a.np), a.x_plane), beta[i0 + n]};
    }, [&](int n, int m, float (&v)[8], const In& in) {
      float y[8];
      join8(in.x, y);
      constexpr float unscale = LAST ? 1.0f / kScaleX : 1.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], unscale / kScaleB, in.beta * y[e] * unscale);
      if constexpr (!LAST) store_parts(a.y + mat * a.x_batch + place<TWO>(i0 + n, j0 + m, a.np), a.x_plane, v);
      else if constexpr (!TURN) put_result(z, mat, i0 + n, j0 + m, v);
    }, [&](int m, int n, float (&v)[8]) {
      if constexpr (LAST) put_result(z, mat, j0 + m, i0 + n, v);
    });
}

// ---- plans ---------------------------------------------------------------------------
uint32_t up(uint32_t n, uint32_t to) { return (n + to - 1) / to * to; }
uint64_t up64(uint64_t n) { return (n + 255) / 256 * 256; }

// The ways of a product: side of its tiles, stages in flight.  SQUARE: of row operands alone.
template <bool SQUARE, class Go> void way(const NsWay& w, bool two, Go&& go) {
  auto pick = [&](auto t) {
#define MRR_WAY(s, ns) go(std::integral_constant<int, s>(), std::integral_constant<int, ns>(), t)
    if (w.tile == 64) MRR_WAY(64, 4);
    else if (w.tile == 128 && w.stages == 4) MRR_WAY(128, 4);
    else if (w.tile == 128) MRR_WAY(128, 2);
    if constexpr (SQUARE) {
      if (w.tile == 192) MRR_WAY(192, 3);
    }
    if constexpr (!decltype(t)::value) {
      if (w.tile == 256) MRR_WAY(256, 2);
    }
#undef MRR_WAY
  };
  if (two) pick(std::true_type());
  else pick(std::false_type());
}

void step(const NsPlan& p, const NsArgs& a, const NsLast& z, uint32_t batch, bool last, bool turn, hipStream_t st) {
  auto lower = [&](const NsWay& w) {  // (with its splits)
    const uint64_t side = (a.mp + w.tile - 1) / w.tile;
    return dim3((uint32_t)(side * (side + 1) / 2 * w.splits * batch));
  };
  if (a.mp == 64) {
    // (sides of up to 64 always have two parts)
    hipLaunchKernelGGL((short_k<4, true>), lower(p.gram), dim3(tile_threads(64)), 0, st, a, p.gram.splits);
  } else {
    way<true>(p.gram, p.parts == 2, [&](auto s, auto ns, auto two) {
      hipLaunchKernelGGL((gram_k<s, ns, two>), lower(p.gram), dim3(tile_threads(s)), 0, st, a, p.gram.splits);
    });
    way<true>(p.square, p.parts == 2, [&](auto s, auto ns, auto two) {
      hipLaunchKernelGGL((square_k<s, ns, two>), lower(p.square), dim3(tile_threads(s)), 0, st, a);
    });
  }
  way<false>(p.apply, p.parts == 2, [&](auto s, auto ns, auto two) {
    const dim3 grid((a.mp / s) * (a.np / s) * batch), block(tile_threads(s));
    if (!last) hipLaunchKernelGGL((apply_k<s, ns, two, false, false>), grid, block, 0, st, a, z);
    else if (!turn) hipLaunchKernelGGL((apply_k<s, ns, two, true, false>), grid, block, 0, st, a, z);
    else hipLaunchKernelGGL((apply_k<s, ns, two, true, true>), grid, block, 0, st, a, z);
  });
}

// Workgroups of the passes over a matrix that sum its squares.
uint32_t sum_parts(uint64_t rows, uint64_t cols) {
  const uint64_t n = rows * cols / (kSumThreads * 32) + 1;
  return n < kMaxParts ? (uint32_t)n : kMaxParts;
}

// X_0 from the source, its squares summed already (parts of them; 0: few elements, not yet); then
// the steps.
hipError_t run_steps(const NsCall& c, const NsPlan& p, const NsSource& src, int t, uint32_t parts, const NsLast& z, hipStream_t s) {
  uint8_t* ws = (uint8_t*)c.workspace;
  const double* partial = (const double*)(ws + p.partial);
  const bool two = p.parts == 2, turn = c.rows > c.cols;
  NsArgs a{};
  a.x = a.y = ws + p.x;
  a.o = ws + p.o;
  a.b = ws + p.b;
  a.d = (float*)(ws + p.d);
  a.beta = (float*)(ws + p.beta);
  a.part = (float*)(ws + p.part);
  a.counter = (uint32_t*)(ws + p.counter);
  a.counters = p.counters;
  a.x_plane = two ? 64 : p.x_plane;
  a.x_batch = 2 * p.x_plane;
  a.o_batch = p.parts * p.o_plane;
  a.batch = c.batch;
  a.mp = p.mp;
  a.np = p.np;
  a.m_stages = p.m_stages;
  a.n_stages = p.n_stages;
  auto begin = [&](auto type, auto tw) {
    if (parts == 0) {
      if (turn) hipLaunchKernelGGL((few_k<type, tw, true>), dim3(1, c.batch), dim3(kFewThreads), 0, s, src, a, c.eps);
      else hipLaunchKernelGGL((few_k<type, tw, false>), dim3(1, c.batch), dim3(kFewThreads), 0, s, src, a, c.eps);
    } else if (turn) {
      hipLaunchKernelGGL((turn_k<type, tw>), dim3(a.mp / 64 * (a.np / 64), c.batch), dim3(kSumThreads), 0, s, src, a, partial, parts, c.eps);
    } else {
      const uint64_t blocks = ((uint64_t)a.mp * a.np / 8 + kSumThreads - 1) / kSumThreads;
      hipLaunchKernelGGL((spread_k<type, tw>), dim3((uint32_t)(blocks < 4096 ? blocks : 4096), c.batch), dim3(kSumThreads), 0, s, src, a,
                         partial, parts, c.eps);
    }
  };
  auto typed = [&](auto type) { two ? begin(type, std::true_type()) : begin(type, std::false_type()); };
  if (t == kF32) typed(std::integral_constant<int, kF32>());
  else if (t == kF16) typed(std::integral_constant<int, kF16>());
  else typed(std::integral_constant<int, kBF16>());
  for (int k = 0; k < c.steps; ++k) {
    a.x = ws + p.x + (k % 2) * p.x_bytes;
    a.y = ws + p.x + ((k + 1) % 2) * p.x_bytes;
    a.ca = c.coefficients[3 * k];
    a.cb = c.coefficients[3 * k + 1];
    a.cc = c.coefficients[3 * k + 2];
    step(p, a, z, c.batch, k + 1 == c.steps, turn, s);
  }
  return hipGetLastError();
}

template <int T> void squares(const NsSource& src, uint32_t batch, uint32_t parts, double* partial, hipStream_t s) {
  NsSource flat = src;
  if (src.ld == src.cols) flat.cols = src.rows * src.cols, flat.rows = 1;
  hipLaunchKernelGGL((squares_k<T>), dim3(parts, batch), dim3(kSumThreads), 0, s, flat, partial);
}

}  // namespace

bool ns_bounds(const float* co, int steps) {
  // the largest singular value before a step, and the polynomial's largest over all below;
  // 1 % above it, for what rounding adds
  double top = 1.0;
  for (int k = 0; k < steps; ++k) {
    const double a = co[3 * k], b = co[3 * k + 1], c = co[3 * k + 2], l = top * top;
    if (!(top < 7.5)) return false;
    // b x + c x^2 over [0, l]
    double most = fabs(b * l + c * l * l);
    if (c != 0.0 && -b / (2 * c) > 0.0 && -b / (2 * c) < l) most = fmax(most, fabs(b * b / (4 * c)));
    if (!(most < 1000.0)) return false;
    // a s + b s^3 + c s^5 over [0, top]: its ends, and where a + 3 b x + 5 c x^2 = 0
    auto value = [&](double x) { return fabs(sqrt(x) * (a + x * (b + x * c))); };
    double next = value(l);
    // (the roots by their sum and product, which lose no digits where one is far from the other;
    // where there is none, or c is 0, they are infinite or NaN and in no range)
    const double q = 9 * b * b - 20 * a * c;
    if (q >= 0.0) {
      const double t = -(3 * b + copysign(sqrt(q), b)) / 2;
      for (const double r : {t / (5 * c), a / t})
        if (r > 0.0 && r < l) next = fmax(next, value(r));
    }
    if (!(next < 1e30)) return false;
    top = 1.01 * next;
  }
  return true;
}

// The way of a product that a model of its time finds shortest: `tiles(s)` tiles of side s,
// in `stages` stages.  The times were measured with 256 CUs: a stage of a workgroup that has
// its CU to itself (64: what one CU draws from beyond its L2, 16 KiB in 0.25 us, bounds
// it, and neither more stages in flight nor fewer waits for LDS change that), of all that a
// CU holds, and what a workgroup's launch, first loads and end take.  520 x 1600 f32: 142 us
// with tiles of 64, 293 with 128; 2048 x 2048 in two parts 769 with 64, 648 with 128 and four stages in
// flight, 743 with two (in 11 bits 375, 342, 411); 4096 x 4096 in two parts 4092 with 128, 3656 with 192 for
// the symmetric products, in 11 bits 1807 with 128, 1481 with 256, 1467 with 192 for the symmetric
// ones (the 136 tiles of 256 leave CUs idle, the 253 of 192 do not).  Splits of k, up to `most`,
// for A = X X^T alone, whose k is the longer side: 8192 x 256 in two parts 309 us without, 148 with 8.  (The others' k is the
// shorter side: few tiles mean a short k there, and no shape of 400000 between 1 and 65536 a side had a use for them.)
template <class Tiles> static NsWay choose(uint32_t pad, bool two, bool square, uint64_t batch, uint32_t stages, uint32_t most, Tiles&& tiles) {
  struct Kind {
    uint32_t tile, ns, per_cu;
    double alone, full, rest, join;  // microseconds
  };
  static const Kind one[] = {{64, 4, 2, 0.23, 0.35, 3.4, 0.8}, {128, 4, 1, 0.55, 0.65, 5.5, 4.0}, {128, 2, 2, 0.62, 0.90, 6.7, 4.0},
                             {192, 3, 1, 0.98, 0.98, 20.0, 0.0}, {256, 2, 1, 1.43, 1.43, 14.0, 0.0}};
  static const Kind parts2[] = {{64, 4, 2, 0.23, 0.37, 3.4, 0.8}, {128, 4, 1, 0.55, 0.65, 5.5, 4.0}, {128, 2, 2, 0.65, 1.23, 5.5, 4.0},
                                 {192, 3, 1, 1.60, 1.60, 20.0, 0.0}};
  const Kind* kinds = two ? parts2 : one;
  NsWay best{};
  double least = 1e30;
  for (int i = 0; i < (two ? 4 : 5); ++i) {
    const Kind& k = kinds[i];
    if (k.tile == 192 ? !square : k.tile > pad) continue;
    for (uint32_t splits = 1; splits <= (k.tile >= 192 ? 1u : most) && splits <= stages; splits *= 2) {
      const uint64_t groups = tiles(k.tile) * batch * splits, slots = 256 * k.per_cu, rounds = groups / slots, rest = groups % slots;
      if (splits > 1 && groups > 512) break;
      const double per = (stages + splits - 1) / splits;
      const double last = rest ? per * (rest > 256 ? k.full : k.alone) + k.rest : 0.0;
      const double t = rounds * (per * k.full + k.rest) + last + (splits > 1 ? 2.0 + splits * k.join : 0.0);
      if (t < least) least = t, best = {k.tile, k.ns, splits, t};
    }
  }
  return best;
}

NsPlan ns_plan(uint64_t rows, uint64_t cols, uint64_t batch, int parts, bool with_u) {
  NsPlan p{};
  const uint32_t m = (uint32_t)(rows < cols ? rows : cols), n = (uint32_t)(rows < cols ? cols : rows);
  const bool two = parts == 2;
  const uint32_t deep = two ? 32 : 64;  // k of a stage
  p.parts = parts;
  p.m_stages = (m + deep - 1) / deep;
  p.n_stages = (n + deep - 1) / deep;
  double least = 1e30;
  for (uint32_t pad = 64; pad <= (two ? 128u : 256u); pad *= 2) {
    const uint32_t mp = up(m, pad), np = up(n, pad);
    auto lower = [&](uint32_t s) { return (uint64_t)((mp + s - 1) / s) * ((mp + s - 1) / s + 1) / 2; };
    const NsWay g = choose(pad, two, true, batch, p.n_stages, 8, lower), q = choose(pad, two, true, batch, p.m_stages, 1, lower),
                x = choose(pad, two, false, batch, p.m_stages, 1, [&](uint32_t s) { return (uint64_t)(mp / s) * (np / s); });
    const double t = g.us + q.us + x.us;
    if (t < least) least = t, p.gram = g, p.square = q, p.apply = x, p.mp = mp, p.np = np;
  }
  p.x_plane = (uint64_t)p.mp * p.np * 2;
  p.o_plane = (uint64_t)p.mp * p.mp * 2;
  p.x_bytes = 2 * p.x_plane * batch;
  const uint64_t o_bytes = parts * p.o_plane * batch;
  uint64_t part_bytes = 0;
  if (p.gram.splits > 1) {
    p.counters = p.mp / p.gram.tile * (p.mp / p.gram.tile + 1) / 2;
    part_bytes = (uint64_t)p.counters * batch * p.gram.splits * p.gram.tile * p.gram.tile * 4;
  }
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += up64(bytes);
    return here;
  };
  p.x = take(2 * p.x_bytes);
  p.o = take(o_bytes);
  p.b = take(o_bytes);
  p.d = take((uint64_t)p.mp * 4 * batch);
  p.beta = take((uint64_t)p.mp * 4 * batch);
  p.partial = take((uint64_t)kMaxParts * 8 * batch);
  p.part = take(part_bytes);
  p.counter = take((uint64_t)p.counters * 4 * batch);
  p.u = with_u ? take(rows * cols * 4 * batch) : 0;
  p.bytes = at;
  return p;
}

hipError_t launch_orthogonalize(const NsCall& c, const NsPlan& p, int t, hipStream_t s) {
  const NsSource src{c.in, c.rows, c.cols, c.ld_in, c.stride_in};
  const uint32_t parts = (uint64_t)p.mp * p.np <= kFewElements ? 0 : sum_parts(c.rows, c.cols);
  double* partial = (double*)((uint8_t*)c.workspace + p.partial);
  if (parts) {
    if (t == kF32) squares<kF32>(src, c.batch, parts, partial, s);
    else if (t == kF16) squares<kF16>(src, c.batch, parts, partial, s);
    else squares<kBF16>(src, c.batch, parts, partial, s);
  }
  NsLast z{};
  z.out[0] = c.out;
  z.nranks = 1;
  z.rows = (uint32_t)c.rows;
  z.cols = (uint32_t)c.cols;
  z.ld = c.ld_out;
  z.stride = c.stride_out;
  z.type = t;
  return run_steps(c, p, src, t, parts, z, s);
}

hipError_t launch_muon(const NsCall& c, const NsPlan& p, MuonArgs m, NsLast z, int tg, int tw, hipStream_t s) {
  uint8_t* ws = (uint8_t*)c.workspace;
  const uint32_t parts = sum_parts(c.rows, c.cols);
  if (m.u) m.u = (float*)(ws + p.u);
  NsSource src{m.momentum_out, c.rows, c.cols, m.ld_weight, m.stride_weight};
  if (m.u) src = {m.u, c.rows, c.cols, c.cols, c.rows * c.cols};
  m.rows = c.rows;
  m.cols = c.cols;
  if (m.ld_grad == c.cols && m.ld_weight == c.cols) m.cols = c.rows * c.cols, m.rows = 1;
  double* partial = (double*)(ws + p.partial);
  const dim3 grid(parts, c.batch), block(kSumThreads);
  if (tg == kF32) hipLaunchKernelGGL(momentum_k<kF32>, grid, block, 0, s, m, partial);
  else if (tg == kF16) hipLaunchKernelGGL(momentum_k<kF16>, grid, block, 0, s, m, partial);
  else hipLaunchKernelGGL(momentum_k<kBF16>, grid, block, 0, s, m, partial);
  z.rows = (uint32_t)c.rows;
  z.cols = (uint32_t)c.cols;
  z.type = tw;
  return run_steps(c, p, src, kF32, parts, z, s);
}

}  // namespace mrr
