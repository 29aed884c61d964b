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
// not carry the rounding of the large ones.  The products take the upper parts alone (PL 1),
// 11 bits: they reach X only as a correction B X beside a X, which is added in f32 from both
// parts.  The diagonals of A and B, which are far larger than what lies beside them, stay in
// f32 and out of the products:  with A = D + O,
//   A^2 = O O + D O + O D + D^2,   a X + B X = (a + diag B) X + off(B) X.
// The results are then off by their own rounding to 16 bits and up to 1.1e-3 beside it
// (with X in one part, diagonals in f16: 1.5e-2 where few singular values stand out of
// many).  For f32 and f16 results (PL 2) O and B have two parts as well and a product is
// three of the parts', which leaves 2^-22 of each term.
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
// 8 values to an upper f16 part and what it leaves.
__device__ __forceinline__ void split8(const float* x, u32x4& hi, u32x4& lo) {
  float h[8], l[8];
  hi = encode16<kF16>(x);
  decode16<kF16>(hi, h);
#pragma unroll
  for (int e = 0; e < 8; ++e) l[e] = x[e] - h[e];
  lo = encode16<kF16>(l);
}
template <bool LO> __device__ __forceinline__ void join8(const uint8_t* p, uint64_t plane, float* x) {
  decode16<kF16>(*reinterpret_cast<const u32x4*>(p), x);
  if constexpr (LO) {
    float l[8];
    decode16<kF16>(*reinterpret_cast<const u32x4*>(p + plane), l);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += l[e];
  }
}
template <bool LO> __device__ __forceinline__ void store_parts(uint8_t* p, uint64_t plane, const float* x) {
  u32x4 hi, lo;
  split8(x, hi, lo);
  *reinterpret_cast<u32x4*>(p) = hi;
  if constexpr (LO) *reinterpret_cast<u32x4*>(p + plane) = lo;
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
template <int T> __global__ void __launch_bounds__(kSumThreads) momentum_k(MuonArgs a, double* partial) {
  const uint64_t units = (a.cols + 7) / 8, total = units * a.rows, y = blockIdx.y;
  double s = 0.0;
  for (uint64_t i = (uint64_t)blockIdx.x * kSumThreads + threadIdx.x; i < total; i += (uint64_t)gridDim.x * kSumThreads) {
    const uint64_t row = a.rows == 1 ? 0 : i / units, c = (i - row * units) * 8;
    const int n = a.cols - c < 8 ? (int)(a.cols - c) : 8;
    const uint64_t from = y * a.stride_grad + row * a.ld_grad + c, to = y * a.stride_weight + row * a.ld_weight + c;
    float g[8], m[8];
    load8<T>(at<T>(a.grads[0], from), n, g);
    for (int r = 1; r < a.nranks; ++r) {
      float x[8];
      load8<T>(at<T>(a.grads[r], from), n, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) g[e] += x[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) g[e] *= a.grad_scale, m[e] = 0.0f;
    if (a.momentum) load8<kF32>(a.momentum + to, n, m);
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

// 1 / (norm + eps), times X's scale; every thread of the workgroup has it.
__device__ __forceinline__ float inverse_norm(const double* partial, uint32_t parts, float eps) {
  __shared__ double lds[kSumThreads / 64];
  double s = threadIdx.x < parts ? partial[(uint64_t)blockIdx.y * parts + threadIdx.x] : 0.0;
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) s += __shfl_xor(s, m);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = s;
  __syncthreads();
  s = lds[0];
#pragma unroll
  for (int k = 1; k < kSumThreads / 64; ++k) s += lds[k];
  const double norm = __builtin_sqrt(s) + (double)eps;
  // a matrix of zeros, without eps, stays one
  return norm == 0.0 ? 0.0f : (float)((double)kScaleX / norm);
}

// X_0 in two parts, padded with zeros to whole tiles.
template <int T> __global__ void __launch_bounds__(kSumThreads) spread_k(NsSource src, NsArgs a, const double* partial, uint32_t parts, float eps) {
  const float scale = inverse_norm(partial, parts, eps);
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
      for (int e = 0; e < 8; ++e) x[e] *= scale;
    }
    store_parts<true>(to + u * 16, a.x_plane, x);
  }
}

// The same of the transpose: 64 x 64 through LDS.
template <int T> __global__ void __launch_bounds__(kSumThreads) turn_k(NsSource src, NsArgs a, const double* partial, uint32_t parts, float eps) {
  __shared__ float lds[64][65];
  const float scale = inverse_norm(partial, parts, eps);
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
    for (int e = 0; e < 8; ++e) x[e] = lds[r][c + e] * scale;
    store_parts<true>(to + ((uint64_t)(c0 + r) * a.np + r0 + c) * 2, a.x_plane, x);
  }
}

// ---- the products -------------------------------------------------------------------
// The id-th tile (row, column <= row) on or below the diagonal, `side` tiles a side; XCDs
// get contiguous runs of the rows.
__device__ __forceinline__ bool lower_tile(uint32_t id, uint32_t side, uint32_t& r, uint32_t& c) {
  const uint32_t total = side * (side + 1) / 2, per = total / 8, extra = total % 8, x = id & 7, j = id >> 3;
  if (j >= per + (x < extra ? 1u : 0u)) return false;
  const uint32_t t = x * per + (x < extra ? x : extra) + j;
  r = (uint32_t)((__builtin_sqrtf(8.0f * (float)t + 1.0f) - 1.0f) * 0.5f);
  while (r * (r + 1) / 2 > t) --r;
  while ((r + 1) * (r + 2) / 2 <= t) ++r;
  c = t - r * (r + 1) / 2;
  return true;
}

// Parts that a product's seg-th pass takes: the small terms first.
template <int PL> __device__ __forceinline__ uint32_t part_a(uint32_t seg) { return PL == 2 && seg == 0 ? 1u : 0u; }
template <int PL> __device__ __forceinline__ uint32_t part_b(uint32_t seg) { return PL == 2 && seg == 1 ? 1u : 0u; }

// A tile of P P^T for P = X (A = X X^T) or O (O O): both operands are rows of P.
template <int S, int NS, int PL> __device__ __forceinline__ void
square_tile(Tile<kF16, false, false, S, NS>& p, const uint8_t* base, uint64_t plane, uint32_t ld, uint32_t k64, uint32_t m0,
            uint32_t n0, lds8* lds) {
  typedef Tile<kF16, false, false, S, NS> Prod;
  const int tid = threadIdx.x;
  uint32_t k = 0, seg = 0;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) oa[i] = ob[i] = row_src_row<S>(tid, i) * ld + row_src_chunk(tid) * 16;
    }
    const uint8_t* at = base + (uint64_t)k * (kTileK * 2);
    pa = at + (uint64_t)m0 * ld + part_a<PL>(seg) * plane;
    pb = at + (uint64_t)n0 * ld + part_b<PL>(seg) * plane;
    if (++k == k64) k = 0, ++seg;
  };
  p.run((int)k64 * (PL == 2 ? 3 : 1), lds, src);
}

// A = X X^T: what lies beside the diagonal to O, the diagonal to d.
template <int S, int NS, int PL> __global__ void __launch_bounds__(tile_threads(S)) gram_k(NsArgs a) {
  typedef Tile<kF16, false, false, S, NS> Prod;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Prod::kLds];
  uint32_t r, c;
  if (!lower_tile(blockIdx.x, a.mp / S, r, c)) return;
  const uint32_t m0 = r * S, n0 = c * S;
  Prod p;
  square_tile<S, NS, PL>(p, a.x + blockIdx.y * a.x_batch, a.x_plane, a.np * 2, a.n64, m0, n0, (lds8*)lds);
  __syncthreads();
  uint8_t* o = a.o + blockIdx.y * a.o_batch;
  float* d = a.d + blockIdx.y * a.mp;
  constexpr float unscale = 1.0f / (kScaleX * kScaleX);
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, true>((lds8*)lds, j, [&](int n, int m, float (&x)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] *= unscale;
        if (n0 + n == m0 + m + e) d[n0 + n] = x[e], x[e] = 0.0f;
        x[e] *= kScaleA;
      }
      store_parts<PL == 2>(o + ((uint64_t)(n0 + n) * a.mp + m0 + m) * 2, a.o_plane, x);
    }, [&](int m, int n, const float (&x)[8]) {
      if (r != c) store_parts<PL == 2>(o + ((uint64_t)(m0 + m) * a.mp + n0 + n) * 2, a.o_plane, x);
    });
}

// B = b A + c A^2: what lies beside the diagonal to B, a + its diagonal to beta.
template <int S, int NS, int PL> __global__ void __launch_bounds__(tile_threads(S)) square_k(NsArgs a) {
  typedef Tile<kF16, false, false, S, NS> Prod;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Prod::kLds];
  uint32_t r, c;
  if (!lower_tile(blockIdx.x, a.mp / S, r, c)) return;
  const uint32_t m0 = r * S, n0 = c * S;
  const uint8_t* o = a.o + blockIdx.y * a.o_batch;
  uint8_t* b = a.b + blockIdx.y * a.o_batch;
  const float* d = a.d + blockIdx.y * a.mp;
  float* beta = a.beta + blockIdx.y * a.mp;
  Prod p;
  square_tile<S, NS, PL>(p, o, a.o_plane, a.mp * 2, a.m64, m0, n0, (lds8*)lds);
  __syncthreads();
  constexpr float unscale = 1.0f / (kScaleA * kScaleA);
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, true>((lds8*)lds, j, [&](int n, int m, float (&x)[8]) {
      const uint64_t at = ((uint64_t)(n0 + n) * a.mp + m0 + m) * 2;
      float y[8];
      join8<PL == 2>(o + at, a.o_plane, y);
      const float dn = d[n0 + n];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float dm = d[m0 + m + e], off = y[e] * (1.0f / kScaleA), sq = x[e] * unscale;
        x[e] = (a.cb * off + a.cc * (sq + (dn + dm) * off)) * kScaleB;
        if (n0 + n == m0 + m + e) beta[n0 + n] = a.ca + (a.cb * dn + a.cc * (sq + dn * dn)), x[e] = 0.0f;
      }
      store_parts<PL == 2>(b + at, a.o_plane, x);
    }, [&](int m, int n, const float (&x)[8]) {
      if (r != c) store_parts<PL == 2>(b + ((uint64_t)(m0 + m) * a.mp + n0 + n) * 2, a.o_plane, x);
    });
}

// Results of the last step: X, or the weights' update by it, of 8 values of a row of the
// result, n of them in it.
template <int OUT> __device__ __forceinline__ void put_result(const NsLast& z, uint64_t at8, int n, float* x) {
  if (z.weight) {
    float w[8];
    load8<OUT>(at<OUT>(z.weight, at8), n, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = __builtin_fmaf(-z.rate, x[e], z.keep * w[e]);
  }
  for (int r = 0; r < z.nranks; ++r) store8<OUT>(at<OUT>(z.out[r], at8), n, x);
}

// X <- (a + diag B) X + off(B) X, in parts (OUT 0) or as the result.
template <int S, int NS, int PL, int OUT, bool TURN> __global__ void __launch_bounds__(tile_threads(S)) apply_k(NsArgs a, NsLast z) {
  typedef Tile<kF16, true, false, S, NS> Prod;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[Prod::kLds];
  uint32_t mt, nt, split;
  if (!tile_of(blockIdx.x, a.np / S, a.mp / S, 1, mt, nt, split)) return;
  const uint32_t j0 = mt * S, i0 = nt * S;  // column and row of X
  const uint8_t* x = a.x + blockIdx.y * a.x_batch;
  const uint8_t* b = a.b + blockIdx.y * a.o_batch;
  const float* beta = a.beta + blockIdx.y * a.mp;
  const int tid = threadIdx.x;
  const uint32_t ldx = a.np * 2, ldb = a.mp * 2;
  uint32_t k = 0, seg = 0;
  auto src = [&](int s, const uint8_t*& pa, const uint8_t*& pb, uint32_t (&oa)[Prod::L], uint32_t (&ob)[Prod::L]) {
    if (s == 0) {
#pragma unroll
      for (int i = 0; i < Prod::L; ++i) {
        oa[i] = col_src_k<S>(tid, i) * ldx + col_src_chunk<S>(tid) * 16;
        ob[i] = row_src_row<S>(tid, i) * ldb + row_src_chunk(tid) * 16;
      }
    }
    pa = x + part_a<PL>(seg) * a.x_plane + (uint64_t)k * kTileK * ldx + j0 * 2;
    pb = b + part_b<PL>(seg) * a.o_plane + (uint64_t)i0 * ldb + (uint64_t)k * (kTileK * 2);
    if (++k == a.m64) k = 0, ++seg;
  };
  Prod p;
  p.run((int)a.m64 * (PL == 2 ? 3 : 1), (lds8*)lds, src);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < Prod::FN; ++j)
    p.template both_out<8, TURN>((lds8*)lds, j, [&](int n, int m, float (&v)[8]) {
      const uint32_t row = i0 + n, col = j0 + m;
      const uint64_t at = ((uint64_t)row * a.np + col) * 2;
      float y[8];
      join8<true>(x + at, a.x_plane, y);
      const float bt = beta[row];
      if constexpr (OUT == 0) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], 1.0f / kScaleB, bt * y[e]);
        store_parts<true>(a.y + blockIdx.y * a.x_batch + at, a.x_plane, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], 1.0f / (kScaleB * kScaleX), bt * y[e] * (1.0f / kScaleX));
        if (!TURN && row < z.rows && col < z.cols)
          put_result<OUT>(z, blockIdx.y * z.stride + (uint64_t)row * z.ld + col, z.cols - col < 8 ? (int)(z.cols - col) : 8, v);
      }
    }, [&](int m, int n, float (&v)[8]) {
      if constexpr (OUT != 0) {
        const uint32_t row = j0 + m, col = i0 + n;
        if (row < z.rows && col < z.cols)
          put_result<OUT>(z, blockIdx.y * z.stride + (uint64_t)row * z.ld + col, z.cols - col < 8 ? (int)(z.cols - col) : 8, v);
      }
    });
}

// ---- plans ---------------------------------------------------------------------------
uint32_t up(uint32_t n, uint32_t to) { return (n + to - 1) / to * to; }
uint64_t up64(uint64_t n) { return (n + 255) / 256 * 256; }

template <int S, int PL> void products(const NsArgs& a, uint32_t batch, hipStream_t s) {
  const uint32_t side = a.mp / S;
  const dim3 grid(tile_grid((uint64_t)side * (side + 1) / 2), batch), block(tile_threads(S));
  hipLaunchKernelGGL((gram_k<S, 2, PL>), grid, block, 0, s, a);
  hipLaunchKernelGGL((square_k<S, 2, PL>), grid, block, 0, s, a);
}

template <int S, int PL> void apply(const NsArgs& a, const NsLast& z, uint32_t batch, int out, bool turn, hipStream_t s) {
  const dim3 grid(tile_grid((uint64_t)(a.mp / S) * (a.np / S)), batch), block(tile_threads(S));
  auto go = [&](auto o, auto t) { hipLaunchKernelGGL((apply_k<S, 2, PL, o, t>), grid, block, 0, s, a, z); };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  if (out == 0) go(std::integral_constant<int, 0>(), no);
  else if (out == kF32) turn ? go(std::integral_constant<int, kF32>(), yes) : go(std::integral_constant<int, kF32>(), no);
  else if (out == kF16) turn ? go(std::integral_constant<int, kF16>(), yes) : go(std::integral_constant<int, kF16>(), no);
  else turn ? go(std::integral_constant<int, kBF16>(), yes) : go(std::integral_constant<int, kBF16>(), no);
}

template <int S> void step(const NsArgs& a, const NsLast& z, uint32_t batch, int parts, int out, bool turn, hipStream_t s) {
  if (parts == 2) products<S, 2>(a, batch, s), apply<S, 2>(a, z, batch, out, turn, s);
  else products<S, 1>(a, batch, s), apply<S, 1>(a, z, batch, out, turn, s);
}

// Workgroups of the passes over a matrix that sum its squares.
uint32_t sum_parts(uint64_t rows, uint64_t cols) {
  const uint64_t n = rows * cols / (kSumThreads * 32) + 1;
  return n < kSumThreads ? (uint32_t)n : (uint32_t)kSumThreads;
}

// X_0 from the source, its squares summed already; then the steps.
hipError_t run_steps(const NsCall& c, const NsPlan& p, const NsSource& src, int t, uint32_t parts, const NsLast& z, int out, hipStream_t s) {
  uint8_t* ws = (uint8_t*)c.workspace;
  const double* partial = (const double*)(ws + p.partial);
  NsArgs a{};
  a.x = a.y = ws + p.x;
  a.o = ws + p.o;
  a.b = ws + p.b;
  a.d = (float*)(ws + p.d);
  a.beta = (float*)(ws + p.beta);
  a.x_plane = p.x_plane;
  a.x_batch = 2 * p.x_plane;
  a.o_plane = p.o_plane;
  a.o_batch = p.parts * p.o_plane;
  a.mp = p.mp;
  a.np = p.np;
  const bool turn = c.rows > c.cols;
  a.m64 = (uint32_t)((turn ? c.cols : c.rows) + kTileK - 1) / kTileK;
  a.n64 = (uint32_t)((turn ? c.rows : c.cols) + kTileK - 1) / kTileK;
  auto begin = [&](auto type) {
    if (turn) {
      hipLaunchKernelGGL((turn_k<type>), dim3(a.mp / 64 * (a.np / 64), c.batch), dim3(kSumThreads), 0, s, src, a, partial, parts, c.eps);
    } else {
      const uint64_t blocks = ((uint64_t)a.mp * a.np / 8 + kSumThreads - 1) / kSumThreads;
      hipLaunchKernelGGL((spread_k<type>), dim3((uint32_t)(blocks < 4096 ? blocks : 4096), c.batch), dim3(kSumThreads), 0, s, src, a, partial,
                         parts, c.eps);
    }
  };
  if (t == kF32) begin(std::integral_constant<int, kF32>());
  else if (t == kF16) begin(std::integral_constant<int, kF16>());
  else begin(std::integral_constant<int, kBF16>());
  for (int k = 0; k < c.steps; ++k) {
    a.x = ws + p.x + (k % 2) * p.x_bytes;
    a.y = ws + p.x + ((k + 1) % 2) * p.x_bytes;
    a.ca = c.coefficients[3 * k];
    a.cb = c.coefficients[3 * k + 1];
    a.cc = c.coefficients[3 * k + 2];
    const int to = k + 1 == c.steps ? out : 0;
    if (p.tile == 256) step<256>(a, z, c.batch, p.parts, to, turn, s);
    else step<128>(a, z, c.batch, p.parts, to, turn, s);
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
  // the largest singular value before a step, and the polynomial's largest over all below
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
    const double q = 9 * b * b - 20 * a * c;
    if (c != 0.0 && q >= 0.0) {
      for (const double r : {(-3 * b + sqrt(q)) / (10 * c), (-3 * b - sqrt(q)) / (10 * c)})
        if (r > 0.0 && r < l) next = fmax(next, value(r));
    } else if (c == 0.0 && b != 0.0) {
      const double r = -a / (3 * b);
      if (r > 0.0 && r < l) next = fmax(next, value(r));
    }
    if (!(next < 1e30)) return false;
    top = next;
  }
  return true;
}

NsPlan ns_plan(uint64_t rows, uint64_t cols, uint64_t batch, int parts, bool with_u) {
  NsPlan p{};
  const uint32_t m = (uint32_t)(rows < cols ? rows : cols), n = (uint32_t)(rows < cols ? cols : rows);
  p.parts = parts;
  const uint64_t big = (uint64_t)(up(m, 256) / 256) * (up(n, 256) / 256) * batch;
  p.tile = big >= 200 ? 256 : 128;
  p.mp = up(m, p.tile);
  p.np = up(n, p.tile);
  p.x_plane = (uint64_t)p.mp * p.np * 2;
  p.o_plane = (uint64_t)p.mp * p.mp * 2;
  p.x_bytes = 2 * p.x_plane * batch;
  const uint64_t o_bytes = parts * p.o_plane * batch;
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
  p.partial = take((uint64_t)kSumThreads * 8 * batch);
  p.u = with_u ? take(rows * cols * 4 * batch) : 0;
  p.bytes = at;
  return p;
}

hipError_t launch_orthogonalize(const NsCall& c, const NsPlan& p, int t, hipStream_t s) {
  const NsSource src{c.in, c.rows, c.cols, c.ld_in, c.stride_in};
  const uint32_t parts = sum_parts(c.rows, c.cols);
  double* partial = (double*)((uint8_t*)c.workspace + p.partial);
  if (t == kF32) squares<kF32>(src, c.batch, parts, partial, s);
  else if (t == kF16) squares<kF16>(src, c.batch, parts, partial, s);
  else squares<kBF16>(src, c.batch, parts, partial, s);
  NsLast z{};
  z.out[0] = c.out;
  z.nranks = 1;
  z.rows = (uint32_t)c.rows;
  z.cols = (uint32_t)c.cols;
  z.ld = c.ld_out;
  z.stride = c.stride_out;
  return run_steps(c, p, src, t, parts, z, t, s);
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
  return run_steps(c, p, src, kF32, parts, z, tw, s);
}

}  // namespace mrr
