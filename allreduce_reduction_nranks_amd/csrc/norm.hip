// norm.hip -- layer norm of the sum of N rank buffers and a residual, and its
// gradient.
//
//   h    = round(x_0 + ... + x_{N-1} + res)        summed in that order in f32
//   mu   = mean(h), var = mean((h - mu)^2), rs = 1 / sqrt(var + eps)
//   y    = (h - mu) rs w + b
//
//   xhat = (h - mu) rs, g = dy w
//   dh   = rs (g - mean(g) - xhat mean(g xhat)) + dres
//   dw   = sum over rows of dy xhat, db = sum over rows of dy
//
// Both are HBM-bound: a few operations an element against 2 or 4 bytes of each
// tensor.  A row is held in the registers of TPR lanes, E elements a lane, so
// every tensor is read once; the variance is the mean of squared differences
// from the finished mean, which loses nothing when the mean is large.  Statistics,
// sums and the weight gradients are f32 throughout; the stored h and y are
// rounded once each, and y is the norm of the stored (rounded) h, so that the
// gradient, which reads h, is that of the same function.
//
// A lane's elements come in units of 16 bytes, unit u of a lane being unit
// u * TPR + lane of the row: a wave's loads are contiguous.  Rows need no
// alignment beyond their element's: gfx950 loads 16 bytes from any address, and
// only the row's last, partial unit goes element by element.
#include "mrr_device.hpp"
#include "mrr_internal.hpp"
#include "mrr_ops.hpp"
#include "mrr_rows.hpp"

namespace mrr {
namespace {

// The same past the caches (NT) or through them.
template <int T, bool NT> __device__ __forceinline__ u32x4 load_in(const void* p, int n) {
  if (NT && n >= Vec<T>::VW) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  return load_raw<T>(p, n);
}
template <int T, bool NT> __device__ __forceinline__ void store_out(void* p, int n, u32x4 v) {
  if (NT && n >= Vec<T>::VW) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  else store_raw<T>(p, n, v);
}

// V weights from column c on, widened; `fill` where there is no weight.
template <int T>
__device__ __forceinline__ void load_weights(const void* w, int wf32, uint32_t c, int n, float fill,
                                             float* x) {
  constexpr int V = Vec<T>::VW;
  if (!w) {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = fill;
  } else if (T == kF32 || wf32) {
#pragma unroll
    for (int h = 0; h < V / 4; ++h) decode16<kF32>(load_raw<kF32>(at<kF32>(w, c + 4 * h), n - 4 * h), x + 4 * h);
  } else {
    decode16<T>(load_raw<T>(at<T>(w, c), n), x);
  }
}

// Sum of one value, or of two, over the TPR lanes of a row.  Rows of more than a
// wave join through LDS, in wave order; `lds` holds 2 values a wave, and the
// caller alternates between two such areas so that one barrier is enough.
template <int TPR> __device__ __forceinline__ float2 row_sum(float2 v, float2* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) {
    v.x += __shfl_xor(v.x, m);
    v.y += __shfl_xor(v.y, m);
  }
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) lds[wave] = v;
    __syncthreads();
    const int first = wave / (TPR / 64) * (TPR / 64);
    v = lds[first];
#pragma unroll
    for (int k = 1; k < TPR / 64; ++k) {
      const float2 o = lds[first + k];
      v.x += o.x;
      v.y += o.y;
    }
  }
  return v;
}

// Lanes of a workgroup: rows of up to 256 lanes share one of 256.
constexpr int block_threads(int tpr) { return tpr < 256 ? 256 : tpr; }

// Elements of a lane's unit at column c that exist.
__device__ __forceinline__ int unit_left(uint32_t cols, uint32_t c) { return c < cols ? (int)(cols - c) : 0; }

template <int T, int TPR, int E, bool NTL, bool NTS>
__global__ void __launch_bounds__(block_threads(TPR)) norm_fwd_k(NormFwdArgs a) {
  constexpr int V = Vec<T>::VW, U = E / V, RPB = block_threads(TPR) / TPR;
  // ranks whose loads are in flight together
  constexpr int G = U >= 4 ? 2 : 4;
  __shared__ float2 lds[2][block_threads(TPR) / 64];
  const uint32_t lane = threadIdx.x % TPR;
  const uint32_t sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  // every lane of a workgroup walks the same number of rows, as they share barriers
  for (uint64_t row0 = (uint64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (uint64_t)gridDim.x * RPB) {
    const uint64_t row = row0 + sub;
    const bool live = row < a.rows;
    float x[E];
    u32x4 raw[G][U];
    for (int r0 = 0; r0 < a.nranks; r0 += G) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (r0 + g < a.nranks) {
          const uint8_t* p = at<T>(a.in[r0 + g], row * a.ld_in);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const uint32_t c = (u * TPR + lane) * V;
            raw[g][u] = load_in<T, NTL>(p + (uint64_t)c * Ty<T>::size, live ? unit_left(a.cols, c) : 0);
          }
        }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (r0 + g < a.nranks) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float d[V];
            decode16<T>(raw[g][u], d);
#pragma unroll
            for (int j = 0; j < V; ++j) x[u * V + j] = r0 + g == 0 ? d[j] : x[u * V + j] + d[j];
          }
        }
      }
    }
    if (a.residual) {
      const uint8_t* p = at<T>(a.residual, row * a.ld_in);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t c = (u * TPR + lane) * V;
        raw[0][u] = load_in<T, NTL>(p + (uint64_t)c * Ty<T>::size, live ? unit_left(a.cols, c) : 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float d[V];
        decode16<T>(raw[0][u], d);
#pragma unroll
        for (int j = 0; j < V; ++j) x[u * V + j] += d[j];
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const u32x4 h = encode16<T>(x + u * V);
      if (a.sum) {
        const uint32_t c = (u * TPR + lane) * V;
        store_out<T, NTS>(at<T>(a.sum, row * a.ld_out + c), live ? unit_left(a.cols, c) : 0, h);
      }
      decode16<T>(h, x + u * V);
#pragma unroll
      for (int j = 0; j < V; ++j) s += x[u * V + j];  // elements past the row are zeros
    }
    const float mean = row_sum<TPR>(make_float2(s, 0.0f), lds[0]).x * inv;
    float q = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = unit_left(a.cols, (u * TPR + lane) * V);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = x[u * V + j] - mean;
        x[u * V + j] = d;
        if (j < n) q = __builtin_fmaf(d, d, q);
      }
    }
    const float var = row_sum<TPR>(make_float2(q, 0.0f), lds[1]).x * inv;
    const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
    if (live && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = (u * TPR + lane) * V;
      const int n = live ? unit_left(a.cols, c) : 0;
      float w[V], b[V];
      load_weights<T>(a.weight, a.wf32, c, n, 1.0f, w);
      load_weights<T>(a.bias, a.wf32, c, n, 0.0f, b);
#pragma unroll
      for (int j = 0; j < V; ++j) b[j] = __builtin_fmaf(x[u * V + j] * rstd, w[j], b[j]);
      store_out<T, NTS>(at<T>(a.out, row * a.ld_out + c), n, encode16<T>(b));
    }
  }
}

// Rows too long for registers: the same three passes with the sum computed
// again in each.  Element by element; a lane reads what it overwrites, so the
// outputs may take an input's place here too.
constexpr int kWideThreads = 1024;

template <int T> __device__ __forceinline__ float rank_sum(const NormFwdArgs& a, uint64_t i) {
  float s = load_elem<T>(a.in[0], i);
  for (int r = 1; r < a.nranks; ++r) s += load_elem<T>(a.in[r], i);
  if (a.residual) s += load_elem<T>(a.residual, i);
  return to_f32<T>(from_f32<T>(s));
}

template <int T> __global__ void __launch_bounds__(kWideThreads) norm_fwd_wide_k(NormFwdArgs a) {
  __shared__ float2 lds[2][kWideThreads / 64];
  const float inv = 1.0f / (float)a.cols;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const uint64_t in = row * a.ld_in, out = row * a.ld_out;
    float s = 0.0f;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kWideThreads) s += rank_sum<T>(a, in + c);
    const float mean = row_sum<kWideThreads>(make_float2(s, 0.0f), lds[0]).x * inv;
    float q = 0.0f;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float d = rank_sum<T>(a, in + c) - mean;
      q = __builtin_fmaf(d, d, q);
    }
    const float var = row_sum<kWideThreads>(make_float2(q, 0.0f), lds[1]).x * inv;
    const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (uint32_t c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float h = rank_sum<T>(a, in + c);
      const float w = !a.weight ? 1.0f : a.wf32 ? load_elem<kF32>(a.weight, c) : load_elem<T>(a.weight, c);
      const float b = !a.bias ? 0.0f : a.wf32 ? load_elem<kF32>(a.bias, c) : load_elem<T>(a.bias, c);
      if (a.sum) store_elem<T>(a.sum, out + c, h);
      store_elem<T>(a.out, out + c, __builtin_fmaf((h - mean) * rstd, w, b));
    }
  }
}

// A workgroup of BT lanes takes BT / TPR rows at a time, every gridDim-th such set; its
// lanes keep the weight and bias gradients of their columns in registers over all of
// them.  At the end the workgroup's rows are joined in LDS, in order, and written
// once: the sums over rows take a fixed order.
template <int T, int TPR, int E, int BT, bool AHEAD, bool NT> __global__ void __launch_bounds__(BT) norm_bwd_k(NormBwdArgs a) {
  constexpr int V = Vec<T>::VW, U = E / V, RPB = BT / TPR;
  __shared__ float2 lds[2][BT / 64];
  const uint32_t lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  float dw[E], db[E], w[E];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t c = (u * TPR + lane) * V;
    load_weights<T>(a.weight, a.wf32, c, unit_left(a.cols, c), 1.0f, w + u * V);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.0f;
  struct Row {
    u32x4 dy[U], h[U], res[U];
    float mean, rstd;
  };
  auto fetch = [&](uint64_t row0, Row& x) {
    const uint64_t row = row0 + sub;
    const bool live = row < a.rows;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = (u * TPR + lane) * V;
      const int n = live ? unit_left(a.cols, c) : 0;
      x.dy[u] = load_in<T, NT>(at<T>(a.dout, row * a.ld_in + c), n);
      x.h[u] = load_in<T, NT>(at<T>(a.sum, row * a.ld_in + c), n);
      if (a.dresidual && a.dsum) x.res[u] = load_in<T, NT>(at<T>(a.dresidual, row * a.ld_in + c), n);
    }
    x.mean = live ? a.mean[row] : 0.0f;
    x.rstd = live ? a.rstd[row] : 0.0f;
  };
  int flip = 0;
  const uint64_t step = (uint64_t)gridDim.x * RPB;
  Row now, next;
  if (AHEAD) fetch((uint64_t)blockIdx.x * RPB, next);
  for (uint64_t row0 = (uint64_t)blockIdx.x * RPB; row0 < a.rows; row0 += step, flip ^= 1) {
    const uint64_t row = row0 + sub;
    const bool live = row < a.rows;
    if (AHEAD) {
      now = next;
      if (row0 + step < a.rows) fetch(row0 + step, next);
    } else {
      fetch(row0, now);
    }
    const float mean = now.mean, rstd = now.rstd;
    float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int n = live ? unit_left(a.cols, (u * TPR + lane) * V) : 0;
      float dy[V], h[V];
      decode16<T>(now.dy[u], dy);
      decode16<T>(now.h[u], h);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (j < n) {
          const float xhat = (h[j] - mean) * rstd, g = dy[j] * w[u * V + j];
          s.x += g;
          s.y = __builtin_fmaf(g, xhat, s.y);
          dw[u * V + j] = __builtin_fmaf(dy[j], xhat, dw[u * V + j]);
          db[u * V + j] += dy[j];
        }
      }
    }
    if (!a.dsum) continue;
    s = row_sum<TPR>(s, lds[flip]);
    const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = (u * TPR + lane) * V;
      const int n = live ? unit_left(a.cols, c) : 0;
      float dy[V], h[V], d[V];
      decode16<T>(now.dy[u], dy);
      decode16<T>(now.h[u], h);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float xhat = (h[j] - mean) * rstd;
        d[j] = (dy[j] * w[u * V + j] - c1 - xhat * c2) * rstd;
      }
      if (a.dresidual) {
        decode16<T>(now.res[u], h);
#pragma unroll
        for (int j = 0; j < V; ++j) d[j] += h[j];
      }
      store_out<T, NT>(at<T>(a.dsum, row * a.ld_out + c), n, encode16<T>(d));
    }
  }
  if (!a.dweight && !a.dbias) return;
  if constexpr (RPB > 1) {
    __shared__ float sums[RPB / 2][2 * E][TPR];
#pragma unroll
    for (uint32_t half = RPB / 2; half > 0; half /= 2) {
      if (sub >= half && sub < 2 * half) {
#pragma unroll
        for (int e = 0; e < E; ++e) sums[sub - half][e][lane] = dw[e], sums[sub - half][E + e][lane] = db[e];
      }
      __syncthreads();
      if (sub < half) {
#pragma unroll
        for (int e = 0; e < E; ++e) dw[e] += sums[sub][e][lane], db[e] += sums[sub][E + e][lane];
      }
      __syncthreads();
    }
  }
  if (sub == 0) {
    float* p = a.partial + (uint64_t)blockIdx.x * 2 * a.cols;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = (u * TPR + lane) * V;
      const int n = unit_left(a.cols, c);
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        store_raw<kF32>(p + c + 4 * h, n - 4 * h, encode16<kF32>(dw + u * V + 4 * h));
        store_raw<kF32>(p + a.cols + c + 4 * h, n - 4 * h, encode16<kF32>(db + u * V + 4 * h));
      }
    }
  }
}

// Long rows: the gradient of h, one workgroup a row.
template <int T> __global__ void __launch_bounds__(kWideThreads) norm_bwd_wide_k(NormBwdArgs a) {
  __shared__ float2 lds[2][kWideThreads / 64];
  const float inv = 1.0f / (float)a.cols;
  int flip = 0;
  for (uint64_t row = blockIdx.x; row < a.rows; row += gridDim.x, flip ^= 1) {
    const uint64_t in = row * a.ld_in, out = row * a.ld_out;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float2 s = make_float2(0.0f, 0.0f);
    for (uint32_t c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float w = !a.weight ? 1.0f : a.wf32 ? load_elem<kF32>(a.weight, c) : load_elem<T>(a.weight, c);
      const float g = load_elem<T>(a.dout, in + c) * w;
      s.x += g;
      s.y = __builtin_fmaf(g, (load_elem<T>(a.sum, in + c) - mean) * rstd, s.y);
    }
    s = row_sum<kWideThreads>(s, lds[flip]);
    const float c1 = s.x * inv, c2 = s.y * inv;
    for (uint32_t c = threadIdx.x; c < a.cols; c += kWideThreads) {
      const float w = !a.weight ? 1.0f : a.wf32 ? load_elem<kF32>(a.weight, c) : load_elem<T>(a.weight, c);
      const float xhat = (load_elem<T>(a.sum, in + c) - mean) * rstd;
      float d = (load_elem<T>(a.dout, in + c) * w - c1 - xhat * c2) * rstd;
      if (a.dresidual) d += load_elem<T>(a.dresidual, in + c);
      store_elem<T>(a.dsum, out + c, d);
    }
  }
}

// Long rows: the weight gradients of row group blockIdx.y, a column a lane.
template <int T> __global__ void __launch_bounds__(256) norm_bwd_cols_k(NormBwdArgs a) {
  const uint32_t c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (uint64_t row = blockIdx.y; row < a.rows; row += a.groups) {
    const float dy = load_elem<T>(a.dout, row * a.ld_in + c);
    const float xhat = (load_elem<T>(a.sum, row * a.ld_in + c) - a.mean[row]) * a.rstd[row];
    dw = __builtin_fmaf(dy, xhat, dw);
    db += dy;
  }
  float* p = a.partial + (uint64_t)blockIdx.y * 2 * a.cols;
  p[c] = dw;
  p[a.cols + c] = db;
}

// dweight and dbias: the groups' sums joined in group order (16 strided chains,
// then those in order), rounded once.  64 columns a workgroup; blockIdx.y 0 is
// the weight, 1 the bias.
constexpr int kJoinCols = 64, kJoinChains = 16;

template <int T> __global__ void __launch_bounds__(kJoinCols * kJoinChains) norm_bwd_join_k(NormBwdArgs a) {
  __shared__ float lds[kJoinChains][kJoinCols];
  void* to = blockIdx.y ? a.dbias : a.dweight;
  if (!to) return;
  const uint32_t x = threadIdx.x % kJoinCols, chain = threadIdx.x / kJoinCols;
  const uint32_t c = blockIdx.x * kJoinCols + x;
  float s = 0.0f;
  if (c < a.cols) {
    const float* p = a.partial + (uint64_t)blockIdx.y * a.cols + c;
#pragma unroll 4
    for (uint32_t g = chain; g < a.groups; g += kJoinChains) s += p[(uint64_t)g * 2 * a.cols];
  }
  lds[chain][x] = s;
  __syncthreads();
  if (chain == 0 && c < a.cols) {
#pragma unroll
    for (int k = 1; k < kJoinChains; ++k) s += lds[k][x];
    if (a.wf32) store_elem<kF32>(to, c, s);
    else store_elem<T>(to, c, s);
  }
}

// Lanes a row and elements a lane: the fewest lanes that hold the row at 16
// elements each (8 for rows that one wave holds so), up to 1024 lanes.  0: the
// row does not fit; 32 elements a lane of 1024 would not leave registers enough.
struct RowShape {
  int tpr, e;
};
RowShape row_shape(uint32_t cols) {
  if (cols <= 512) return {64, 8};
  if (cols <= 1024) return {64, 16};
  if (cols <= 2048) return {128, 16};
  if (cols <= 4096) return {256, 16};
  if (cols <= 8192) return {512, 16};
  if (cols <= 16384) return {1024, 16};
  return {0, 0};
}

constexpr uint32_t kMaxGrid = 1u << 20;  // rows past it are walked in strides

// Calls that move more than the 256 MiB of the Infinity Cache store past the caches,
// and from 2 ranks on load past them: 16384 x 4096 bf16, 1 rank with residual, 103 us
// plain, 89 with such stores, 100 with both; 4096 x 8192, 4 ranks with residual, 97 /
// 90 / 87; 8192 x 4096, 8 ranks, 125 / 121 / 111.  Smaller calls may find their inputs
// in that cache (the gradient of 16384 x 1024: 38 us plain, 44 past it).
constexpr uint64_t kCacheBytes = 256ull << 20;

template <int T, int TPR, int E> hipError_t fwd(const NormFwdArgs& a, hipStream_t s) {
  constexpr uint64_t rpb = block_threads(TPR) / TPR;
  const uint64_t blocks = (a.rows + rpb - 1) / rpb;
  const dim3 grid((uint32_t)(blocks < kMaxGrid ? blocks : kMaxGrid)), block(block_threads(TPR));
  const uint64_t tensors = a.nranks + (a.residual ? 1 : 0) + (a.sum ? 1 : 0) + 1;
  const bool stream = a.rows * a.cols * Ty<T>::size * tensors > kCacheBytes;
  if (stream && a.nranks >= 2) hipLaunchKernelGGL((norm_fwd_k<T, TPR, E, true, true>), grid, block, 0, s, a);
  else if (stream) hipLaunchKernelGGL((norm_fwd_k<T, TPR, E, false, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_k<T, TPR, E, false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

template <int T> hipError_t fwd_typed(const NormFwdArgs& a, hipStream_t s) {
  const RowShape r = row_shape(a.cols);
  if (r.tpr == 64) return r.e == 8 ? fwd<T, 64, 8>(a, s) : fwd<T, 64, 16>(a, s);
  if (r.tpr == 128) return fwd<T, 128, 16>(a, s);
  if (r.tpr == 256) return fwd<T, 256, 16>(a, s);
  if (r.tpr == 512) return fwd<T, 512, 16>(a, s);
  if (r.tpr == 1024) return fwd<T, 1024, 16>(a, s);
  hipLaunchKernelGGL(norm_fwd_wide_k<T>, dim3((uint32_t)(a.rows < kMaxGrid ? a.rows : kMaxGrid)),
                     dim3(kWideThreads), 0, s, a);
  return hipGetLastError();
}

// Workgroup of norm_bwd_k: 1024 lanes, one a CU, which leaves 128 registers a lane and
// few parts to join (16384 x 4096 bf16 with residual: 99 us, 113 with 512 lanes).  Rows
// of 512 lanes would go two a workgroup, in step at each barrier: those take 512 lanes
// and load the next row ahead (8192 x 8192: 105 us with 1024 lanes, 100 with 512, 87
// loading ahead; 93 with two such a CU).  f32: 512 lanes, two a CU.
constexpr int bwd_threads(int t, int tpr) { return t == kF32 || tpr == 512 ? 512 : 1024; }
constexpr bool bwd_ahead(int t, int tpr) { return t != kF32 && tpr == 512; }
uint32_t bwd_blocks(uint64_t rows, uint32_t cols, int t) {
  const RowShape r = row_shape(cols);
  if (r.tpr == 0 || (t == kF32 && r.tpr > 512)) return rows < 256 ? (uint32_t)rows : 256;  // the kernels of long rows
  const uint32_t bt = bwd_threads(t, r.tpr), rpb = bt / r.tpr, most = t == kF32 ? 512 : 256;
  const uint64_t blocks = (rows + rpb - 1) / rpb;
  return blocks < most ? (uint32_t)blocks : most;
}

template <int T, int TPR, int E> void bwd(const NormBwdArgs& a, hipStream_t s) {
  constexpr int BT = bwd_threads(T, TPR);
  const uint64_t tensors = 2 + (a.dsum ? 1 : 0) + (a.dsum && a.dresidual ? 1 : 0);
  if (a.rows * a.cols * Ty<T>::size * tensors > kCacheBytes)
    hipLaunchKernelGGL((norm_bwd_k<T, TPR, E, BT, bwd_ahead(T, TPR), true>), dim3(a.groups), dim3(BT), 0, s, a);
  else hipLaunchKernelGGL((norm_bwd_k<T, TPR, E, BT, bwd_ahead(T, TPR), false>), dim3(a.groups), dim3(BT), 0, s, a);
}

template <int T> void bwd_1024(const NormBwdArgs& a, hipStream_t s) {
  if constexpr (T != kF32) bwd<T, 1024, 16>(a, s);
}

template <int T> hipError_t bwd_typed(const NormBwdArgs& a, hipStream_t s) {
  if (a.rows > 0) {
    const RowShape r = row_shape(a.cols);
    if (r.tpr == 64 && r.e == 8) bwd<T, 64, 8>(a, s);
    else if (r.tpr == 64) bwd<T, 64, 16>(a, s);
    else if (r.tpr == 128) bwd<T, 128, 16>(a, s);
    else if (r.tpr == 256) bwd<T, 256, 16>(a, s);
    else if (r.tpr == 512) bwd<T, 512, 16>(a, s);
    else if (r.tpr == 1024 && T != kF32) bwd_1024<T>(a, s);
    else {  // f32 rows of 1024 lanes as well: the raw data alone would take half of a lane's 128 registers
      // the column sums first: the gradient of h may take the place of what they read
      if (a.dweight || a.dbias)
        hipLaunchKernelGGL(norm_bwd_cols_k<T>, dim3((a.cols + 255) / 256, a.groups), dim3(256), 0, s, a);
      if (a.dsum)
        hipLaunchKernelGGL(norm_bwd_wide_k<T>, dim3((uint32_t)(a.rows < kMaxGrid ? a.rows : kMaxGrid)),
                           dim3(kWideThreads), 0, s, a);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.dweight || a.dbias) {
    hipLaunchKernelGGL(norm_bwd_join_k<T>, dim3((a.cols + kJoinCols - 1) / kJoinCols, 2),
                       dim3(kJoinCols * kJoinChains), 0, s, a);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace

// Parts that the weight gradients' sums take, whatever the type.
uint32_t norm_bwd_groups(uint64_t rows, uint32_t cols) {
  const uint32_t a = bwd_blocks(rows, cols, kF32), b = bwd_blocks(rows, cols, kBF16);
  return a > b ? a : b;
}

hipError_t launch_norm_fwd(const NormFwdArgs& a, int t, hipStream_t stream) {
  if (t == kF32) return fwd_typed<kF32>(a, stream);
  if (t == kF16) return fwd_typed<kF16>(a, stream);
  return fwd_typed<kBF16>(a, stream);
}

hipError_t launch_norm_bwd(NormBwdArgs a, int t, hipStream_t stream) {
  a.groups = bwd_blocks(a.rows, a.cols, t);
  if (t == kF32) return bwd_typed<kF32>(a, stream);
  if (t == kF16) return bwd_typed<kF16>(a, stream);
  return bwd_typed<kBF16>(a, stream);
}

}  // namespace mrr
