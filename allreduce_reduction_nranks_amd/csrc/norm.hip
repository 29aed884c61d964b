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
// tensor.  A row of 8 to 16384 columns (f32 gradients: 8192) is held in the registers of
// TPR lanes, E elements a lane, so every tensor is read once; longer and shorter rows are
// read again for each pass, element by element.  The variance is the mean of squared
// differences from the finished mean, which loses nothing when the mean is large.  Statistics,
// sums and the weight gradients are f32 throughout; the stored h and y are
// rounded once each, and y is the norm of the stored (rounded) h, so that the
// gradient, which reads h, is that of the same function.
//
// A lane's elements come in units of 16 bytes, unit u of a lane being unit
// u * TPR + lane of the row: a wave's loads are contiguous.  Rows need no
// alignment beyond their element's: gfx950 loads 16 bytes from any address.  Where
// the row ends inside a unit, the unit is moved back to end with the row.  Its first
// `over` elements are then the neighbour's too: they are left out of sums along the row,
// and both lanes store the same value.  No access of theirs goes element by element, which keeps
// the code a third of its size: a call of few rows runs it once, out of a cold cache.
#include <type_traits>

#include "mrr_device.hpp"
#include "mrr_internal.hpp"
#include "mrr_ops.hpp"
#include "mrr_rows.hpp"

namespace mrr {
namespace {

// The unit of a row of `cols` elements (a unit's worth at least) that begins at column c.
template <int T> struct Unit {
  uint32_t at, over;
  __device__ __forceinline__ Unit(uint32_t cols, uint32_t c) {
    at = c < cols - Vec<T>::VW ? c : cols - Vec<T>::VW;
    over = c - at;
  }
  __device__ __forceinline__ bool any() const { return over < (uint32_t)Vec<T>::VW; }
};

// 16 bytes, past the caches (NT) or through them.
template <bool NT> __device__ __forceinline__ u32x4 load_unit(const void* p) {
  if (NT) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
  return *reinterpret_cast<const u32x4_any*>(p);
}
template <bool NT> __device__ __forceinline__ void store_unit(void* p, u32x4 v) {
  if (NT) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  else *reinterpret_cast<u32x4_any*>(p) = v;
}

// V weights from column `at` on as they lie in memory, and widened; `fill` where there
// are none.
template <int T> struct RawWeights {
  static constexpr int N = T == kF32 ? 1 : 2;  // f32 weights beside 16-bit data take two loads
  u32x4 v[N];
  __device__ __forceinline__ void load(const void* w, int wf32, uint32_t c) {
    if (!w) return;
    if (T == kF32 || wf32) {
#pragma unroll
      for (int h = 0; h < N; ++h) v[h] = load_unit<false>(at<kF32>(w, c + 4 * h));
    } else {
      v[0] = load_unit<false>(at<T>(w, c));
    }
  }
  __device__ __forceinline__ void get(const void* w, int wf32, float fill, float* x) const {
    if (!w) {
#pragma unroll
      for (int j = 0; j < Vec<T>::VW; ++j) x[j] = fill;
    } else if (T == kF32 || wf32) {
#pragma unroll
      for (int h = 0; h < N; ++h) decode16<kF32>(v[h], x + 4 * h);
    } else {
      decode16<T>(v[0], x);
    }
  }
};

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

// ONE: the workgroup has one set of rows, and all it reads is asked for at once (1 x 4096,
// 8 ranks: 5.6 us a call in a graph, of which 4.5 are a call of any size).  TAIL:
// rows may end inside a unit; without it, a unit is whole or not there.  4096 x 8192 bf16
// of 4 ranks with residual: 83 us, 5.7 TB/s of the 6.6 that a copy reaches.
template <int T, int TPR, int E, bool NTL, bool NTS, bool ONE, bool TAIL>
__global__ void __launch_bounds__(block_threads(TPR)) norm_fwd_k(NormFwdArgs a) {
  constexpr int V = Vec<T>::VW, U = E / V, RPB = block_threads(TPR) / TPR;
  // ranks whose loads are in flight together
  constexpr int G = ONE ? (U >= 4 ? 4 : 8) : U >= 4 || TPR == 1024 ? 2 : 4;
  __shared__ float2 lds[2][block_threads(TPR) / 64];
  const uint32_t lane = threadIdx.x % TPR;
  const uint32_t sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  // every lane of a workgroup walks the same number of rows, as they share barriers
  for (uint64_t row0 = (uint64_t)blockIdx.x * RPB; row0 < a.rows; row0 += (uint64_t)gridDim.x * RPB) {
    const bool live = row0 + sub < a.rows;
    const uint64_t row = live ? row0 + sub : a.rows - 1;  // a lane without a row reads the last one
    float x[E];
    u32x4 raw[G + (ONE ? 1 : 0)][U];  // ONE: the residual has a place of its own
    u32x4(&res)[U] = raw[ONE ? G : 0];
    RawWeights<T> w[U], b[U];
    auto load_residual = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) res[u] = load_unit<NTL>(at<T>(a.residual, row * a.ld_in + Unit<T>(a.cols, (u * TPR + lane) * V).at));
    };
    auto load_weights = [&](int u) {
      const uint32_t c = Unit<T>(a.cols, (u * TPR + lane) * V).at;
      w[u].load(a.weight, a.wf32, c);
      b[u].load(a.bias, a.wf32, c);
    };
    if constexpr (ONE) {
      if (a.residual) load_residual();
#pragma unroll
      for (int u = 0; u < U; ++u) load_weights(u);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = -0.0f;  // (the first sum is then exactly x_0)
    for (int r0 = 0; r0 < a.nranks; r0 += G) {
#pragma unroll
      for (int g = 0; g < G; ++g) {
        if (r0 + g < a.nranks) {
#pragma unroll
          for (int u = 0; u < U; ++u)
            raw[g][u] = load_unit<NTL>(at<T>(a.in[r0 + g], row * a.ld_in + Unit<T>(a.cols, (u * TPR + lane) * V).at));
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
            for (int j = 0; j < V; ++j) x[u * V + j] += d[j];
          }
        }
      }
    }
    if (a.residual) {
      if constexpr (!ONE) load_residual();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float d[V];
        decode16<T>(res[u], d);
#pragma unroll
        for (int j = 0; j < V; ++j) x[u * V + j] += d[j];
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      decode16<T>(encode16<T>(x + u * V), x + u * V);
      const uint32_t over = Unit<T>(a.cols, (u * TPR + lane) * V).over;
      float su = 0.0f;
      if (over == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) su += x[u * V + j];
      } else if (TAIL) {
#pragma unroll
        for (int j = 0; j < V; ++j) su += (uint32_t)j >= over ? x[u * V + j] : 0.0f;
      }
      s += su;
    }
    auto store_sum = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const Unit<T> unit(a.cols, (u * TPR + lane) * V);
        if (live && unit.any()) store_unit<NTS>(at<T>(a.sum, row * a.ld_out + unit.at), encode16<T>(x + u * V));
      }
    };
    // in an input's place, when every wave has read its units (else early: f32 rows of
    // 1024 lanes are 5 % faster)
    if (a.sum && !a.in_place) store_sum();
    const float mean = row_sum<TPR>(make_float2(s, 0.0f), lds[0]).x * inv;
    if (a.sum && a.in_place) store_sum();
    float q = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit<T> unit(a.cols, (u * TPR + lane) * V);
      float qu = 0.0f;
#pragma unroll
      for (int j = 0; j < V; ++j) x[u * V + j] -= mean;
      if (unit.over == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) qu = __builtin_fmaf(x[u * V + j], x[u * V + j], qu);
      } else if (TAIL) {
#pragma unroll
        for (int j = 0; j < V; ++j) qu = __builtin_fmaf(x[u * V + j], (uint32_t)j >= unit.over ? x[u * V + j] : 0.0f, qu);
      }
      q += qu;
    }
    const float var = row_sum<TPR>(make_float2(q, 0.0f), lds[1]).x * inv;
    const float rstd = 1.0f / __builtin_sqrtf(var + a.eps);
    if (live && lane == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit<T> unit(a.cols, (u * TPR + lane) * V);
      float wx[V], y[V];
      if constexpr (!ONE) load_weights(u);
      w[u].get(a.weight, a.wf32, 1.0f, wx);
      b[u].get(a.bias, a.wf32, 0.0f, y);
#pragma unroll
      for (int j = 0; j < V; ++j) y[j] = __builtin_fmaf(x[u * V + j] * rstd, wx[j], y[j]);
      if (live && unit.any()) store_unit<NTS>(at<T>(a.out, row * a.ld_out + unit.at), encode16<T>(y));
    }
  }
}

// Rows too long for registers (or shorter than a unit): the same three passes with the sum computed
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
// once: the sums over rows take a fixed order.  16384 x 4096 bf16 with residual: 91 us,
// 5.9 TB/s, and 4.6 for the join of the 256 workgroups' sums.
//
// DX: the gradient of h is wanted.  What is in flight at the end of a turn is known to
// the compiler (a branch around some of the stores would make it wait for all of them
// before the next turn's loads: 4 %, and 14 % of a call that loads ahead).
template <int T, int TPR, int E, int BT, bool AHEAD, bool NT, bool TAIL, bool DX>
__global__ void __launch_bounds__(BT) norm_bwd_k(NormBwdArgs a) {
  constexpr int V = Vec<T>::VW, U = E / V, RPB = BT / TPR;
  __shared__ float2 lds[2][BT / 64];
  const uint32_t lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)a.cols;
  float dw[E], db[E], w[E];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    RawWeights<T> raw;
    raw.load(a.weight, a.wf32, Unit<T>(a.cols, (u * TPR + lane) * V).at);
    raw.get(a.weight, a.wf32, 1.0f, w + u * V);
  }
#pragma unroll
  for (int e = 0; e < E; ++e) dw[e] = db[e] = 0.0f;
  struct Row {
    u32x4 dy[U], h[U], res[U];
    float mean, rstd;
  };
  auto fetch = [&](uint64_t row0, Row& x) {
    const uint64_t row = row0 + sub < a.rows ? row0 + sub : a.rows - 1;
    const uint64_t from = row * a.ld_in;
    x.mean = a.mean[row];
    x.rstd = a.rstd[row];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t c = Unit<T>(a.cols, (u * TPR + lane) * V).at;
      x.dy[u] = load_unit<NT>(at<T>(a.dout, from + c));
      x.h[u] = load_unit<NT>(at<T>(a.sum, from + c));
    }
    if (DX && a.dresidual) {
#pragma unroll
      for (int u = 0; u < U; ++u) x.res[u] = load_unit<NT>(at<T>(a.dresidual, from + Unit<T>(a.cols, (u * TPR + lane) * V).at));
    }
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
    if (live) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t over = Unit<T>(a.cols, (u * TPR + lane) * V).over;
        if (over >= (TAIL ? (uint32_t)V : 1u)) continue;
        float dy[V], h[V];
        decode16<T>(now.dy[u], dy);
        decode16<T>(now.h[u], h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float xhat = (h[j] - mean) * rstd;
          const float g = !TAIL || (uint32_t)j >= over ? dy[j] * w[u * V + j] : 0.0f;
          s.x += g;
          s.y = __builtin_fmaf(g, xhat, s.y);
          dw[u * V + j] = __builtin_fmaf(dy[j], xhat, dw[u * V + j]);
          db[u * V + j] += dy[j];
        }
      }
    }
    if (!DX) continue;
    // Elements that two lanes store are read by both before either stores: dsum may lie in
    // the place of any of the three, so they have arrived (are used) by the barrier.
    if constexpr (AHEAD || TAIL) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        asm volatile("" ::"v"(now.dy[u]), "v"(now.h[u]));
        if (a.dresidual) asm volatile("" ::"v"(now.res[u]));
      }
    }
    s = row_sum<TPR>(s, lds[flip]);
    const float c1 = s.x * inv, c2 = s.y * inv;
    if (!AHEAD) __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the loads of this turn
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Unit<T> unit(a.cols, (u * TPR + lane) * V);
      // (loading ahead, lanes past the row's end have its last unit and store it again)
      if (!AHEAD && (!live || !unit.any())) continue;
      float dy[V], h[V], d[V];
      // widened again: kept from above, the values would take twice the registers
      if (TAIL || TPR == 1024) asm volatile("" : "+v"(now.dy[u]), "+v"(now.h[u]));
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
      store_unit<NT>(at<T>(a.dsum, row * a.ld_out + unit.at), encode16<T>(d));
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
      const Unit<T> unit(a.cols, (u * TPR + lane) * V);
      if (!unit.any()) continue;
#pragma unroll
      for (int h = 0; h < V / 4; ++h) {
        store_unit<false>(p + unit.at + 4 * h, encode16<kF32>(dw + u * V + 4 * h));
        store_unit<false>(p + a.cols + unit.at + 4 * h, encode16<kF32>(db + u * V + 4 * h));
      }
    }
  }
}

// Both gradients of few rows in one launch: the first `row_blocks` workgroups take rows
// as above, without sums over them; the others take 16 V columns each and read all rows
// again, 64 at a time, so that nothing has to be joined in another launch.  (Where dsum
// lies in the place of what they read, they go first, in a launch of their own.)
// One launch against two: 8 x 16384 bf16 5.2 us against 9.3 in a graph, 513 x 1600 f32 5.7
// against 9.4; at its border (below, 4 MiB a tensor and 1024 rows) 10 against 10 to 12.
constexpr int kSmallThreads = 1024, kSmallLanes = 16, kSmallRows = kSmallThreads / kSmallLanes;

template <int T, int TPR, int E>
__device__ __forceinline__ void small_rows(const NormBwdArgs& a, float2 (*lds)[kSmallThreads / 64]) {
  constexpr int V = Vec<T>::VW, U = E / V, RPB = kSmallThreads / TPR;
  const uint32_t lane = threadIdx.x % TPR;
  const uint64_t mine = (uint64_t)blockIdx.x * RPB + threadIdx.x / TPR, row = mine < a.rows ? mine : a.rows - 1;
  const float inv = 1.0f / (float)a.cols;
  u32x4 rdy[U], rh[U], res[U];
  RawWeights<T> rw[U];
  const float mean = a.mean[row], rstd = a.rstd[row];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Unit<T> unit(a.cols, (u * TPR + lane) * V);
    rdy[u] = load_unit<false>(at<T>(a.dout, row * a.ld_in + unit.at));
    rh[u] = load_unit<false>(at<T>(a.sum, row * a.ld_in + unit.at));
    rw[u].load(a.weight, a.wf32, unit.at);
    if (a.dresidual) res[u] = load_unit<false>(at<T>(a.dresidual, row * a.ld_in + unit.at));
  }
  float g[E], xhat[E];
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t over = Unit<T>(a.cols, (u * TPR + lane) * V).over;
    float w[V];
    rw[u].get(a.weight, a.wf32, 1.0f, w);
    decode16<T>(rdy[u], g + u * V);
    decode16<T>(rh[u], xhat + u * V);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = u * V + j;
      xhat[e] = (xhat[e] - mean) * rstd;
      g[e] *= w[j];
      if ((uint32_t)j >= over) s.x += g[e], s.y = __builtin_fmaf(g[e], xhat[e], s.y);
    }
  }
  // as above: what two lanes store has been read by both
  if (a.dresidual) {
#pragma unroll
    for (int u = 0; u < U; ++u) asm volatile("" ::"v"(res[u]));
  }
  s = row_sum<TPR>(s, lds[0]);
  if (mine >= a.rows) return;
  const float c1 = s.x * inv, c2 = s.y * inv;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const Unit<T> unit(a.cols, (u * TPR + lane) * V);
    float d[V];
#pragma unroll
    for (int j = 0; j < V; ++j) d[j] = (g[u * V + j] - c1 - xhat[u * V + j] * c2) * rstd;
    if (a.dresidual) {
      float r[V];
      decode16<T>(res[u], r);
#pragma unroll
      for (int j = 0; j < V; ++j) d[j] += r[j];
    }
    if (unit.any()) store_unit<false>(at<T>(a.dsum, row * a.ld_out + unit.at), encode16<T>(d));
  }
}

template <int T, int TPR, int E> __global__ void __launch_bounds__(kSmallThreads) norm_bwd_small_k(NormBwdArgs a, uint32_t row_blocks) {
  constexpr int V = Vec<T>::VW, kWaves = kSmallThreads / 64;
  __shared__ union {
    float2 rows[1][kWaves];
    float cols[kWaves][2 * V][kSmallLanes];
  } lds;
  if (blockIdx.x < row_blocks) return small_rows<T, TPR, E>(a, lds.rows);
  const uint32_t x = threadIdx.x % kSmallLanes, wave = threadIdx.x >> 6;
  const Unit<T> unit(a.cols, ((blockIdx.x - row_blocks) * kSmallLanes + x) * V);
  float dw[V], db[V];
#pragma unroll
  for (int j = 0; j < V; ++j) dw[j] = db[j] = 0.0f;
#pragma unroll 4
  for (uint32_t row = threadIdx.x / kSmallLanes; row < (uint32_t)a.rows; row += kSmallRows) {
    float dy[V], h[V];
    const float mean = a.mean[row], rstd = a.rstd[row];
    decode16<T>(load_unit<false>(at<T>(a.dout, row * a.ld_in + unit.at)), dy);
    decode16<T>(load_unit<false>(at<T>(a.sum, row * a.ld_in + unit.at)), h);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dw[j] = __builtin_fmaf(dy[j], (h[j] - mean) * rstd, dw[j]);
      db[j] += dy[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
#pragma unroll
    for (int m = kSmallLanes; m < 64; m *= 2) {
      dw[j] += __shfl_xor(dw[j], m);
      db[j] += __shfl_xor(db[j], m);
    }
    if ((threadIdx.x & 63) < kSmallLanes) lds.cols[wave][j][x] = dw[j], lds.cols[wave][V + j][x] = db[j];
  }
  __syncthreads();
  const uint32_t j = threadIdx.x / kSmallLanes, col = unit.at + j % V;
  if (j >= 2 * V || !unit.any()) return;
  float s = 0.0f;
#pragma unroll
  for (int k = 0; k < kWaves; ++k) s += lds.cols[k][j][x];
  void* to = j < V ? a.dweight : a.dbias;
  if (!to) return;
  if (a.wf32) store_elem<kF32>(to, col, s);
  else store_elem<T>(to, col, s);
}

// Such rows: the gradient of h, one workgroup a row.  dout and the sum are read three times
// with the column sums below: 4096 x 12288 f32 249 us, 2.4 TB/s of what has to move, and 8 x
// 12288 14.5 us (4096 x 8192, in registers: 86 us, 4.7 TB/s).
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

// Such rows: the weight gradients of row group blockIdx.y, a column a lane.
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
// elements each (8 for rows that one wave holds so), up to 1024 lanes.  (4096 x 8192 bf16
// of 4 ranks: 83 us; at 8 elements a lane, with more waves but longer joins, 98; at 32, 91.
// 16384 x 2048 f16 of 2 ranks: 59, 61, 72.)  0: the row does not fit; 32 elements a lane of
// 1024 would not leave registers enough.  Nor does one that is shorter than a unit.  Rows of
// less than a wave's 512 elements leave lanes idle: 131072 x 256 bf16 67 us forward and 55 for
// the gradient, 262144 x 128 122 and 90 (1.1 and 2.3 TB/s).
struct RowShape {
  int tpr, e;
};
RowShape row_shape(uint32_t cols) {
  if (cols < 8) return {0, 0};
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
  auto go = [&](auto ntl, auto nts, auto one, auto tail) {
    hipLaunchKernelGGL((norm_fwd_k<T, TPR, E, ntl, nts, one, tail>), grid, block, 0, s, a);
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  const bool tail = a.cols % Vec<T>::VW != 0;
  if (TPR < 1024 && blocks <= 256 && !stream) go(no, no, std::bool_constant<(TPR < 1024)>(), yes);
  else if (stream && a.nranks >= 2) tail ? go(yes, yes, no, yes) : go(yes, yes, no, no);
  else if (stream) tail ? go(no, yes, no, yes) : go(no, yes, no, no);
  else tail ? go(no, no, no, yes) : go(no, no, no, no);
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
  if (r.tpr == 0 || (t == kF32 && r.tpr > 512)) return rows < 256 ? (uint32_t)rows : 256;  // the kernels of such rows
  const uint32_t bt = bwd_threads(t, r.tpr), rpb = bt / r.tpr, most = t == kF32 ? 512 : 256;
  const uint64_t blocks = (rows + rpb - 1) / rpb;
  return blocks < most ? (uint32_t)blocks : most;
}

// Whether norm_bwd_small_k takes the call.
template <int T> bool bwd_small(const NormBwdArgs& a) {
  return (a.dweight || a.dbias) && a.rows <= 1024 && a.rows * a.cols * Ty<T>::size <= (4u << 20);
}

// True: the weight gradients' parts are left to join.
template <int T, int TPR, int E> bool bwd(const NormBwdArgs& a, hipStream_t s) {
  if (bwd_small<T>(a)) {
    constexpr uint32_t rpb = kSmallThreads / TPR, cpb = kSmallLanes * Vec<T>::VW;
    const uint32_t rows = a.dsum ? (uint32_t)(a.rows + rpb - 1) / rpb : 0u;
    const uint32_t cols = (a.cols + cpb - 1) / cpb;
    if (a.dsum == a.dout || a.dsum == a.sum) {
      hipLaunchKernelGGL((norm_bwd_small_k<T, TPR, E>), dim3(cols), dim3(kSmallThreads), 0, s, a, 0u);
      hipLaunchKernelGGL((norm_bwd_small_k<T, TPR, E>), dim3(rows), dim3(kSmallThreads), 0, s, a, rows);
    } else {
      hipLaunchKernelGGL((norm_bwd_small_k<T, TPR, E>), dim3(rows + cols), dim3(kSmallThreads), 0, s, a, rows);
    }
    return false;
  }
  constexpr int BT = bwd_threads(T, TPR);
  const uint64_t tensors = 2 + (a.dsum ? 1 : 0) + (a.dsum && a.dresidual ? 1 : 0);
  auto go = [&](auto ahead, auto nt, auto tail, auto dx) {
    hipLaunchKernelGGL((norm_bwd_k<T, TPR, E, BT, ahead, nt, tail, dx>), dim3(a.groups), dim3(BT), 0, s, a);
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  constexpr std::bool_constant<bwd_ahead(T, TPR)> ahead;
  const bool tail = a.cols % Vec<T>::VW != 0;
  if (!a.dsum) go(no, no, yes, no);
  else if (a.rows * a.cols * Ty<T>::size * tensors > kCacheBytes) tail ? go(ahead, yes, yes, yes) : go(ahead, yes, no, yes);
  else tail ? go(ahead, no, yes, yes) : go(ahead, no, no, yes);
  return a.dweight || a.dbias;
}

template <int T> bool bwd_1024(const NormBwdArgs& a, hipStream_t s) {
  if constexpr (T != kF32) return bwd<T, 1024, 16>(a, s);
  return false;
}

template <int T> hipError_t bwd_typed(const NormBwdArgs& a, hipStream_t s) {
  bool join = a.dweight || a.dbias;
  if (a.rows > 0) {
    const RowShape r = row_shape(a.cols);
    if (r.tpr == 64 && r.e == 8) join = bwd<T, 64, 8>(a, s);
    else if (r.tpr == 64) join = bwd<T, 64, 16>(a, s);
    else if (r.tpr == 128) join = bwd<T, 128, 16>(a, s);
    else if (r.tpr == 256) join = bwd<T, 256, 16>(a, s);
    else if (r.tpr == 512) join = bwd<T, 512, 16>(a, s);
    else if (r.tpr == 1024 && T != kF32) join = bwd_1024<T>(a, s);
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
  if (join) {
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
