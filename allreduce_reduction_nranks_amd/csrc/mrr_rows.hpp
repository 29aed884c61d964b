// mrr_rows.hpp -- 16-byte access to rows that need no alignment beyond their
// element's: gfx950 loads and stores 16 bytes at any address, and only a row's
// last, partial unit goes element by element.
#pragma once

#include "mrr_device.hpp"

namespace mrr {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// V elements from `p` on, of which the first `n` exist; zeros after them.
template <int T> __device__ __forceinline__ u32x4 load_raw(const void* p, int n) {
  constexpr int V = Vec<T>::VW;
  if (n >= V) return *reinterpret_cast<const u32x4_any*>(p);
  u32x4 v = {0u, 0u, 0u, 0u};
  if constexpr (T == kF32) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) v[j] = reinterpret_cast<const uint32_t*>(p)[j];
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) v[j / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j] << (16 * (j & 1));
  }
  return v;
}

// V elements from column c on of a row of `cols`; zeros after its last.  One load, of the
// row's last V where it ends before c + V.
template <int T> __device__ __forceinline__ u32x4 load_cols(const uint8_t* row, uint32_t c, uint32_t cols) {
  constexpr uint32_t V = Vec<T>::VW, size = Ty<T>::size;
  if (cols < V) return load_raw<T>(row + (uint64_t)c * size, c < cols ? (int)(cols - c) : 0);
  const uint32_t at = c < cols - V ? c : cols - V, over = c - at;
  u32x4 v = *reinterpret_cast<const u32x4_any*>(row + (uint64_t)at * size);
  if (over) {
    const uint32_t bits = over * size * 8;
    uint64_t lo = (uint64_t)v.y << 32 | v.x, hi = (uint64_t)v.w << 32 | v.z;
    if (bits < 64) lo = lo >> bits | hi << (64 - bits), hi >>= bits;
    else lo = bits < 128 ? hi >> (bits - 64) : 0, hi = 0;
    v = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
  }
  return v;
}

template <int T> __device__ __forceinline__ void store_raw(void* p, int n, u32x4 v) {
  constexpr int V = Vec<T>::VW;
  if (n >= V) {
    *reinterpret_cast<u32x4_any*>(p) = v;
    return;
  }
  if constexpr (T == kF32) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) reinterpret_cast<uint32_t*>(p)[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (j < n) reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
  }
}

template <int T> __device__ __forceinline__ const uint8_t* at(const void* p, uint64_t i) {
  return reinterpret_cast<const uint8_t*>(p) + i * Ty<T>::size;
}
template <int T> __device__ __forceinline__ uint8_t* at(void* p, uint64_t i) {
  return reinterpret_cast<uint8_t*>(p) + i * Ty<T>::size;
}

// Four values, of which the first `n` are stored, rounded to T.
typedef u32x2 u32x2_any __attribute__((aligned(2)));
template <int T> __device__ __forceinline__ void store4(void* p, int n, const float* x) {
  if constexpr (T == kF32) {
    store_raw<kF32>(p, n, encode16<kF32>(x));
  } else if (n >= 4) {
    *reinterpret_cast<u32x2_any*>(p) = u32x2{from_f32<T>(x[0]) | from_f32<T>(x[1]) << 16,
                                             from_f32<T>(x[2]) | from_f32<T>(x[3]) << 16};
  } else {
#pragma unroll
    for (int j = 0; j < 3; ++j)
      if (j < n) reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)from_f32<T>(x[j]);
  }
}

}  // namespace mrr
