// mrr_gemm.hpp -- the tile product that the cross entropy kernels share: one workgroup
// computes D[m][n] = sum over k of A[m][k] B[n][k] for a tile of S m by S n in f32, from
// 16-bit operands, and hands each wave its part.
//
// An operand lies in memory either with k contiguous ("row": a row for each m)
// or with m contiguous ("col": a row for each k).  Both reach LDS by loads that
// bypass registers (16 bytes a lane, a wave's 1 KiB contiguous in LDS), 64 k a
// stage, two stages.  A row operand is read from LDS 16 bytes a lane; a col
// operand with the transposing 64-bit read, so no operand is transposed in
// memory.  Chunks are permuted within a stage (the permutation is made on the
// global address, since the LDS side of the load is fixed) so that the lanes
// that LDS serves together touch different banks.
//
// Two sizes of tile, S x S.  256: 8 waves, 2 a SIMD, each with 128 x 64 accumulators;
// a stage's products take 2048 cycles of a CU's matrix units against 1536 of LDS reads.
// 128: 4 waves with 64 x 64 each, two workgroups a CU; as many cycles of LDS reads as of
// products, but four times the workgroups, for calls with too few large tiles.  Matrix
// instructions are 32x32x16.  The fragments of the
// next 16 k are read while those of the present ones multiply, over the end of a
// stage as well: the one barrier of a stage stands before its last quarter, when
// all its reads are done, so that the stage's buffer can be refilled and the next
// stage's first fragments fetched under that quarter's products.
#pragma once

#include <type_traits>

#include "mrr_rows.hpp"

namespace mrr {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));

constexpr int kTileV = 256;  // vocabulary shards are padded to multiples of this
constexpr int kTileK = 64;
constexpr int tile_threads(int s) { return s == 256 ? 512 : 256; }

template <int T> __device__ __forceinline__ f32x16 mfma(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (T == kF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Lane l of a wave's accumulator tile: n is l % 32, element i's m is this.
__device__ __forceinline__ int acc_row(int lane, int i) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// ---- addresses -----------------------------------------------------------------
// Row operand: a stage is [S rows][64 k], 128 bytes a row in chunks of 16.  Load i of
// thread t brings row i threads / 8 + t / 8; chunk c of row r lies at position c ^ f(r),
// f(r) = (r & 7) ^ (r >> 3 & 1): any 8 rows, and any 16 over 64 banks, differ.
template <int S> __device__ __forceinline__ uint32_t row_src_row(int tid, int i) {
  return (uint32_t)(i * (tile_threads(S) / 8) + (tid >> 3));
}
__device__ __forceinline__ uint32_t row_src_chunk(int tid) {
  return (uint32_t)((tid & 7) ^ ((tid >> 3) & 7) ^ ((tid >> 6) & 1));
}
// Byte offset of lane's 8 k of quarter 0 in the row tile that starts at `row0`
// (a multiple of 32); quarter kk is at offset ^ (kk * 32).
__device__ __forceinline__ uint32_t row_frag(int row0, int lane) {
  const int r = lane & 31;
  return (uint32_t)((row0 + r) * 128 + (((lane >> 5) ^ (r & 7) ^ ((r >> 3) & 1)) << 4));
}
// Col operand: a stage is [64 k][S m], 2 S bytes a k.  Load i of thread t brings k
// i threads 8 / S + t 8 / S; 64-byte units are at unit ^ (k modulo their count).
template <int S> __device__ __forceinline__ uint32_t col_src_k(int tid, int i) {
  return (uint32_t)(i * (tile_threads(S) / (S / 8)) + tid / (S / 8));
}
template <int S> __device__ __forceinline__ uint32_t col_src_chunk(int tid) {
  return (uint32_t)((tid % (S / 8)) ^ ((tid / (S / 8) % (S / 32)) << 2));
}
// A transposing read serves 16 lanes with a block of 4 k x 16 m: lane j of the
// 16 addresses k j / 4, m 4 (j % 4), and receives the 4 k of m j.  Byte offset
// for the 32 m from m0 on, k 0..3 (+ 4 for r = 1) and 8..11.
template <int S> __device__ __forceinline__ uint32_t col_frag(int m0, int r, int lane) {
  const int k = 8 * (lane >> 5) + 4 * r + ((lane >> 2) & 3);
  const int unit = (m0 >> 5) ^ (k % (S / 32));
  return (uint32_t)(k * (2 * S) + unit * 64 + 32 * ((lane >> 4) & 1) + 8 * (lane & 3));
}

typedef __attribute__((address_space(3))) uint8_t lds8;
typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;

__device__ __forceinline__ u32x4 read_row(const lds8* p) { return *(const lds_u32x4*)p; }
__device__ __forceinline__ u32x4 read_col(const lds8* lo, const lds8* hi) {
  const u32x2 a = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)lo));
  const u32x2 b = __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)hi));
  return u32x4{a.x, a.y, b.x, b.y};
}

// 16 bytes a lane from base + off to LDS, lane l's at lds + 16 l.  In assembly
// because the compiler, given the builtin, waits for the loads in flight before it
// reads the other stage's buffer; there is no output register, and run() below
// waits for them.  The LDS address goes in m0, as an operand that the compiler sets; the
// wait state between the two is the statement's own.
__device__ __forceinline__ void load_lds(const uint8_t* base, uint32_t off, lds8* lds) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :: "{m0}"((uint32_t)(uintptr_t)lds), "v"(off), "s"(base));
}

// The product over `steps` stages of 64 k, NS of them in LDS.  src(s, pa, pb, oa, ob) sets
// the (wave-uniform) addresses and the lane offsets of stage s; it is called once for
// each s in order.
template <int T, bool ACOL, bool BCOL, int S, int NS> struct Tile {
  static constexpr int WN = S == 256 ? 4 : 2, WM = 2;        // waves along n and m
  static constexpr int FM = S / WM / 32, FN = S / WN / 32;   // 32 x 32 tiles of a wave
  static constexpr int kStage = S * kTileK * 2;                 // bytes of an operand's stage
  static constexpr int kLoad = tile_threads(S) * 16, L = kStage / kLoad;  // bytes of a load, loads of a lane
  static constexpr int kLds = 2 * NS * kStage;               // A's stages, then B's
  static constexpr int Q = kTileK / 16;                      // quarters of a stage, which multiply together
  f32x16 acc[FM][FN];

  template <class Src> __device__ __forceinline__ void run(int steps, lds8* lds, Src&& src) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m0 = wave / WN * (FM * 32), n0 = wave % WN * (FN * 32);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    if (steps <= 0) return;
    // offsets of this lane's fragments in the present stage, and of its wave's loads in
    // the one that is filled next
    constexpr int NA = ACOL ? 2 * FM : Q, NB = BCOL ? 2 * FN : Q;
    uint32_t fa[NA], fb[NB];
    uint32_t at = 0, fill = 0;
#pragma unroll
    for (int i = 0; i < NA; ++i) fa[i] = ACOL ? col_frag<S>(m0 + 32 * (i >> 1), i & 1, lane) : row_frag(m0, lane) ^ (i * 32);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      fb[i] = NS * kStage + (BCOL ? col_frag<S>(n0 + 32 * (i >> 1), i & 1, lane) : row_frag(n0, lane) ^ (i * 32));
    lds8* const wave_lds = lds + wave * 1024;
    const uint8_t *pa, *pb;
    uint32_t oa[L], ob[L];
    u32x4 va[2][FM], vb[2][FN];

    auto fetch = [&](int i) {
      if (i < L) load_lds(pa, oa[i % L], wave_lds + fill + i * kLoad);
      else load_lds(pb, ob[i % L], wave_lds + fill + NS * kStage + (i - L) * kLoad);
    };
    auto filled = [&]() { fill = fill == (NS - 1) * kStage ? 0 : fill + kStage; };
    auto read = [&](int f, int kk) {
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (BCOL) vb[f][j] = read_col(lds + fb[2 * j] + kk * (32 * S), lds + fb[2 * j + 1] + kk * (32 * S));
        else vb[f][j] = read_row(lds + fb[kk] + j * 4096);
      }
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (ACOL) va[f][i] = read_col(lds + fa[2 * i] + kk * (32 * S), lds + fa[2 * i + 1] + kk * (32 * S));
        else va[f][i] = read_row(lds + fa[kk] + i * 4096);
      }
    };
    auto product = [&](int f, int p) {
      acc[p / FN][p % FN] = mfma<T>(va[f][p / FN], vb[f][p % FN], acc[p / FN][p % FN]);
    };
    constexpr int kProducts = FM * FN;
    // fragments f multiply while the others are read from quarter kk
    auto quarter = [&](int f, int kk) {
      constexpr int reads = (ACOL ? 2 : 1) * FM + (BCOL ? 2 : 1) * FN;
      constexpr int each = (reads + kProducts - 1) / kProducts;
      read(f ^ 1, kk);
#pragma unroll
      for (int p = 0; p < kProducts; ++p) product(f, p);
#pragma unroll
      for (int p = 0; p < kProducts; ++p) {
        __builtin_amdgcn_sched_group_barrier(0x100, each, 0);  // LDS reads
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // a matrix instruction
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // this wave's reads of the present stage are done and its loads of the next have
    // arrived, then every wave's; all but the last stages have NS - 2 more in flight
    auto turn = [&](auto more) {
      if constexpr (more) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"((NS - 2) * 2 * L) : "memory");
      else asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
      const uint32_t next = at == (NS - 1) * kStage ? 0u : at + kStage, d = next - at;
      at = next;
#pragma unroll
      for (int i = 0; i < NA; ++i) fa[i] += d;
#pragma unroll
      for (int i = 0; i < NB; ++i) fb[i] += d;
    };
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      if (s < steps) {
        src(s, pa, pb, oa, ob);
#pragma unroll
        for (int i = 0; i < 2 * L; ++i) fetch(i);
        filled();
      }
    }
    if (steps >= NS) asm volatile("s_waitcnt vmcnt(%0)" :: "n"((NS - 1) * 2 * L) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    read(0, 0);
    int s = 0;
    for (; s + NS < steps; ++s) {
#pragma unroll
      for (int q = 0; q < Q - 1; ++q) quarter(q & 1, q + 1);
      turn(std::true_type{});
      src(s + NS, pa, pb, oa, ob);
      read(0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // a wave that is past the barrier goes first: 1.3 % on large products
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int p = 0; p < kProducts || p < 2 * L; ++p) {
        if (p < kProducts) product(1, p);
        if (p < 2 * L) fetch(p);
        __builtin_amdgcn_sched_barrier(0);
      }
      __builtin_amdgcn_s_setprio(0);
      filled();
    }
    for (; s + 1 < steps; ++s) {
#pragma unroll
      for (int q = 0; q < Q - 1; ++q) quarter(q & 1, q + 1);
      turn(std::false_type{});
      quarter(1, 0);
    }
#pragma unroll
    for (int q = 0; q < Q - 1; ++q) quarter(q & 1, q + 1);
#pragma unroll
    for (int p = 0; p < kProducts; ++p) product(1, p);
  }

  // Hands out the accumulators of the wave's j-th 32 columns by rows of n, through LDS so
  // that neighbouring lanes hold neighbouring m: put(n, m, x) for W consecutive m from m
  // on, n and m within the tile.  Before that fix(add) may add to rows: add(r, m, x) to 4
  // values of the wave's r-th row, m from its first.  The caller has a barrier between
  // run() and the first call.
  template <int W, class Fix, class Put> __device__ __forceinline__ void rows_out(lds8* lds, int j, Fix&& fix, Put&& put) const {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    constexpr int kRow = FM * 128, kUnits = FM * 32 / W;  // bytes of a row of m, units of W in it
    lds8* mine = lds + wave * (32 * kRow);
    const int n = lane & 31;
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int chunk = (i * 8 + 2 * q + (lane >> 5)) ^ (n & 15);
        const f32x16& v = acc[i][j];
        *(lds_f32x4*)(mine + n * kRow + chunk * 16) = f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
      }
    auto settle = [] {
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    };
    settle();
    fix([&](int r, int m, const float (&x)[4]) {
      lds_f32x4* at = (lds_f32x4*)(mine + r * kRow + (((m >> 2) ^ (r & 15)) << 4));
      f32x4 v = *at;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += x[e];
      *at = v;
      settle();
    });
#pragma unroll 4
    for (int r = 0; r < 32 * kUnits / 64; ++r) {
      const int at = r * 64 + lane, row = at / kUnits, unit = at % kUnits;
      float x[W];
#pragma unroll
      for (int b = 0; b < W / 4; ++b) {
        const f32x4 v = *(const lds_f32x4*)(mine + row * kRow + (((unit * (W / 4) + b) ^ (row & 15)) << 4));
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * b + e] = v[e];
      }
      put((wave % WN * FN + j) * 32 + row, wave / WN * (FM * 32) + unit * W, x);
    }
    __builtin_amdgcn_wave_barrier();
  }
};

}  // namespace mrr
