// Matrix-instruction pieces shared by the latent attention kernels: operands
// of 16 bytes a lane, loads from global memory straight into LDS, and the
// order in which LDS holds a tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_device.hpp"

namespace kda {

typedef float f16v __attribute__((ext_vector_type(16)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef uint32_t u2 __attribute__((ext_vector_type(2)));
typedef uint32_t u4 __attribute__((ext_vector_type(4)));
typedef short s4 __attribute__((ext_vector_type(4)));

// A 32 x 32 product over the 16 bytes of each of the two lane halves: lane l
// holds row (or column) l % 32 and, of the summed index, the chunk l / 32.
// The result's column is l % 32; register i holds row 8 (i / 4) + 4 (l / 32)
// + i % 4.
template <bool BF16>
__device__ __forceinline__ f16v mma(u4 a, u4 b, f16v c) {
  if constexpr (BF16) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(
        __builtin_bit_cast(b8, a), __builtin_bit_cast(b8, b), c, 0, 0, 0);
  } else {
    // one place of each chunk at a time: true fp32 products
#pragma unroll
    for (int e = 0; e < 4; ++e)
      c = __builtin_amdgcn_mfma_f32_32x32x2f32(
          __uint_as_float(a[e]), __uint_as_float(b[e]), c, 0, 0, 0);
    return c;
  }
}

// Two floats as bf16, rounded to nearest even; the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{a, b}, b2));
}

// Row that register i of lane half h holds of a 32 x 32 result.
__device__ __forceinline__ constexpr int acc_row(int i, int h) {
  return 8 * (i / 4) + 4 * h + i % 4;
}

// The largest, or the sum, of a value of lane l and that of lane l ^ 32.
__device__ __forceinline__ float halves_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
}
__device__ __forceinline__ float halves_sum(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float(s[0]) + __uint_as_float(s[1]);
}

// One wave's load of 64 x 16 bytes into LDS, in lane order, from an address
// of each lane, or from a uniform one plus an offset of each lane.  The wait
// is by hand (wait_vm): the compiler keeps no count of these loads.
__device__ __forceinline__ void load_lds(const char* addr, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(addr)
      : "memory");
}
__device__ __forceinline__ void load_lds(uint64_t base, uint32_t off,
                                         uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory");
}

// Wait until at most N of this wave's global memory operations are under way
// (they end in the order in which they began).
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "count");
  asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const char*)p));
}

// Where LDS holds chunk c (16 bytes) of row r of a tile whose rows have CH
// chunks: rows stay apart, chunks within a row are permuted, so that neither
// 16 rows of one chunk (an operand read as it lies) nor 4 rows of 4 chunks (a
// transposed one) meet in a bank.  In chunks, from the tile's start.
template <int CH>
__device__ __forceinline__ constexpr int swizzle(int r) {
  return CH >= 16 ? ((r & 3) << 2) | ((r >> 2) & 3) : (r >> 1) & 7;
}
template <int CH>
__device__ __forceinline__ constexpr int place(int r, int c) {
  return r * CH + (c ^ swizzle<CH>(r));
}

// The left operand of a product with the transpose of rows [t, t + 16) of a
// bf16 tile: result row m = l % 32 is element 32 blk + m of the tile's rows;
// lane half h sums over rows t + 4 h + {0..3} and t + 8 + 4 h + {0..3}, the
// order in which a product's result has its own rows.
template <int CH>
__device__ __forceinline__ u4 load_transposed(const char* tile, int t,
                                              int blk) {
  typedef s4 __attribute__((address_space(3))) * lp;
  const int l = threadIdx.x & 63, i = l & 15;
  const int row = t + 4 * (l >> 5) + (i >> 2);
  const int c = 4 * blk + 2 * ((l >> 4) & 1) + ((i & 3) >> 1);
  const char* a = tile + place<CH>(row, c) * 16 + (i & 1) * 8;
  const char* b = tile + place<CH>(row + 8, c) * 16 + (i & 1) * 8;
  const u2 x = __builtin_bit_cast(
      u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)a));
  const u2 y = __builtin_bit_cast(
      u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)b));
  return u4{x[0], x[1], y[0], y[1]};
}

// The running maximum is only moved when it is passed by more than this (in
// powers of two): weights of up to 2^kSlack cost nothing in fp32 or bf16, and
// moving it costs a pass over O.
constexpr float kSlack = 8.0f;

// What places without a token read (static: a copy for each source file).
static __device__ const char kZeros[4096] = {};

// Wait for the oldest of the steps under way: `left` steps remain, of which up
// to AHEAD + 1 are under way, with MINE loads each.
template <int AHEAD, int MINE>
__device__ __forceinline__ void wait_tile(int left,
                                          std::integral_constant<int, MINE>) {
  if constexpr (AHEAD * MINE < 64 && AHEAD > 0) {
    if (left > AHEAD) return wait_vm<AHEAD * MINE>();
    wait_tile<AHEAD - 1>(left, std::integral_constant<int, MINE>());
  } else {
    wait_vm<0>();
  }
}

// 32 tokens against a wave's 32 queries, one a lane: S^T = K q^T, the softmax's
// running maximum (`top`, in powers of two) and sum, O^T += V^T P^T.  Keys are
// two tiles side by side (CH and CHP chunks a row), values NB blocks of 32 of a
// tile's rows from block `blk` on.  `live`: which tokens are there; the lane's
// query sees the first `left` of them.
template <bool BF16, int CH, int CHP, int CHV, int KF, int NB>
__device__ __forceinline__ void attend(const char* keys, const char* ropes,
                                       const char* values, int blk,
                                       const u4 (&q)[KF], f16v (&o)[NB],
                                       float& top, float& sum, uint32_t live,
                                       int left, float scale) {
  constexpr int kTile = 32;
  // (operands are read a few ahead of their products; without the borders
  // the compiler reads them all at once and has no registers left)
  constexpr int G = 3;
  const int lane = fresh_tid() & 63, half = lane >> 5;
  auto key = [&](int k) -> u4 {
    const int ch = 2 * k + half;
    const char* a =
        2 * k < CH ? keys + place<CH>(lane & 31, ch) * 16
                   : ropes + place<(CHP > 0 ? CHP : 8)>(lane & 31, ch - CH) *
                                 16;
    return *reinterpret_cast<const u4*>(a);
  };
  f16v x0;
#pragma unroll
  for (int i = 0; i < 16; ++i) x0[i] = 0.0f;
  u4 kk[2][G];
#pragma unroll
  for (int j = 0; j < G && j < KF; ++j) kk[0][j] = key(j);
#pragma unroll
  for (int k = 0; k < KF; k += G) {
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (k + G + j < KF) kk[(k / G + 1) & 1][j] = key(k + G + j);
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (k + j < KF) x0 = mma<BF16>(kk[(k / G) & 1][j], q[k + j], x0);
    __builtin_amdgcn_sched_barrier(0);
  }
  float x[16], m = -INFINITY;
  if (__all(left == kTile) && live == 0xffffffffu) {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = x0[i] * scale;
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = acc_row(i, half);
      const bool see = t < left && ((live >> t) & 1);
      x[i] = see ? x0[i] * scale : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, x[i]);
  m = halves_max(m);
  if (__any(m > top + kSlack)) {
    const float to = fmaxf(top, m);
    const float by = top == -INFINITY ? 0.0f : exp2f(top - to);
    top = to;
    sum *= by;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[k][i] *= by;
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __builtin_amdgcn_exp2f(x[i] - base);
    sum += x[i];
  }
  if constexpr (BF16) {
    u4 pr[2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      pr[t] = u4{pack_bf16(x[8 * t], x[8 * t + 1]),
                 pack_bf16(x[8 * t + 2], x[8 * t + 3]),
                 pack_bf16(x[8 * t + 4], x[8 * t + 5]),
                 pack_bf16(x[8 * t + 6], x[8 * t + 7])};
    u4 v[2][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
      v[0][t] = load_transposed<CHV>(values, 16 * t, blk);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (k + 1 < NB)
          v[(k + 1) & 1][t] =
              load_transposed<CHV>(values, 16 * t, blk + k + 1);
#pragma unroll
      for (int t = 0; t < 2; ++t) o[k] = mma<true>(v[k & 1][t], pr[t], o[k]);
      __builtin_amdgcn_sched_barrier(0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int t = acc_row(i, half);
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        const int e = 32 * (blk + k) + (lane & 31);
        const float v = *reinterpret_cast<const float*>(
            values + place<CHV>(t, e / 4) * 16 + e % 4 * 4);
        o[k] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, x[i], o[k], 0, 0, 0);
      }
      if (i & 1) __builtin_amdgcn_sched_barrier(0);
    }
  }
}

}  // namespace kda
