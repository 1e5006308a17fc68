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

}  // namespace kda
