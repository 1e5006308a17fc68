// Matrix-instruction pieces shared by the latent attention kernels: operands
// of 16 bytes a lane, loads from global memory straight into LDS, and the
// order in which LDS holds a tile.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kda_device.hpp"

namespace kda {

typedef float f2 __attribute__((ext_vector_type(2)));
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
// is by hand (wait_vm): the compiler keeps no count of these loads.  (m0 is a
// reserved register, which the compiler warns of; named, its own settings of m0
// are not merged across.)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void load_lds(const char* addr, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, off"
      :
      : "s"(lds), "v"(addr)
      : "memory", "m0");
}
__device__ __forceinline__ void load_lds(uint64_t base, uint32_t off,
                                         uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(lds), "v"(off), "s"(base)
      : "memory", "m0");
}
#pragma clang diagnostic pop

// Two registers' worth of four bf16 values of one row of a result's columns,
// those of registers 8 k + {0..3} and 8 k + {4..7}, as eight neighbouring
// values: from row 16 k on in lanes 0 .. 31, from row 16 k + 8 on in the others.
__device__ __forceinline__ u4 neighbours(u2 a, u2 b) {
  const auto x = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
  const auto y = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
  return u4{x[0], y[0], x[1], y[1]};
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

// The operands of row l % 32 that share `part` of PARTS reads: its k-th is
// chunk 2 (PARTS k + part) + l / 32.  The swizzle repeats every 16 chunks (8 in
// rows of 8), so a few addresses and immediate offsets serve a whole row, and
// rows 32 further on; the addresses move with the tile.
typedef __attribute__((address_space(3))) const u4* lds_u4;
template <int CH, int PARTS>
struct RowReader {
  static constexpr int PERIOD = CH >= 16 ? 16 : 8;
  static constexpr int N = PERIOD / (2 * PARTS);   // operands of a period
  static_assert(N >= 1, "parts");
  uint32_t at[N];
  __device__ __forceinline__ RowReader(uint32_t tile, int lane, int part) {
#pragma unroll
    for (int k = 0; k < N; ++k)
      at[k] = tile + place<CH>(lane & 31,
                               2 * (PARTS * k + part) + (lane >> 5)) * 16;
  }
  __device__ __forceinline__ u4 operator()(int k, int row = 0) const {
    return *(lds_u4)uintptr_t(at[k % N] + (k / N * PERIOD + row * CH) * 16);
  }
  __device__ __forceinline__ void move(int by) {
#pragma unroll
    for (int k = 0; k < N; ++k) at[k] += by;
  }
};

// The left operand of a product with the transpose of rows [t, t + 16) of a
// bf16 tile, t a multiple of 16: result row m = l % 32 is element 32 blk + m of
// the tile's rows; lane half h sums over rows t + 4 h + {0..3} and t + 8 + 4 h
// + {0..3}, the order in which a product's result has its own rows.
template <int CH>
struct ColumnReader {
  static constexpr int N = CH >= 16 ? 4 : 2;   // blocks of a swizzle's period
  uint32_t at[N][2];
  // blocks are counted from `blk0` on, at any place of a period
  __device__ __forceinline__ ColumnReader(uint32_t tile, int blk0, int lane) {
    const int i = lane & 15;
    const int row = 4 * (lane >> 5) + (i >> 2);
    const int c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        at[k][e] = tile + place<CH>(row + 8 * e, 4 * (blk0 + k) + c) * 16 +
                   (i & 1) * 8;
  }
  __device__ __forceinline__ u4 operator()(int t, int blk) const {
    typedef s4 __attribute__((address_space(3))) * lp;
    const int off = t * CH * 16 + blk / N * (N * 64);
    const u2 x = __builtin_bit_cast(
        u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lp)uintptr_t(at[blk % N][0] + off)));
    const u2 y = __builtin_bit_cast(
        u2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lp)uintptr_t(at[blk % N][1] + off)));
    return u4{x[0], x[1], y[0], y[1]};
  }
  __device__ __forceinline__ void move(int by) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      at[k][0] += by;
      at[k][1] += by;
    }
  }
};

// The fp32 counterpart: one value, element 32 blk + l % 32 of row t, of a tile
// at `tile`.
template <int CH>
__device__ __forceinline__ float column_value(uint32_t tile, int t, int blk,
                                              int lane) {
  const int e = 32 * blk + (lane & 31);
  return *(__attribute__((address_space(3))) const float*)uintptr_t(
      tile + place<CH>(t, e / 4) * 16 + e % 4 * 4);
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

// S^T = K q^T of 32 tokens and a wave's 32 queries, one a lane: key(k) is the
// k-th operand of the lane's token.
template <bool BF16, int KF, class Key>
__device__ __forceinline__ f16v score(Key key, const u4 (&q)[KF]) {
  // (operands are read a few ahead of their products; without the borders
  // the compiler reads them all at once and has no registers left)
  constexpr int G = 3;
  f16v x;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = 0.0f;
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
      if (k + j < KF) x = mma<BF16>(kk[(k / G) & 1][j], q[k + j], x);
    __builtin_amdgcn_sched_barrier(0);
  }
  return x;
}

// Scores that the lane's query does not see (it sees the first `left` tokens).
__device__ __forceinline__ void hide(f16v& s, int left, int half) {
  if (__all(left >= 32)) return;
  asm volatile("");                    // (a branch of its own)
#pragma unroll
  for (int i = 0; i < 16; ++i)
    s[i] = acc_row(i, half) < left ? s[i] : -INFINITY;
}

// The largest score of the lane's query.
__device__ __forceinline__ float highest(const f16v& s) {
  float m = fmaxf(s[0], s[1]);
#pragma unroll
  for (int i = 2; i < 16; i += 2) m = fmaxf(fmaxf(m, s[i]), s[i + 1]);
  return halves_max(m);
}

// Moves the running maximum `top` (in powers of two) to m where it is passed by
// more than kSlack, and scales the sum and O with it.
template <int NB>
__device__ __forceinline__ void raise(float m, float& top, float& sum,
                                      f16v (&o)[NB]) {
  if (!__any(m > top + kSlack)) return;
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

// Softmax weights of scores under that maximum, and their sum.
__device__ __forceinline__ void soften(const f16v& s, float scale, float top,
                                       float& sum, float (&x)[16]) {
  const float base = top == -INFINITY ? 0.0f : -top;
  float part[4] = {sum, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], scale, base));
    part[i & 3] += x[i];
  }
  sum = (part[0] + part[1]) + (part[2] + part[3]);
}

// Two weights as bf16 values in halves: the leading 8 bits of each, and what
// they leave, rounded.  Together they are off by 2^-15 of a weight at most; one
// bf16 value would be by 2^-8, as much as the output's own rounding.  The second
// is kept above 0 (2^-23 of the weight more): values that are not finite meet
// both, and 0 times infinity would be NaN.
__device__ __forceinline__ u2 split_bf16(float a, float b) {
  const uint32_t i = __float_as_uint(a), j = __float_as_uint(b);
  constexpr float up = 1.0f + 0x1p-23f;
  return u2{__builtin_amdgcn_perm(j, i, 0x07060302u),
            pack_bf16(
                __builtin_fmaf(a, up, -__uint_as_float(i & 0xffff0000u)),
                __builtin_fmaf(b, up, -__uint_as_float(j & 0xffff0000u)))};
}

// The weights of a result's registers as operands, in halves: pr[t] and lo[t]
// hold tokens 16 t + 4 h + {0..3} and 16 t + 8 + 4 h + {0..3}, h = lane / 32.
__device__ __forceinline__ void pack_weights(const float (&x)[16], u4 (&pr)[2],
                                             u4 (&lo)[2]) {
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const u2 w = split_bf16(x[8 * t + 2 * e], x[8 * t + 2 * e + 1]);
      pr[t][e] = w[0];
      lo[t][e] = w[1];
    }
}

// Bits of the tokens acc_row(i, half) of a block that a query sees, the first
// `left` of it.
__device__ __forceinline__ uint32_t seen_bits(int left, int half) {
  uint32_t seen = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i)
    seen |= uint32_t(acc_row(i, half) < left) << i;
  return seen;
}

// Values that are not finite, at tokens that some of a wave's queries see and
// others do not: 0 times them is NaN, so they are taken out of the operands,
// and the largest finite value in their place times 2^100 where a query sees
// them makes its sum +inf, then -inf (NaN: both, which leaves NaN).
__device__ __forceinline__ void spoil_bf16(u4 (&v)[2], uint32_t seen, f16v& o) {
  uint32_t bad = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) bad |= (v[t][e] & 0x7f807f80u) + 0x00800080u;
  if (!__any(bad & 0x80008000u)) return;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    u4 up, down, is;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      up[e] = down[e] = 0;
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        const uint32_t w = (v[t][e] >> h) & 0xffffu;
        if (w == 0x7f80u || (w & 0x7fffu) > 0x7f80u) up[e] |= 0x7f7fu << h;
        if (w == 0xff80u || (w & 0x7fffu) > 0x7f80u) down[e] |= 0xff7fu << h;
        if ((w & 0x7f80u) == 0x7f80u) v[t][e] &= 0xffff0000u >> h;
      }
      const uint32_t s = seen >> (8 * t + 2 * e);
      is[e] = ((s & 1) | (s & 2) << 15) * 0x7180u;        // 2^100
    }
    o = mma<true>(up, is, o);
    o = mma<true>(down, is, o);
  }
}

// O^T += V^T P^T: NB blocks of 32 of the values' rows [row, row + 32).  Of
// these tokens each query of the wave sees all (`all`), or the first `left`.
template <int NB, class Column>
__device__ __forceinline__ void weigh_bf16(const Column& value_at, int row,
                                           const u4 (&pr)[2],
                                           const u4 (&lo)[2], bool all,
                                           int left, f16v (&o)[NB]) {
  u4 v[2][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) v[0][t] = value_at(row + 16 * t, 0);
#pragma unroll
  for (int k = 0; k < NB; ++k) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (k + 1 < NB) v[(k + 1) & 1][t] = value_at(row + 16 * t, k + 1);
    // (here it takes 1 % of the prompts' time; a loop of its own for such
    // steps, or two blocks at a time, take more registers than there are)
    if (!all)
      spoil_bf16(v[k & 1], seen_bits(left, (fresh_tid() >> 5) & 1), o[k]);
#pragma unroll
    for (int t = 0; t < 2; ++t) o[k] = mma<true>(v[k & 1][t], pr[t], o[k]);
#pragma unroll
    for (int t = 0; t < 2; ++t) o[k] = mma<true>(v[k & 1][t], lo[t], o[k]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// The same for the fp32 values of tokens acc_row(i, lane / 32), by bf16
// products (an fp32 one adds to its sum before it overflows: +inf would stay).
__device__ __forceinline__ void spoil_f32(float& v, int i, int left, f16v& o) {
  if (!__any(!(fabsf(v) < INFINITY))) return;
  const bool see = acc_row(i, (fresh_tid() >> 5) & 1) < left;
  const bool up = v == INFINITY || v != v, down = v == -INFINITY || v != v;
  if (up || down) v = 0.0f;
  auto add = [&](uint32_t a) {
    o = __builtin_amdgcn_mfma_f32_32x32x8bf16_1k(
        __builtin_bit_cast(s4, u2{a, 0}),
        __builtin_bit_cast(s4, u2{see ? 0x7180u : 0u, 0}), o, 0, 0, 0);
  };
  add(up ? 0x7f7fu : 0u);
  add(down ? 0xff7fu : 0u);
}

// fp32: x[i] is the weight of token acc_row(i, lane / 32) of the tile's.
template <int CHV, int NB>
__device__ __forceinline__ void weigh_f32(uint32_t values, int blk,
                                          const float (&x)[16], bool all,
                                          int left, f16v (&o)[NB]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int lane = fresh_tid() & 63;
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      float v = column_value<CHV>(values, acc_row(i, lane >> 5), blk + k, lane);
      if (!all) spoil_f32(v, i, left, o[k]);
      o[k] = __builtin_amdgcn_mfma_f32_32x32x2f32(v, x[i], o[k], 0, 0, 0);
    }
    if (i & 1) __builtin_amdgcn_sched_barrier(0);
  }
}

// Query operands of a scale below 0 are negated, so that scores rise with their
// weights.
template <bool BF16>
__device__ __forceinline__ u4 negated(u4 q, bool yes) {
  const uint32_t flip = !yes ? 0u : BF16 ? 0x80008000u : 0x80000000u;
#pragma unroll
  for (int e = 0; e < 4; ++e) q[e] ^= flip;
  return q;
}

}  // namespace kda
