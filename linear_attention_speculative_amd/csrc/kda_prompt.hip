// Attention over prompts in the expanded form: keys and values of every head
// from the cached latents, and the causal attention that reads them.
//
//   k_j,h = W_k,h c_j,  v_j,h = W_v,h c_j            kda_latent_expand_kernel
//   s_j = scale (q_h . (k_j,h | r_j)),  out_h = softmax(s) v_.,h
//                                                   kda_latent_prefill_kernel
//
// Per pair of a query and a key this costs 2 (2 D + P) operations a head, where
// the absorbed form has 2 (2 R + P): for prompts it is worth the one product
// with W.
//
// The attention takes both products transposed, with a query a lane (see
// score(), soften() and weigh_bf16() in kda_mma.hpp): a wave has 32 queries of
// one head, a workgroup eight waves, which share 64 keys and values at a time
// in LDS.  The expansion is a matrix product of gathered cache rows with W.
//
// What bounds them (R = 512, P = 64, 32 heads of 128, bf16): the prompt
// attention is bound by the matrix cores.  One prompt of 8192 takes 866 us: 687
// GFLOP of the operator's, 970 of instructions with the weights' second halves,
// which run at 1.12 PFLOP/s (a product of 8192^3 in the library: 1.20).  Other
// orders of instructions within a block of keys take as long.  Scores a block of
// keys ahead of their exponentials took the whole call from 834 us to 798, with
// one half.
// The expansion of its 8192 tokens takes 78 us alone, 69 GFLOP and 134 MB of
// keys and values written: an operand of W out of LDS feeds one product, so that
// its reads take as long as the products; and a token's heads are written 128
// bytes apart in time (110 us in pieces of 8 bytes a lane).
// fp32: 2048 tokens take 140 us (123 TFLOP/s) and 744 us, one tile in LDS.
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// ---- expansion ---------------------------------------------------------------

constexpr int kExpand = 128;       // tokens and columns of a workgroup

// Number of the request of row t: the last b with start[b] <= t.
__device__ __forceinline__ int request_of(const int32_t* start, int B, int t) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (start[m] <= t)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

// Cache entry of key row s, null where nothing is written, kZeros where its
// block is null.
__device__ __forceinline__ const char* key_entry(const ExpandParams& p,
                                                 int s) {
  const PagedParams& c = p.c;
  if (s >= p.S || s < c.qsl[0] || s >= c.qsl[c.B]) return nullptr;
  const int b = request_of(c.qsl, c.B, s);
  const int row = c.req_idx ? c.req_idx[b] : b;
  const int pos = s - max(c.qsl[b], 0);
  const int e = pos / c.block;
  if (row < 0 || row >= c.rows || e >= c.width) return kZeros;
  const int id = c.table[row * c.s_tab_row + e * c.s_tab_col];
  if (id <= c.null_id || id >= c.N) return kZeros;
  return c.cache + id * c.s_blk + int64_t(pos - e * c.block) * c.s_tok;
}

// The rope keys of key rows [s0, s0 + count).
__device__ __forceinline__ void copy_ropes(const ExpandParams& p,
                                           const char* const* entry, int s0,
                                           int count, int offset) {
  for (int i = threadIdx.x; i < count * p.rope_chunks; i += blockDim.x) {
    const int t = i / p.rope_chunks, ch = i - t * p.rope_chunks;
    const char* e = entry[t];
    if (e)
      *reinterpret_cast<u4*>(p.rope + (s0 + t) * p.s_rope + ch * 16) =
          *reinterpret_cast<const u4*>(e == kZeros ? e
                                                   : e + offset + ch * 16);
  }
}

// bf16: a wave keeps the latents of 32 tokens in registers, as the right
// operand, and the workgroup's 256 tokens go through tiles of 32 KB of W in
// LDS, two of them under way.  The products are transposed (columns of W as
// rows): a lane ends with four neighbouring values of one token.  Workgroups
// take equal runs of (256 tokens, tile of W).  (Both operands through LDS, 128
// x 128 a workgroup, took 129 us for 8192 tokens of 32 heads.)
constexpr int kRowTokens = 256, kRowThreads = 512, kRowTile = 32768;
template <int R>
__global__ void __launch_bounds__(kRowThreads, 2)
    kda_latent_expand_rows_kernel(ExpandParams p) {
  constexpr int CH = R / 8;                    // chunks of a row
  constexpr int NC = kRowTile / (R * 2);       // columns of a tile
  constexpr int KF = R / 16, kLoads = kRowTile / 1024 / 8, kBufs = 3;
  constexpr int kLine = NC >= 64 ? NC / 32 : 2;    // blocks of 32 columns
  extern __shared__ __align__(16) char smem[];
  __shared__ const char* entry[kRowTokens];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  const int tiles = p.H * 2 * p.D / NC;
  const int64_t total = int64_t((p.S + kRowTokens - 1) / kRowTokens) * tiles;
  const int64_t per = (total + gridDim.x - 1) / gridDim.x;
  int64_t at = blockIdx.x * per;
  const int64_t last = min(at + per, total);
  const int part_shift = p.D == 64 ? 6 : 7;    // of a column's part
  const uint32_t lds0 = lds_addr(smem);
  auto stage = [&](int tile, int buf) {
    const int l = fresh_tid() & 63;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int i = j * 8 + wave;
      const int rw = i * 64 / CH + (CH < 64 ? l / CH : 0);
      const int n = tile * NC + rw;
      const int h = n >> (part_shift + 1), d = n & (2 * p.D - 1);
      load_lds(p.w + h * p.s_w_head + d * p.s_w_row +
                   (((i * 64 + l) % CH) ^ swizzle<CH>(rw)) * 16,
               uniform(lds0 + buf * kRowTile + i * 1024));
    }
  };
  while (at < last) {
    // one group of tokens: tiles [c0, c1)
    const int group = int(at / tiles), c0 = int(at - int64_t(group) * tiles);
    const int c1 = int(min(int64_t(tiles), c0 + (last - at)));
    const int s0 = group * kRowTokens;
    __syncthreads();                           // the last group is done
    if (tid < kRowTokens) entry[tid] = key_entry(p, s0 + tid);
    __syncthreads();
    stage(c0, 0);
    if (c0 + 1 < c1) stage(c0 + 1, 1);
    if (c0 == 0) copy_ropes(p, entry, s0, kRowTokens, R * 2);
    const char* mine = entry[wave * 32 + (lane & 31)];
    u4 tok[KF];
    {
      const char* src = (mine ? mine : kZeros) + half * 16;
#pragma unroll
      for (int k = 0; k < KF; ++k)
        tok[k] = *reinterpret_cast<const u4*>(src + 32 * k);
#pragma unroll
      for (int k = 0; k < KF; ++k) asm volatile("" : "+v"(tok[k]));
    }
    const int64_t s = s0 + wave * 32 + (lane & 31);
    char* key = p.key + s * p.s_k_tok;
    char* value = p.value + s * p.s_v_tok;
    RowReader<CH, 1> w(lds0, lane, 0);
    // products of tiles that are not written yet: whole lines of 128 bytes are
    u4 done[kLine][2];
    auto write = [&](int n0, int count) {      // 32 columns each, from n0 on
      if (!mine) return;
#pragma unroll
      for (int j = 0; j < kLine; ++j) {
        if (j >= count) break;
        const int n = n0 + 32 * j;
        const int h = n >> (part_shift + 1), d = n & (2 * p.D - 1);
        char* dst = d < p.D ? key + h * p.s_k_head + d * 2
                            : value + h * p.s_v_head + (d - p.D) * 2;
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<u4*>(dst + (16 * e + 8 * half) * 2) = done[j][e];
      }
    };
    auto write_second = [&]() {                // a line's second half alone
      done[0][0] = done[1][0];
      done[0][1] = done[1][1];
      write(c0 * NC, 1);
    };
    int buf = 0;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      // (of what is younger than this tile's loads, the next one's alone may be
      // under way: the stores before them are a tile old)
      if (c + 1 < c1)
        wait_vm<kLoads>();
      else
        wait_vm<0>();
      lds_barrier();                           // and the last tile is read
      if (c > c0) {
        if constexpr (NC >= 64)
          write((c - 1) * NC, kLine);
        else if (c % 2 == 0)
          c - 1 > c0 ? write((c - 2) * NC, 2) : write_second();
      }
      if (c + 2 < c1) stage(c + 2, buf >= 1 ? buf - 1 : 2);
#pragma unroll
      for (int j = 0; j < NC / 32; ++j) {
        const f16v x = score<true>(
            [&](int k) { return w(k, 32 * j); }, tok);
        u4 v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          v[e] = neighbours(u2{pack_bf16(x[8 * e], x[8 * e + 1]),
                               pack_bf16(x[8 * e + 2], x[8 * e + 3])},
                            u2{pack_bf16(x[8 * e + 4], x[8 * e + 5]),
                               pack_bf16(x[8 * e + 6], x[8 * e + 7])});
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (NC >= 64) {
            done[j][e] = v[e];
          } else {
            if (c % 2 == 0)
              done[0][e] = v[e];
            else
              done[1][e] = v[e];
          }
        }
      }
      const bool wrap = buf + 1 == kBufs;
      w.move(uniform(wrap ? -buf * kRowTile : kRowTile));
      buf = wrap ? 0 : buf + 1;
    }
    if constexpr (NC >= 64) {
      write((c1 - 1) * NC, kLine);
    } else {
      // the last tile, with the one before it where they share a line
      if (c1 % 2 == 1)
        write((c1 - 1) * NC, 1);
      else if (c1 - 1 > c0)
        write((c1 - 2) * NC, 2);
      else
        write_second();
    }
    at += c1 - c0;
  }
}

// fp32: 128 tokens x 128 columns, four waves of 64 x 64, both operands through
// LDS, the summed index 128 bytes at a time, transposed as above.
__global__ void __launch_bounds__(256, 2)
    kda_latent_expand_kernel(ExpandParams p) {
  constexpr int ES = 4;
  constexpr int kPart = kExpand * 128;         // bytes of one operand's tile
  extern __shared__ __align__(16) char smem[];
  __shared__ const char* entry[kExpand];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  const int cols = p.H * 2 * p.D;
  const int s0 = blockIdx.x * kExpand, n0 = blockIdx.y * kExpand;
  if (tid < kExpand) entry[tid] = key_entry(p, s0 + tid);
  __syncthreads();
  if (blockIdx.y == 0) copy_ropes(p, entry, s0, kExpand, p.R * ES);
  // a wave's loads: 8 rows of 128 bytes each, four of tokens, four of W
  const char* src[8];
  const int ch = lane & 7;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int rw = (wave * 4 + j) * 8 + (lane >> 3);
    const char* e = entry[rw];
    // (zeros' row is shorter than R: its loads stay at its start)
    src[j] = e == nullptr || e == kZeros ? nullptr
                                         : e + (ch ^ swizzle<8>(rw)) * 16;
    const int n = n0 + rw;
    const int h = n / (2 * p.D), d = n - h * 2 * p.D;
    src[4 + j] = n < cols ? p.w + h * p.s_w_head + d * p.s_w_row +
                                (ch ^ swizzle<8>(rw)) * 16
                          : nullptr;
  }
  const uint32_t lds0 = lds_addr(smem);
  auto stage = [&](int k, int buf) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      load_lds(src[j] ? src[j] + k * 128 : kZeros,
               uniform(lds0 + buf * 2 * kPart + (j >> 2) * kPart +
                       (wave * 4 + (j & 3)) * 1024));
  };
  f16v acc[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
  const int wt = (wave & 1) * 64, wn = (wave >> 1) * 64;
  const int steps = p.R * ES / 128;
  stage(0, 0);
#pragma unroll 1
  for (int k = 0; k < steps; ++k) {
    wait_vm<0>();
    lds_barrier();
    if (k + 1 < steps) stage(k + 1, (k + 1) & 1);
    const char* tok = smem + (k & 1) * 2 * kPart;
    const char* w = tok + kPart;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      u4 a[2], b[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        a[i] = *reinterpret_cast<const u4*>(
            w + place<8>(wn + 32 * i + (lane & 31), 2 * c + half) * 16);
        b[i] = *reinterpret_cast<const u4*>(
            tok + place<8>(wt + 32 * i + (lane & 31), 2 * c + half) * 16);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mma<false>(a[i], b[j],
                                                           acc[i][j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = wt + 32 * j + (lane & 31);
    const int64_t s = s0 + t;
    if (entry[t] == nullptr) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        const int n = n0 + wn + 32 * i + acc_row(e, half);
        if (n >= cols) continue;
        const int h = n / (2 * p.D), d = n - h * 2 * p.D;
        char* dst = d < p.D ? p.key + s * p.s_k_tok + h * p.s_k_head + d * ES
                            : p.value + s * p.s_v_tok + h * p.s_v_head +
                                  (d - p.D) * ES;
        const f16v& v = acc[i][j];
        *reinterpret_cast<f4*>(dst) = f4{v[e], v[e + 1], v[e + 2], v[e + 3]};
      }
  }
}

// ---- attention -----------------------------------------------------------------

constexpr int kWaves = 8;
constexpr int kQueries = 32 * kWaves;
constexpr int kKeys = 64;          // keys of a step

template <bool BF16, int D, int P>
struct Prompt {
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int CH = D * ES / 16, CHP = P * ES / 16;
  static constexpr int KF = (D + P) * ES / 32;
  static constexpr int NB = D / 32;
  static constexpr int LK = kKeys * CH / 64, LP = kKeys * CHP / 64;  // loads
  static constexpr int MINE = (2 * LK + LP) / kWaves;
  static constexpr int TILE = kKeys * (2 * CH + CHP) * 16;
  static constexpr int NBUF = BF16 ? 3 : 1;    // (fp32: one fits)
  static constexpr int ROPE = kKeys * CH * 16, VALUE = ROPE + kKeys * CHP * 16;
  static_assert(LK % kWaves == 0 && LP % kWaves == 0, "loads");
};

template <bool BF16, int D, int P>
__global__ void __launch_bounds__(64 * kWaves, 2)
    kda_latent_prefill_kernel(PromptParams p) {
  using Z = Prompt<BF16, D, P>;
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  // blocks i, i + 8, .. are on one XCD: a head's query tiles, which read the
  // same keys, where H is a multiple of 8.  The last tiles, which have the
  // most keys, come first.
  const int h = blockIdx.x % p.H, item = blockIdx.x / p.H;
  int64_t* red = reinterpret_cast<int64_t*>(smem);
  int32_t* found = reinterpret_cast<int32_t*>(smem + 64);
  if (tid == 0) found[0] = -1;
  int64_t done = 0;
  for (int b0 = 0; b0 < p.B; b0 += 64 * kWaves) {
    // requests from the last to the first
    const int b = p.B - 1 - (b0 + tid);
    int v = 0;
    if (b >= 0) {
      const int bos = min(max(p.qsl[b], 0), p.T);
      v = (min(max(p.qsl[b + 1], bos), p.T) - bos + kQueries - 1) / kQueries;
    }
    int64_t upto = v;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    __syncthreads();
    if (lane == 63) red[wave] = upto;
    __syncthreads();
    int64_t before = done;
    for (int k = 0; k < wave; ++k) before += red[k];
    const int64_t at = before + upto - v;
    if (v > 0 && at <= item && item < at + v) {
      found[0] = b;
      found[1] = v - 1 - int(item - at);       // its last tiles first
    }
    for (int k = 0; k < kWaves; ++k) done += red[k];
    if (done > item) break;
  }
  __syncthreads();
  const int b = uniform(found[0]), tile = uniform(found[1]);
  __syncthreads();
  if (b < 0) return;
  const int bos = min(max(p.qsl[b], 0), p.T);
  const int len = min(max(p.qsl[b + 1], bos), p.T) - bos;
  const int kbos = min(max(p.ksl[b], 0), p.S);
  const int keys = min(max(p.ksl[b + 1], kbos), p.S) - kbos;
  const int ahead = keys - len;                // keys in front of the queries
  const int t0 = tile * kQueries + wave * 32;
  const int tok = t0 + (lane & 31);
  // keys of this lane's query, of the wave and of the workgroup
  const int lim = ahead + min(tok, len - 1) + 1;
  const int wave_lim = t0 < len ? ahead + min(t0 + 32, len) : 0;
  const int n = ahead + min((tile + 1) * kQueries, len);
  const int steps = n > 0 ? (n + kKeys - 1) / kKeys : 0;

  f16v o[Z::NB];
#pragma unroll
  for (int k = 0; k < Z::NB; ++k)
#pragma unroll
    for (int i = 0; i < 16; ++i) o[k][i] = 0.0f;
  float top = -INFINITY, sum = 0.0f;

  const char* key = p.key + int64_t(kbos) * p.s_k_tok + h * p.s_k_head;
  const char* value = p.value + int64_t(kbos) * p.s_v_tok + h * p.s_v_head;
  const char* rope = p.rope + int64_t(kbos) * p.s_rope;
  const uint32_t lds0 = lds_addr(smem);
  // This lane's places of the next step's loads.
  const char* src[Z::MINE];
  auto row_of = [&](int j, int l) {
    const int i = j * kWaves + wave;
    constexpr int CP = Z::CHP > 0 ? Z::CHP : 8;
    return j * kWaves < Z::LK ? i * (64 / Z::CH) + l / Z::CH
           : j * kWaves < Z::LK + Z::LP
               ? (i - Z::LK) * (64 / CP) + l / CP
               : (i - Z::LK - Z::LP) * (64 / Z::CH) + l / Z::CH;
  };
  auto stride_of = [&](int j) {
    return j * kWaves < Z::LK            ? p.s_k_tok
           : j * kWaves < Z::LK + Z::LP ? p.s_rope
                                        : p.s_v_tok;
  };
  auto place_of = [&](int j, int l) {
    constexpr int CP = Z::CHP > 0 ? Z::CHP : 8;
    const bool is_rope = j * kWaves >= Z::LK && j * kWaves < Z::LK + Z::LP;
    const int rw = row_of(j, l);
    const int ch = is_rope ? (l % CP) ^ swizzle<CP>(rw)
                           : (l % Z::CH) ^ swizzle<Z::CH>(rw);
    return (j * kWaves < Z::LK ? key : is_rope ? rope : value) +
           rw * stride_of(j) + ch * 16;
  };
  // (fp32 queries leave no registers for the places: formed for each step)
  if constexpr (BF16)
#pragma unroll
    for (int j = 0; j < Z::MINE; ++j) src[j] = place_of(j, lane);
  auto stage = [&](int step, int buf) {
    const uint32_t to = uniform(lds0 + buf * Z::TILE + wave * 1024);
    const int l = fresh_tid() & 63;
    if constexpr (!BF16)
#pragma unroll
      for (int j = 0; j < Z::MINE; ++j)
        src[j] = place_of(j, l) + int64_t(step) * kKeys * stride_of(j);
    if ((step + 1) * kKeys <= n) {
#pragma unroll
      for (int j = 0; j < Z::MINE; ++j)
        load_lds(src[j], to + j * kWaves * 1024);
    } else {
#pragma unroll
      for (int j = 0; j < Z::MINE; ++j)
        load_lds(step * kKeys + row_of(j, l) < n ? src[j] : kZeros,
                 to + j * kWaves * 1024);
    }
    if constexpr (BF16)
#pragma unroll
      for (int j = 0; j < Z::MINE; ++j) src[j] += kKeys * stride_of(j);
  };

  constexpr int kAhead = Z::NBUF > 1 ? Z::NBUF - 1 : 0;
#pragma unroll
  for (int k = 0; k < kAhead; ++k)
    if (k < steps) stage(k, k);
  // The queries, after the first tiles' loads and waited for here: a wait in
  // the loop would wait for the tiles under way, too.
  u4 q[Z::KF];
  {
    const char* src = p.q + int64_t(bos + min(tok, len - 1)) * p.s_q_tok +
                      h * p.s_q_head + half * 16;
#pragma unroll
    for (int k = 0; k < Z::KF; ++k)
      q[k] = negated<BF16>(*reinterpret_cast<const u4*>(src + 32 * k),
                           p.negate);
#pragma unroll
    for (int k = 0; k < Z::KF; ++k) asm volatile("" : "+v"(q[k]));
  }
  RowReader<Z::CH, 1> heads(lds0, lane, 0);
  RowReader<(Z::CHP > 0 ? Z::CHP : 8), 1> ropes(lds0 + Z::ROPE, lane, 0);
  if constexpr (BF16) {
    // Scores are one block of 32 keys ahead: their products run beside the
    // exponentials of the block before, the values' beside the search for the
    // maximum.  The next step's tile is there from the middle of a step on.
    ColumnReader<Z::CH> values(lds0 + Z::VALUE, 0, lane);
    auto next_scores = [&](int row) {
      f16v x;
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll
      for (int i = 0; i < Z::KF; ++i)
        x = mma<true>(i < Z::CH / 2 ? heads(i, row)
                                    : ropes(i - Z::CH / 2, row),
                      q[i], x);
      return x;
    };
    f16v ahead_scores;
    float m = -INFINITY;
    if (steps > 0) {
      wait_tile<kAhead - 1>(steps, std::integral_constant<int, Z::MINE>());
      lds_barrier();
      ahead_scores = next_scores(0);
      hide(ahead_scores, lim, half);
      m = highest(ahead_scores);
    }
    // one block: keys `at` .., the next block's in rows [next, next + 32) of
    // the tile that the readers are at
    auto block = [&](int at, int row, int next) {
      raise(m * p.scale, top, sum, o);
      const f16v now = ahead_scores;
      float x[16];
      u4 pr[2], lo[2];
      __builtin_amdgcn_sched_barrier(0);
      ahead_scores = next_scores(next);
      soften(now, p.scale, top, sum, x);
      pack_weights(x, pr, lo);
      // (here, not where they are used)
      asm volatile("" : "+v"(pr[0]), "+v"(pr[1]), "+v"(lo[0]), "+v"(lo[1]),
                   "+v"(sum));
      // two reads ahead, then for each product a read, four additions or
      // multiplications and two exponentials
      __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
#pragma unroll
      for (int i = 0; i < Z::KF; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        __builtin_amdgcn_sched_group_barrier(0x400, 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      hide(ahead_scores, lim - at - 32, half);
      m = highest(ahead_scores);
      weigh_bf16(values, row, pr, lo, __all(lim - at >= 32), lim - at, o);
    };
    int buf = 0;
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      const int at = s * kKeys;
      if (at < wave_lim) block(at, 0, 32);
      const bool wrap = buf + 1 == Z::NBUF;
      const int by = uniform(wrap ? -buf * Z::TILE : Z::TILE);
      heads.move(by);
      if (Z::CHP > 0) ropes.move(by);
      if (s + 1 < steps) {
        // (the tile after it goes where the last step's was, which every wave
        // has read by now)
        wait_vm<0>();
        lds_barrier();
        if (s + 2 < steps) stage(s + 2, (buf + 2) % Z::NBUF);
      }
      if (at + 32 < wave_lim) block(at + 32, 32, 0);
      values.move(by);
      buf = wrap ? 0 : buf + 1;
    }
  } else {
#pragma unroll 1
    for (int s = 0; s < steps; ++s) {
      lds_barrier();                       // the last step's tile is read
      stage(s, 0);
      wait_vm<0>();
      lds_barrier();
#pragma unroll
      for (int k = 0; k < kKeys; k += 32) {
        const int at = s * kKeys + k;
        if (at < wave_lim) {
          f16v sc = score<false>(
              [&](int i) {
                return i < Z::CH / 2 ? heads(i, k) : ropes(i - Z::CH / 2, k);
              },
              q);
          hide(sc, lim - at, half);
          raise(highest(sc) * p.scale, top, sum, o);
          float x[16];
          soften(sc, p.scale, top, sum, x);
          weigh_f32<Z::CH>(lds0 + Z::VALUE + k * Z::CH * 16, 0, x,
                           __all(lim - at >= 32), lim - at, o);
        }
      }
    }
  }
  sum = halves_sum(sum);
  if (tok >= len) return;
  const float by = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
  char* dst = p.out + int64_t(bos + tok) * p.s_out_tok + h * p.s_out_head;
#pragma unroll
  for (int k = 0; k < Z::NB; ++k)
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      const int e = 32 * k + acc_row(i, half);
      if constexpr (BF16)
        *reinterpret_cast<u2*>(dst + e * 2) =
            u2{pack_bf16(o[k][i] * by, o[k][i + 1] * by),
               pack_bf16(o[k][i + 2] * by, o[k][i + 3] * by)};
      else
        *reinterpret_cast<f4*>(dst + e * 4) = f4{
            o[k][i] * by, o[k][i + 1] * by, o[k][i + 2] * by,
            o[k][i + 3] * by};
    }
  if (p.lse && half == 0)
    p.lse[int64_t(bos + tok) * p.s_lse_tok + h * p.s_lse_head] =
        sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

template <bool BF16, int D, int P>
int launch(const PromptParams& p, hipStream_t stream) {
  using Z = Prompt<BF16, D, P>;
  constexpr int lds = Z::NBUF * Z::TILE;
  static_assert(lds <= 160 * 1024, "LDS");
  const auto kernel = kda_latent_prefill_kernel<BF16, D, P>;
  const hipError_t e = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kernel),
      hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return int(e);
  launch_kernel(kernel, dim3(uint32_t(prompt_tiles(p.T, p.B) * p.H)),
                dim3(64 * kWaves), lds, stream, p);
  return int(hipGetLastError());
}

template <bool BF16>
int launch_dims(const PromptParams& p, int D, int P, hipStream_t stream) {
  if (D == 128 && P == 64) return launch<BF16, 128, 64>(p, stream);
  if (D == 128 && P == 0) return launch<BF16, 128, 0>(p, stream);
  if (D == 64 && P == 64) return launch<BF16, 64, 64>(p, stream);
  if (D == 64 && P == 0) return launch<BF16, 64, 0>(p, stream);
  return int(hipErrorInvalidValue);
}

}  // namespace

// Query tiles of T tokens in B requests, at most.
int64_t prompt_tiles(int64_t T, int64_t B) { return T / kQueries + B; }

int launch_latent_prefill(const PromptParams& p, int D, int P, bool bf16,
                          hipStream_t stream) {
  return bf16 ? launch_dims<true>(p, D, P, stream)
              : launch_dims<false>(p, D, P, stream);
}

namespace {
template <int R>
int launch_rows(const ExpandParams& p, hipStream_t stream) {
  const auto kernel = kda_latent_expand_rows_kernel<R>;
  const hipError_t e = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kernel),
      hipFuncAttributeMaxDynamicSharedMemorySize, 3 * kRowTile);
  if (e != hipSuccess) return int(e);
  launch_kernel(kernel, dim3(256), dim3(kRowThreads), 3 * kRowTile, stream, p);
  return int(hipGetLastError());
}
}  // namespace

int launch_latent_expand(const ExpandParams& p, bool bf16,
                         hipStream_t stream) {
  if (bf16) {
    if (p.R == 512) return launch_rows<512>(p, stream);
    if (p.R == 256) return launch_rows<256>(p, stream);
    if (p.R == 128) return launch_rows<128>(p, stream);
    return int(hipErrorInvalidValue);
  }
  // (beside the static entries: more than the 64 KB that need no leave)
  constexpr int lds = 4 * kExpand * 128;
  static_assert(lds + kExpand * 8 <= 160 * 1024, "LDS");
  const hipError_t e = hipFuncSetAttribute(
      reinterpret_cast<const void*>(kda_latent_expand_kernel),
      hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return int(e);
  launch_kernel(kda_latent_expand_kernel,
                dim3((p.S + kExpand - 1) / kExpand,
                     (p.H * 2 * p.D + kExpand - 1) / kExpand),
                dim3(256), lds, stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
