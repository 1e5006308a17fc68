// Attention over a paged cache of latent vectors, in the absorbed form, and
// the write into that cache.
//
// A token's cache entry is its latent c_j (R values) and its rope key r_j (P
// values).  With the query of a head already in latent space, q = (q_c | q_r):
//   s_j = scale (q_c . c_j + q_r . r_j),  p = softmax(s),  out = sum_j p_j c_j,
// for j up to the query's own position: every head of a request reads the
// same entries, once as keys and once as values.
//
// Both products are taken transposed, S^T = K q^T and O^T = V^T P^T, with 32
// queries (rows: token, head) as the columns of 32 x 32 products.  A lane
// then has one query throughout: the maximum and the sum of its softmax are
// its own (and lane l ^ 32's), the probabilities become the right operand of
// the second product where they are, and a wave keeps q (R + P values a row)
// and O (R values) in registers.  The values are the keys' tile in LDS, read
// transposed.
//
// A workgroup of four waves takes `RG` groups of 32 rows; the waves that are
// left over divide the tokens of a step (TG token groups of 32), each with a
// softmax of its own, joined through LDS at the end.  (fp32: DS = 2 waves
// share the dimensions of O, which with q would not fit the registers.)
//
// Work is divided by tokens, not by requests: `workers` workgroups take equal
// runs of the steps of all requests laid end to end, so that one long request
// fills the card and ragged batches leave none of it idle.  A run that starts
// or ends inside a request leaves its sums (O, maximum, sum, all fp32) in the
// workspace, and a second kernel joins them.
//
// Rounding: S, the statistics and O are fp32 throughout; probabilities are
// rounded to bf16 for the second product with bf16 caches (2^-9 of a weight
// each, as the values themselves are).
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr int kTile = 32;          // tokens of a wave's step
constexpr int kTab = 512;          // block table entries kept in LDS
constexpr int kThreads = 256;
constexpr float kLog2e = 1.44269504088896340736f;
// A run's piece of a request that another workgroup continues.
struct Piece {
  int32_t b, row_tile, last, pad;   // b < 0: none
};

// One request of the batch.
struct Request {
  int bos, q, row;      // row < 0: outside the tables
  int c, n;             // computed tokens; keys, at most the table's
};

__device__ __forceinline__ Request load_request(const PagedParams& p, int T,
                                                int b) {
  Request r;
  r.bos = min(max(p.qsl[b], 0), T);
  r.q = min(max(p.qsl[b + 1], r.bos), T) - r.bos;
  const int row = p.req_idx ? p.req_idx[b] : b;
  r.row = row >= 0 && row < p.rows ? row : -1;
  r.c = r.row >= 0 ? max(p.computed[r.row], 0) : 0;
  // (a step's tokens behind the last one are counted in 31 bits, too)
  const int64_t most = min(int64_t(p.width) * p.block,
                           int64_t(0x7fffffff - 1024));
  r.n = r.row >= 0 ? int(min(int64_t(r.c) + r.q, most)) : 0;
  return r;
}

template <bool BF16, int R, int P, int RG>
struct Shape {
  static constexpr int ES = BF16 ? 2 : 4;
  // waves that share the values' dimensions: q and O have to fit a wave's
  // registers (each of them forms the same scores)
  static constexpr int DS = R == 512 ? (BF16 ? 2 : 4) : R == 256 && !BF16 ? 2 : 1;
  static constexpr int TG = 4 / (RG * DS);     // token groups
  static constexpr int SHARE = RG * DS;        // waves that share a tile
  static constexpr int CH = R * ES / 16;       // chunks of a latent
  static constexpr int CHP = P * ES / 16;      // and of a rope key
  static constexpr int KF = (R + P) * ES / 32; // operands of a row
  static constexpr int NB = R / 32 / DS;       // blocks of O of a wave
  static constexpr int TILE = kTile * (CH + CHP) * 16;
  static constexpr int NBUF = 147456 / TILE / TG > 4 ? 4 : 147456 / TILE / TG;
  static constexpr int ROPE = kTile * CH * 16; // the rope part of a tile
  static constexpr int LOADS = kTile * (CH + CHP) / 64;
  static constexpr int MINE = LOADS / SHARE;   // loads of a wave
  static constexpr int ROWS = 32 * RG;
  static constexpr int STEP = kTile * TG;      // tokens of a step
  static constexpr int BUFS = TG * NBUF * TILE;
  static constexpr int LDS = BUFS + kTab * 4;
  static_assert(kTile * CH / 64 % SHARE == 0 && kTile * CHP / 64 % SHARE == 0 &&
                    TG >= 1 && NBUF >= 1,
                "shape");
};

__device__ __forceinline__ int steps_of(const Request& r, int H, int rows,
                                            int step, int* tiles) {
  *tiles = int((int64_t(r.q) * H + rows - 1) / rows);
  return max((r.n + step - 1) / step, 1);
}

template <bool BF16, int R, int P, int RG>
__global__ void __launch_bounds__(kThreads, 1)
    kda_latent_attention_kernel(LatentParams p) {
  using Z = Shape<BF16, R, P, RG>;
  extern __shared__ __align__(16) char smem[];
  int32_t* tab = reinterpret_cast<int32_t*>(smem + Z::BUFS);
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  const int tg = wave / Z::SHARE, share = wave % Z::SHARE;
  const int ds = share % Z::DS, rg = share / Z::DS;
  const PagedParams& c = p.c;
  const int W = p.workers, w = blockIdx.x;

  // -- this workgroup's run: steps [first, last) of all requests ------------
  Piece* plan = reinterpret_cast<Piece*>(p.work);
  __shared__ int64_t red[4];
  __shared__ int32_t found_b;
  __shared__ int64_t found_at;
  int64_t total = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    const int b = b0 + tid;
    int64_t v = 0;
    if (b < c.B) {
      const Request r = load_request(c, p.T, b);
      int tiles;
      const int steps = steps_of(r, p.H, Z::ROWS, Z::STEP, &tiles);
      v = int64_t(steps) * tiles;
    }
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    if (lane == 0) red[wave] = v;
    __syncthreads();
    total += red[0] + red[1] + red[2] + red[3];
    __syncthreads();
  }
  const int64_t per = max((total + W - 1) / W, int64_t(1));
  const int64_t first = w * per, last = min(first + per, total);
  if (tid == 0) plan[w].b = -1;
  if (first >= last) return;
  int64_t done = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    const int b = b0 + tid;
    int64_t v = 0;
    if (b < c.B) {
      const Request r = load_request(c, p.T, b);
      int tiles;
      const int steps = steps_of(r, p.H, Z::ROWS, Z::STEP, &tiles);
      v = int64_t(steps) * tiles;
    }
    int64_t upto = v;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    if (lane == 63) red[wave] = upto;
    __syncthreads();
    int64_t before = done;
    for (int k = 0; k < wave; ++k) before += red[k];
    const int64_t at = before + upto - v;
    if (v > 0 && at <= first && first < at + v) {
      found_b = b;
      found_at = at;
    }
    done += red[0] + red[1] + red[2] + red[3];
    __syncthreads();
    if (done > first) break;
  }
  int b = uniform(found_b);
  const int64_t item0 = found_at;      // the request's first step
  Request r = load_request(c, p.T, b);
  int tiles;
  int steps = steps_of(r, p.H, Z::ROWS, Z::STEP, &tiles);
  int rt = int((first - item0) / steps);
  // the run: from step s0 of row tile rt of request b, `left` steps
  int s0 = int(first - item0 - int64_t(rt) * steps);
  int64_t left = last - first;

#pragma unroll 1
  while (true) {
    // -- one piece: steps [s0, s1) of row tile rt of request b ----------------
    const int s1 = int(min(int64_t(steps), s0 + left));
    const int rows = r.q * p.H;
    const int last_tok = min((rt + 1) * Z::ROWS, rows) - 1;
    // keys of the row tile, and of this lane's query
    const int n = int(min(int64_t(r.c) + last_tok / p.H + 1, int64_t(r.n)));
    int lim;
    u4 q[Z::KF];
    {
      const int mine = min(rt * Z::ROWS + rg * 32 + (lane & 31), rows - 1);
      const int tok = mine / p.H, head = mine - tok * p.H;
      lim = int(min(int64_t(r.c) + tok + 1, int64_t(r.n)));
      const char* src = p.q + int64_t(r.bos + tok) * p.s_q_tok +
                        head * p.s_q_head + half * 16;
#pragma unroll
      for (int k = 0; k < Z::KF; ++k)
        q[k] = *reinterpret_cast<const u4*>(src + 32 * k);
    }
    f16v o[Z::NB];
#pragma unroll
    for (int k = 0; k < Z::NB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[k][i] = 0.0f;
    float top = -INFINITY, sum = 0.0f;

    int tab0 = -1;                      // first table entry in LDS
    const int32_t* table = c.table + int64_t(max(r.row, 0)) * c.s_tab_row;
    // A step's tokens: where they are, for the lanes 0..31 of token group tg.
    uint32_t live[Z::NBUF];
    auto stage = [&](int step, int buf) -> uint32_t {
      const int e_lo = step * Z::STEP / c.block;
      const int e_hi = (step * Z::STEP + Z::STEP - 1) / c.block;
      if (tab0 < 0 || e_lo < tab0 || e_hi >= tab0 + kTab) {
        __syncthreads();
        tab0 = e_lo;
        for (int i = tid; i < kTab; i += kThreads)
          tab[i] = int64_t(tab0) + i < c.width && r.row >= 0
                       ? table[int64_t(tab0 + i) * c.s_tab_col]
                       : c.null_id;
        __syncthreads();
      }
      const int t0 = step * Z::STEP + tg * kTile;
      if (t0 >= n) return 0u;
      const int pos = t0 + (lane & 31);
      const int e = pos / c.block;
      const int id = tab[e - tab0];
      const bool ok = pos < n && id > c.null_id && id < c.N;
      const char* addr = ok ? c.cache + id * c.s_blk +
                                  (pos - e * c.block) * c.s_tok
                            : kZeros;
      const uint64_t a = reinterpret_cast<uint64_t>(addr);
      const uint32_t lo = uint32_t(a), hi = uint32_t(a >> 32);
      const uint32_t lds =
          uniform(lds_addr(smem) + (tg * Z::NBUF + buf) * Z::TILE);
      const int l = fresh_tid() & 63;
#pragma unroll
      for (int j = 0; j < Z::MINE; ++j) {
        const int i = uniform(j * Z::SHARE + share);   // of 64 chunks each
        // (the latents' loads come first, for each wave)
        if (j < Z::MINE * Z::CH / (Z::CH + Z::CHP)) {
          if constexpr (Z::CH >= 64) {             // part of one row
            const int rw = i * 64 / Z::CH;
            const uint64_t base =
                (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(hi), rw)))
                 << 32) |
                uint32_t(__builtin_amdgcn_readlane(int(lo), rw));
            load_lds(base,
                     uint32_t(((i * 64 % Z::CH + l) ^ swizzle<Z::CH>(rw)) *
                              16),
                     lds + i * 1024);
          } else {                                 // a few rows
            const int rw = i * (64 / Z::CH) + l / Z::CH;
            const uint32_t alo = __shfl(int(lo), rw),
                           ahi = __shfl(int(hi), rw);
            load_lds(reinterpret_cast<const char*>(
                         (uint64_t(ahi) << 32) | alo) +
                         ((l % Z::CH) ^ swizzle<Z::CH>(rw)) * 16,
                     lds + i * 1024);
          }
        } else if constexpr (Z::CHP > 0) {
          const int rw = (i - kTile * Z::CH / 64) * (64 / Z::CHP) +
                         l / Z::CHP;
          const uint32_t alo = __shfl(int(lo), rw), ahi = __shfl(int(hi), rw);
          load_lds(reinterpret_cast<const char*>((uint64_t(ahi) << 32) | alo) +
                       (Z::CH + ((l % Z::CHP) ^ swizzle<Z::CHP>(rw))) * 16,
                   lds + i * 1024);
        }
      }
      return uint32_t(__ballot(ok));
    };

    // live[k]: which tokens of the step k ahead are there
#pragma unroll
    for (int k = 0; k < Z::NBUF - 1; ++k)
      live[k] = s0 + k < s1 ? stage(s0 + k, k) : 0u;
    int buf = 0;
    // steps of the run in which this token group has tokens
    const int mine = min(s1, (n - tg * kTile + Z::STEP - 1) / Z::STEP);
#pragma unroll 1
    for (int s = s0; s < s1; ++s) {
      constexpr int kAhead = Z::NBUF - 1;
      // the buffer that the last step has read takes the next loads
      if (Z::SHARE > 1) lds_barrier();
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      const int nb = buf == 0 ? kAhead : buf - 1;
      live[kAhead] = s + kAhead < s1 ? stage(s + kAhead, nb) : 0u;
      wait_tile<kAhead>(mine - s, std::integral_constant<int, Z::MINE>());
      if (Z::SHARE > 1) lds_barrier();
      const int t0 = s * Z::STEP + tg * kTile;
      const char* tile = smem + (tg * Z::NBUF + buf) * Z::TILE;
      if (t0 < n)
        attend<BF16, Z::CH, Z::CHP, Z::CH>(tile, tile + Z::ROPE, tile,
                                           ds * Z::NB, q, o, top, sum,
                                           live[0], min(lim - t0, kTile),
                                           p.scale);
#pragma unroll
      for (int k = 0; k < kAhead; ++k) live[k] = live[k + 1];
      buf = buf + 1 == Z::NBUF ? 0 : buf + 1;
    }
    sum = halves_sum(sum);

    // -- the token groups' sums joined: the first of them ends with them ----
    if constexpr (Z::TG > 1) {
      float* box = reinterpret_cast<float*>(smem);
      constexpr int kBlocks = 8;           // blocks of O that move at a time
      static_assert(Z::TG * Z::SHARE * 64 * 2 * 4 <= Z::BUFS, "statistics");
      __syncthreads();
      box[(wave * 64 + lane) * 2] = top;
      box[(wave * 64 + lane) * 2 + 1] = sum;
      __syncthreads();
      float to = top;
#pragma unroll
      for (int g = 0; g < Z::TG; ++g)
        to = fmaxf(to, box[((g * Z::SHARE + share) * 64 + lane) * 2]);
      float all = 0.0f;
#pragma unroll
      for (int g = 0; g < Z::TG; ++g) {
        const float* e = box + ((g * Z::SHARE + share) * 64 + lane) * 2;
        all += e[0] == -INFINITY ? 0.0f : exp2f(e[0] - to) * e[1];
      }
      const float by = top == -INFINITY ? 0.0f : exp2f(top - to);
      top = to;
      sum = all;
#pragma unroll
      for (int k = 0; k < Z::NB; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[k][i] *= by;
#pragma unroll
      for (int k0 = 0; k0 < Z::NB; k0 += kBlocks)
#pragma unroll
        for (int g = 1; g < Z::TG; ++g) {
          __syncthreads();
          if (tg == g)
#pragma unroll
            for (int k = k0; k < k0 + kBlocks && k < Z::NB; ++k)
#pragma unroll
              for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<f4*>(
                    box + (((share * kBlocks + k - k0) * 4 + i / 4) * 64 +
                           lane) * 4) =
                    f4{o[k][i], o[k][i + 1], o[k][i + 2], o[k][i + 3]};
          __syncthreads();
          if (tg == 0)
#pragma unroll
            for (int k = k0; k < k0 + kBlocks && k < Z::NB; ++k)
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const f4 v = *reinterpret_cast<const f4*>(
                    box + (((share * kBlocks + k - k0) * 4 + i / 4) * 64 +
                           lane) * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[k][i + e] += v[e];
              }
        }
    }

    // -- the whole of it: outputs; a piece: to the workspace ------------------
    const bool whole = s0 == 0 && s1 == steps;
    // (positions anew: kept across the loop they would cost it registers)
    const int lane = fresh_tid() & 63, half = lane >> 5;
    const int row = rt * Z::ROWS + rg * 32 + (lane & 31);
    const int tok = row / p.H, head = row - tok * p.H;
    if (tg == 0) {
      if (whole) {
        if (row < rows) {
          const float by = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
          char* dst = p.out + int64_t(r.bos + tok) * p.s_out_tok +
                      head * p.s_out_head;
#pragma unroll
          for (int k = 0; k < Z::NB; ++k)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const int e = 32 * (ds * Z::NB + k) + acc_row(i, half);
              if constexpr (BF16)
                *reinterpret_cast<u2*>(dst + e * 2) =
                    u2{pack_bf16(o[k][i] * by, o[k][i + 1] * by),
                       pack_bf16(o[k][i + 2] * by, o[k][i + 3] * by)};
              else
                *reinterpret_cast<f4*>(dst + e * 4) =
                    f4{o[k][i] * by, o[k][i + 1] * by, o[k][i + 2] * by,
                       o[k][i + 3] * by};
            }
          if (p.lse && half == 0 && ds == 0)
            p.lse[int64_t(r.bos + tok) * p.s_lse_tok + head * p.s_lse_head] =
                sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
        }
      } else {
        const int slot = s0 == 0 ? 2 * w + 1 : 2 * w;
        float* ml = reinterpret_cast<float*>(p.work + W * sizeof(Piece)) +
                    int64_t(slot) * Z::ROWS * 2;
        float* to = reinterpret_cast<float*>(
                        p.work + W * sizeof(Piece) +
                        int64_t(2) * W * Z::ROWS * 8) +
                    (int64_t(slot) * RG + rg) * 32 * R;
        if (half == 0 && ds == 0) {
          ml[(rg * 32 + lane) * 2] = top;
          ml[(rg * 32 + lane) * 2 + 1] = sum;
        }
#pragma unroll
        for (int k = 0; k < Z::NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f4*>(
                to + (((ds * Z::NB + k) * 4 + i / 4) * 64 + lane) * 4) =
                f4{o[k][i], o[k][i + 1], o[k][i + 2], o[k][i + 3]};
        if (s0 == 0 && tid == 0)
          plan[w] = Piece{b, rt, w + int((steps - left + per - 1) / per), 0};
      }
    }
    left -= s1 - s0;
    if (left <= 0) return;
    __syncthreads();                       // LDS is free for the next piece
    s0 = 0;
    if (++rt == tiles) {
      rt = 0;
      do {
        r = load_request(c, p.T, ++b);
      } while (r.q == 0);
      steps = steps_of(r, p.H, Z::ROWS, Z::STEP, &tiles);
    }
  }
}

// Joins the pieces of row tiles that several workgroups shared: a wave takes
// four registers' worth of one 32-row group at a time, in the order in which
// the lanes of the first kernel had them.
template <bool BF16, int R, int RG>
__global__ void __launch_bounds__(kThreads)
    kda_latent_join_kernel(LatentParams p) {
  constexpr int kUnits = R / 8;            // of 4 values for each lane
  const int w = blockIdx.x, rg = blockIdx.z, W = p.workers;
  const Piece piece = reinterpret_cast<const Piece*>(p.work)[w];
  if (piece.b < 0) return;
  const int lane = threadIdx.x & 63, half = lane >> 5;
  const float* ml = reinterpret_cast<const float*>(p.work +
                                                   W * sizeof(Piece));
  const float* parts = ml + int64_t(2) * W * 32 * RG * 2;
  const Request r = load_request(p.c, p.T, piece.b);
  const int row = piece.row_tile * 32 * RG + rg * 32 + (lane & 31);
  const int count = piece.last - w + 1;
  auto slot = [&](int i) { return i == 0 ? 2 * w + 1 : 2 * (w + i); };
  float top = -INFINITY;
  for (int i = 0; i < count; ++i)
    top = fmaxf(top, ml[(int64_t(slot(i)) * 32 * RG + rg * 32 +
                         (lane & 31)) * 2]);
  const int u = blockIdx.y * (kThreads / 64) + (threadIdx.x >> 6);
  float sum = 0.0f;
  f4 acc = {0, 0, 0, 0};
  for (int i = 0; i < count; ++i) {
    const float* e =
        ml + (int64_t(slot(i)) * 32 * RG + rg * 32 + (lane & 31)) * 2;
    const float by = e[0] == -INFINITY ? 0.0f : exp2f(e[0] - top);
    sum += by * e[1];
    const f4 v = *reinterpret_cast<const f4*>(
        parts + (int64_t(slot(i)) * RG + rg) * 32 * R + (u * 64 + lane) * 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc[k] += by * v[k];
  }
  if (row >= r.q * p.H || u >= kUnits) return;
  const int tok = row / p.H, head = row - tok * p.H;
  const float by = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
  const int at = 32 * (u / 4) + acc_row(u % 4 * 4, half);
  char* dst = p.out + int64_t(r.bos + tok) * p.s_out_tok +
              head * p.s_out_head;
  if constexpr (BF16)
    *reinterpret_cast<u2*>(dst + at * 2) =
        u2{pack_bf16(acc[0] * by, acc[1] * by),
           pack_bf16(acc[2] * by, acc[3] * by)};
  else
    *reinterpret_cast<f4*>(dst + at * 4) =
        f4{acc[0] * by, acc[1] * by, acc[2] * by, acc[3] * by};
  if (p.lse && half == 0 && u == 0)
    p.lse[int64_t(r.bos + tok) * p.s_lse_tok + head * p.s_lse_head] =
        sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

template <bool BF16, int R, int P, int RG>
int launch(const LatentParams& p, hipStream_t stream) {
  using Z = Shape<BF16, R, P, RG>;
  static_assert(Z::LDS + 64 <= 160 * 1024, "LDS");
  const hipError_t e = hipFuncSetAttribute(
      reinterpret_cast<const void*>(
          &kda_latent_attention_kernel<BF16, R, P, RG>),
      hipFuncAttributeMaxDynamicSharedMemorySize, Z::LDS);
  if (e != hipSuccess) return int(e);
  launch_kernel(kda_latent_attention_kernel<BF16, R, P, RG>, dim3(p.workers),
                dim3(kThreads), Z::LDS, stream, p);
  launch_kernel(kda_latent_join_kernel<BF16, R, RG>,
                dim3(p.workers, R / 32, RG), dim3(kThreads), 0, stream, p);
  return int(hipGetLastError());
}

template <bool BF16, int R, int P>
int launch_groups(const LatentParams& p, hipStream_t stream) {
  if (p.group == 1) return launch<BF16, R, P, 1>(p, stream);
  if constexpr (BF16 || R < 512)
    if (p.group == 2) return launch<BF16, R, P, 2>(p, stream);
  return int(hipErrorInvalidValue);
}

template <bool BF16>
int launch_dims(const LatentParams& p, int R, int P, hipStream_t stream) {
  if (R == 512 && P == 64) return launch_groups<BF16, 512, 64>(p, stream);
  if (R == 512 && P == 0) return launch_groups<BF16, 512, 0>(p, stream);
  if (R == 256 && P == 64) return launch_groups<BF16, 256, 64>(p, stream);
  if (R == 256 && P == 0) return launch_groups<BF16, 256, 0>(p, stream);
  if (R == 128 && P == 64) return launch_groups<BF16, 128, 64>(p, stream);
  if (R == 128 && P == 0) return launch_groups<BF16, 128, 0>(p, stream);
  return int(hipErrorInvalidValue);
}

// One 16-byte chunk a thread, a token's chunks side by side.
__global__ void __launch_bounds__(256)
    kda_latent_write_kernel(LatentWriteParams p) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = i / p.chunks;
  if (t >= p.T) return;
  const int ch = int(i - t * p.chunks);
  const int64_t slot = p.slots[t];
  if (slot < p.first_slot || slot >= p.total_slots) return;
  const int64_t blk = slot / p.block;
  const char* src = ch < p.lat_chunks
                        ? p.latent + t * p.s_lat + ch * 16
                        : p.rope + t * p.s_rope + (ch - p.lat_chunks) * 16;
  *reinterpret_cast<u4*>(p.cache + blk * p.s_blk +
                         (slot - blk * p.block) * p.s_tok + ch * 16) =
      *reinterpret_cast<const u4*>(src);
}

}  // namespace

int latent_groups(int64_t T, int64_t B, int64_t H, int R,
                  bool bf16) {
  // as many rows as an average request has, so that its tokens are read once
  const int64_t rows = B > 0 ? (T + B - 1) / B * H : H;
  if (rows <= 32) return 1;
  return R == 512 && !bf16 ? 1 : 2;
}

int64_t latent_work_bytes(int group, int R) {
  return int64_t(kLatentWorkers) *
         (sizeof(Piece) + 2 * 32 * group * (8 + int64_t(R) * 4));
}

int launch_latent(const LatentParams& p, int R, int P, bool bf16,
                  hipStream_t stream) {
  return bf16 ? launch_dims<true>(p, R, P, stream)
              : launch_dims<false>(p, R, P, stream);
}

int launch_latent_write(const LatentWriteParams& p, hipStream_t stream) {
  const int64_t n = int64_t(p.T) * p.chunks;
  launch_kernel(kda_latent_write_kernel, dim3(uint32_t((n + 255) / 256)),
                dim3(256), 0, stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
