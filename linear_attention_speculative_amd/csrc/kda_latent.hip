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
// A workgroup takes RG groups of 32 rows (1 or 2) and 32 tokens a step, with
// DS = 4 waves to each group: one with all of q and O has no registers left.
// Each sums a quarter of the R + P products of all scores, gets the others'
// parts of the scores of 8 tokens through LDS, takes their weights, gives
// those to the others, and sums a quarter of the dimensions of O.
//
// Work is divided by tokens, not by requests: `workers` workgroups take equal
// runs of the steps of all requests laid end to end, so that one long request
// fills the card and ragged batches leave none of it idle.  A run that starts
// or ends inside a request leaves its sums (O, maximum, sum, all fp32) in the
// workspace, and a second kernel joins them.
//
// Rounding: S, the statistics and O are fp32 throughout; with bf16 caches the
// probabilities go into the second product as two bf16 values, which leaves
// 2^-15 of a weight at most (split_bf16() in kda_mma.hpp).
//
// What bounds it (R = 512, P = 64, 32 heads, bf16): for 256 single tokens
// behind 3000 others on average, the cache's bytes and a step's chain: 216 us,
// 884 MB at 4.1 TB/s, of which the loop's steps run at 4.6 (2.0 us each; 1.9
// with one bf16 value a weight), and some 6 us a piece go to its queries, its
// first tile and its outputs.  For 48 windows of up to 4 drafts behind 1500
// tokens, two row tiles a request: 51 us, a chain of scores, exchange, weights
// and sums of 2.5 us a step with one workgroup of eight waves on a CU; the
// matrix cores are busy for a fifth of it, and the cache is read once for each
// row tile.  The join takes 11 us of the first, 13 us of the second (37 MB of
// pieces), 5 us of one request.  fp32 holds one or two tiles in LDS: 64 tokens
// behind 3000 take 254 us a call, the 48 windows 203.
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr int kTile = 32;          // tokens of a step
constexpr int kTab = 512;          // block table entries kept in LDS
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

// Block of a position (below 2^31) in its request: position / block.
__device__ __forceinline__ int block_of(const PagedParams& p, int pos) {
  return int((uint64_t(uint32_t(pos)) * p.magic) >> p.shift);
}

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
  static constexpr int DS = 4;                 // waves of a row group
  static constexpr int WAVES = RG * DS, THREADS = 64 * WAVES;
  static constexpr int CH = R * ES / 16;       // chunks of a latent
  static constexpr int CHP = P * ES / 16;      // and of a rope key
  static constexpr int KL = CH / 2 / DS, KP = CHP / 2 / DS;  // operands of a
  static constexpr int KF = KL + KP;                         // row, a wave's
  static constexpr int NB = R / 32 / DS;       // blocks of O of a wave
  static constexpr int TILE = kTile * (CH + CHP) * 16;
  static constexpr int ROPE = kTile * CH * 16; // the rope part of a tile
  static constexpr int LL = kTile * CH / 64, LP = kTile * CHP / 64;  // loads
  static constexpr int NL = LL / WAVES;        // of a wave
  static constexpr int NP = (LP + WAVES - 1) / WAVES;
  static constexpr int MINE = NL + NP;
  static constexpr int ROWS = 32 * RG;
  // what a wave gets of the others: three parts of its scores; then its own
  // weights, maxima and, at the end, sums, for the others
  static constexpr int BOX = 3 * 1024;
  static constexpr int EXCH = WAVES * BOX;
  static constexpr int REST = EXCH + kTab * 4;
  static constexpr int FIT = (160 * 1024 - 256 - REST) / TILE;
  static constexpr int NBUF = FIT > 4 ? 4 : FIT;
  static constexpr int LDS = NBUF * TILE + REST;
  static_assert(LL % WAVES == 0 && NBUF >= 1, "shape");
};

// Row tiles of a request, and steps of each.  A row tile counts kStart steps
// more when work is divided: what its queries, its first loads and its outputs
// take (without them, 48 windows of draft tokens with short requests among them
// took 63 us, the mean workgroup 41).
constexpr int kStart = 4;
__device__ __forceinline__ int steps_of(const Request& r, int H, int rows,
                                        int* tiles) {
  *tiles = int((int64_t(r.q) * H + rows - 1) / rows);
  return max((r.n + kTile - 1) / kTile, 1);
}

template <bool BF16, int R, int P, int RG>
__global__ void __launch_bounds__(256 * RG, RG)
    kda_latent_attention_kernel(LatentParams p) {
  using Z = Shape<BF16, R, P, RG>;
  constexpr int kThreads = Z::THREADS;
  extern __shared__ __align__(16) char smem[];
  char* exch = smem + Z::NBUF * Z::TILE;
  int32_t* tab = reinterpret_cast<int32_t*>(exch + Z::EXCH);
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  const int ds = wave % Z::DS, rg = wave / Z::DS;
  const PagedParams& c = p.c;
  const int W = p.workers, w = blockIdx.x;

  // -- this workgroup's run: steps [first, last) of all requests ------------
  Piece* plan = reinterpret_cast<Piece*>(p.work);
  __shared__ int64_t red[Z::WAVES];
  __shared__ int32_t found_b;
  __shared__ int64_t found_at;
  __shared__ int32_t flag[Z::WAVES];
  auto steps_at = [&](int b) -> int64_t {
    if (b >= c.B) return 0;
    const Request r = load_request(c, p.T, b);
    int tiles;
    const int steps = steps_of(r, p.H, Z::ROWS, &tiles);
    return int64_t(steps + kStart) * tiles;
  };
  auto wave_sums = [&](int64_t v) {            // of all waves, in order
    if (lane == 63) red[wave] = v;
    __syncthreads();
    int64_t all = 0;
    for (int k = 0; k < Z::WAVES; ++k) all += red[k];
    return all;
  };
  int64_t total = 0;
  const int64_t mine0 = steps_at(tid);         // (of most batches, all)
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    int64_t v = b0 == 0 ? mine0 : steps_at(b0 + tid);
#pragma unroll
    for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
    total += wave_sums(v);
    __syncthreads();
  }
  const int64_t per = max((total + W - 1) / W, int64_t(1));
  const int64_t first = w * per, last = min(first + per, total);
  if (tid == 0) plan[w].b = -1;
  if (first >= last) return;
  int64_t done = 0;
  for (int b0 = 0; b0 < c.B; b0 += kThreads) {
    const int64_t v = b0 == 0 ? mine0 : steps_at(b0 + tid);
    int64_t upto = v;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
      const int64_t o = __shfl_up(upto, s);
      if (lane >= s) upto += o;
    }
    const int64_t all = wave_sums(upto);
    int64_t at = done + upto - v;
    for (int k = 0; k < wave; ++k) at += red[k];
    if (v > 0 && at <= first && first < at + v) {
      found_b = b0 + tid;
      found_at = at;
    }
    done += all;
    __syncthreads();
    if (done > first) break;
  }
  int b = uniform(found_b);
  const int64_t item0 = found_at;      // the request's first step
  Request r = load_request(c, p.T, b);
  int tiles;
  int steps = steps_of(r, p.H, Z::ROWS, &tiles);
  int rt = int((first - item0) / (steps + kStart));
  // the run: from unit u0 of row tile rt of request b, `left` units, of which
  // the first kStart of a tile are no steps
  int u0 = int(first - item0 - int64_t(rt) * (steps + kStart));
  int64_t left = last - first;

#pragma unroll 1
  while (true) {
    // -- one piece: steps [s0, s1) of row tile rt of request b ----------------
    const int s0 = max(u0 - kStart, 0);
    const int s1 = int(min(int64_t(steps), u0 + left - kStart));
    if (s1 <= s0) return;               // (the next workgroup starts it)
    const int rows = r.q * p.H;
    const int last_tok = min((rt + 1) * Z::ROWS, rows) - 1;
    // keys of the row tile, and of this lane's query; steps that have any
    const int n = int(min(int64_t(r.c) + last_tok / p.H + 1, int64_t(r.n)));
    const int mine = min(rt * Z::ROWS + rg * 32 + (lane & 31), rows - 1);
    const int lim = int(min(int64_t(r.c) + mine / p.H + 1, int64_t(r.n)));
    const int end = min(s1, (n + kTile - 1) / kTile);
    f16v o[Z::NB];
#pragma unroll
    for (int k = 0; k < Z::NB; ++k)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[k][i] = 0.0f;
    float top = -INFINITY, sum = 0.0f;

    int tab0 = -1;                      // first table entry in LDS
    const int32_t* table = c.table + int64_t(max(r.row, 0)) * c.s_tab_row;
    // Loads a step's tile; returns which of its tokens are there.
    auto stage = [&](int step, int buf) -> uint32_t {
      const int e_hi = block_of(c, step * kTile + kTile - 1);
      if (tab0 < 0 || e_hi >= tab0 + kTab) {
        __syncthreads();
        tab0 = block_of(c, step * kTile);
        for (int i = tid; i < kTab; i += kThreads)
          tab[i] = int64_t(tab0) + i < c.width && r.row >= 0
                       ? table[int64_t(tab0 + i) * c.s_tab_col]
                       : c.null_id;
        __syncthreads();
      }
      // lanes l and l + 32: token l
      const int pos = step * kTile + (lane & 31);
      const int e = block_of(c, pos);
      const int id = tab[e - tab0];
      const bool ok = pos < n && id > c.null_id && id < c.N;
      const char* addr = ok ? c.cache + id * c.s_blk +
                                  (pos - e * c.block) * c.s_tok
                            : kZeros;
      const uint64_t a = reinterpret_cast<uint64_t>(addr);
      const uint32_t lo = uint32_t(a), hi = uint32_t(a >> 32);
      const uint32_t lds = uniform(lds_addr(smem) + buf * Z::TILE);
      const int l = fresh_tid() & 63;
#pragma unroll
      for (int j = 0; j < Z::NL; ++j) {
        const int i = uniform(j * Z::WAVES + wave);    // of 64 chunks each
        if constexpr (Z::CH >= 64) {                 // part of one row
          const int rw = i * 64 / Z::CH;
          const uint64_t base =
              (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(hi), rw)))
               << 32) |
              uint32_t(__builtin_amdgcn_readlane(int(lo), rw));
          load_lds(base,
                   uint32_t(((i * 64 % Z::CH + l) ^ swizzle<Z::CH>(rw)) * 16),
                   lds + i * 1024);
        } else {                                     // a few rows
          const int rw = i * (64 / Z::CH) + l / Z::CH;
          const uint32_t alo = __shfl(int(lo), rw), ahi = __shfl(int(hi), rw);
          load_lds(reinterpret_cast<const char*>((uint64_t(ahi) << 32) | alo) +
                       ((l % Z::CH) ^ swizzle<Z::CH>(rw)) * 16,
                   lds + i * 1024);
        }
      }
      if constexpr (Z::CHP > 0) {
#pragma unroll
        for (int j = 0; j < Z::NP; ++j) {
          // (with fewer loads than waves some are made twice, which keeps
          // the number of every wave's loads the same)
          const int i = uniform((j * Z::WAVES + wave) % Z::LP);
          const int rw = i * (64 / Z::CHP) + l / Z::CHP;
          const uint32_t alo = __shfl(int(lo), rw), ahi = __shfl(int(hi), rw);
          load_lds(reinterpret_cast<const char*>((uint64_t(ahi) << 32) | alo) +
                       (Z::CH + ((l % Z::CHP) ^ swizzle<Z::CHP>(rw))) * 16,
                   lds + Z::ROPE + i * 1024);
        }
      }
      return uint32_t(__ballot(ok));
    };

    constexpr int kAhead = Z::NBUF - 1;
    uint32_t live[Z::NBUF];             // live[k]: of the step k ahead
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
      live[k] = s0 + k < end ? stage(s0 + k, k) : 0u;
    // The queries, after the first tiles' loads and waited for here: a wait
    // in the loop would wait for the tiles under way, too.
    u4 q[Z::KF];
    {
      const int tok = mine / p.H, head = mine - tok * p.H;
      const char* src = p.q + int64_t(r.bos + tok) * p.s_q_tok +
                        head * p.s_q_head + (2 * ds + half) * 16;
#pragma unroll
      for (int k = 0; k < Z::KF; ++k)
        q[k] = negated<BF16>(
            *reinterpret_cast<const u4*>(src + 32 * Z::DS * k), p.negate);
#pragma unroll
      for (int k = 0; k < Z::KF; ++k) asm volatile("" : "+v"(q[k]));
    }
    int buf = 0;
#pragma unroll 1
    for (int s = s0; s < end; ++s) {
      if constexpr (kAhead == 0) {
        lds_barrier();                  // the last step's tile is read
        live[0] = stage(s, 0);
        wait_vm<0>();
        lds_barrier();
      } else {
        wait_tile<kAhead - 1>(end - s,
                              std::integral_constant<int, Z::MINE>());
        lds_barrier();                  // and the last step's tile is read
        live[kAhead] = s + kAhead < end ? stage(s + kAhead, buf ? buf - 1
                                                                : kAhead)
                                        : 0u;
      }
      const uint32_t tile = uniform(lds_addr(smem) + buf * Z::TILE);
      const int l = fresh_tid() & 63;
      const f4* box = reinterpret_cast<const f4*>(exch + wave * Z::BOX) + l;
      // this wave's part of the scores; the others' registers to them
      f4 own;
      {
        const RowReader<Z::CH, Z::DS> latents(tile, l, ds);
        const RowReader<(Z::CHP > 0 ? Z::CHP : 8), Z::DS> ropes(
            tile + Z::ROPE, l, ds);
        const f16v part = score<BF16>(
            [&](int k) { return k < Z::KL ? latents(k) : ropes(k - Z::KL); },
            q);
#pragma unroll
        for (int d = 0; d < Z::DS; ++d) {
          const f4 v = {part[4 * d], part[4 * d + 1], part[4 * d + 2],
                        part[4 * d + 3]};
          if (d == ds)
            own = v;
          else
            reinterpret_cast<f4*>(exch + (rg * Z::DS + d) * Z::BOX)
                [(ds > d ? ds - 1 : ds) * 64 + l] = v;
        }
      }
      lds_barrier();
      // scores of its own eight tokens, their maximum and weights
      float x[4], m = -INFINITY;
#pragma unroll
      for (int d = 0; d < 3; ++d) {
        const f4 v = box[d * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) own[e] += v[e];
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int t = 8 * ds + 4 * (l >> 5) + e;
        const bool see = t < lim - s * kTile && ((live[0] >> t) & 1);
        x[e] = see ? own[e] * p.scale : -INFINITY;
        m = fmaxf(m, x[e]);
      }
      m = halves_max(m);
      const bool high = __any(m > top + kSlack);
      auto weights = [&](float (&y)[4]) {
        const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = __builtin_amdgcn_exp2f(x[e] - base);
        char* to = exch + wave * Z::BOX;
        if constexpr (BF16) {
          const u2 a = split_bf16(y[0], y[1]), b = split_bf16(y[2], y[3]);
          reinterpret_cast<u4*>(to)[l] = u4{a[0], b[0], a[1], b[1]};
        } else {
          reinterpret_cast<f4*>(to)[l] = f4{y[0], y[1], y[2], y[3]};
        }
      };
      float y[4];
      weights(y);
      reinterpret_cast<float*>(exch + wave * Z::BOX + 2048)[l] = m;
      if (l == 0) flag[wave] = high;
      lds_barrier();
      int any = 0;
#pragma unroll
      for (int k = 0; k < Z::WAVES; ++k) any |= flag[k];
      if (uniform(any)) {
        // the running maximum moves: weights anew, O and the sum scaled
        float to = top;
#pragma unroll
        for (int d = 0; d < Z::DS; ++d)
          to = fmaxf(to, reinterpret_cast<const float*>(
                             exch + (rg * Z::DS + d) * Z::BOX + 2048)[l]);
        const float by = top == -INFINITY ? 0.0f : exp2f(top - to);
        top = to;
        sum *= by;
#pragma unroll
        for (int k = 0; k < Z::NB; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[k][i] *= by;
        lds_barrier();
        weights(y);
        lds_barrier();
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) sum += y[e];
      // (places behind token n hold zeros, those of null blocks too)
      const int left = lim - s * kTile;
      const bool all_see = __all(left >= min(n - s * kTile, kTile));
      const char* all = exch + rg * Z::DS * Z::BOX;
      if constexpr (BF16) {
        u4 pr[2], lo[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const u4 a = reinterpret_cast<const u4*>(all + 2 * t * Z::BOX)[l];
          const u4 b = reinterpret_cast<const u4*>(all + (2 * t + 1) *
                                                   Z::BOX)[l];
          pr[t] = u4{a[0], a[1], b[0], b[1]};
          lo[t] = u4{a[2], a[3], b[2], b[3]};
        }
        weigh_bf16(ColumnReader<Z::CH>(tile, ds * Z::NB, l), 0, pr, lo,
                   all_see, left, o);
      } else {
        float z[16];
#pragma unroll
        for (int d = 0; d < Z::DS; ++d) {
          const f4 a = reinterpret_cast<const f4*>(all + d * Z::BOX)[l];
#pragma unroll
          for (int e = 0; e < 4; ++e) z[4 * d + e] = a[e];
        }
        weigh_f32<Z::CH>(tile, ds * Z::NB, z, all_see, left, o);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) live[k] = live[k + 1];
      buf = buf + 1 == Z::NBUF ? 0 : buf + 1;
    }
    {
      // the waves' sums over their own tokens, joined
      sum = halves_sum(sum);
      lds_barrier();
      reinterpret_cast<float*>(exch + wave * Z::BOX)[lane] = sum;
      lds_barrier();
      sum = 0.0f;
#pragma unroll
      for (int d = 0; d < Z::DS; ++d)
        sum += reinterpret_cast<const float*>(
            exch + (rg * Z::DS + d) * Z::BOX)[lane];
    }

    // -- the whole of it: outputs; a piece: to the workspace ------------------
    const bool whole = s0 == 0 && s1 == steps;
    // (positions anew: kept across the loop they would cost it registers)
    const int lane = fresh_tid() & 63, half = lane >> 5;
    const int row = rt * Z::ROWS + rg * 32 + (lane & 31);
    const int tok = row / p.H, head = row - tok * p.H;
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
      float* to = reinterpret_cast<float*>(p.work + W * sizeof(Piece) +
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
        plan[w] = Piece{b, rt, w + int((steps - s1 + per - 1) / per), 0};
    }
    left -= s1 + kStart - u0;
    if (left <= 0) return;
    __syncthreads();                       // LDS is free for the next piece
    u0 = 0;
    if (++rt == tiles) {
      rt = 0;
      do {
        r = load_request(c, p.T, ++b);
      } while (r.q == 0);
      steps = steps_of(r, p.H, Z::ROWS, &tiles);
    }
  }
}

// Joins the pieces of row tiles that several workgroups shared: a workgroup
// takes 32 dimensions of a 32-row group, in the order in which the lanes of the
// first kernel had them, its waves every fourth piece.  Of few pieces each wave
// takes all, for 32 dimensions of its own.
constexpr int kJoinWaves = 4;
template <bool BF16, int R, int RG>
__global__ void __launch_bounds__(64 * kJoinWaves)
    kda_latent_join_kernel(LatentParams p) {
  __shared__ float tops[8][32], sums[kJoinWaves][64];
  __shared__ f4 box[kJoinWaves][4][64];
  const int w = blockIdx.x, rg = blockIdx.z, W = p.workers;
  const Piece piece = reinterpret_cast<const Piece*>(p.work)[w];
  if (piece.b < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = uniform(tid >> 6);
  const float* ml = reinterpret_cast<const float*>(p.work +
                                                   W * sizeof(Piece)) +
                    rg * 64;
  const int count = piece.last - w + 1;
  const bool few = count <= 4;
  if (few && blockIdx.y % kJoinWaves != 0) return;
  const int u = few ? blockIdx.y + wave : blockIdx.y;
  const int start = few ? 0 : wave, stride = few ? 1 : kJoinWaves;
  const f4* parts = reinterpret_cast<const f4*>(
                        p.work + W * sizeof(Piece) +
                        int64_t(2) * W * 32 * RG * 8) +
                    rg * (8 * R) + u * 256 + lane;
  auto slot = [&](int i) {
    return int64_t(i == 0 ? 2 * w + 1 : 2 * (w + i));
  };
  // (the first pieces are under way while the maximum is found)
  constexpr int U = 4;
  f4 acc[4], v[U][4];
  f2 e[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t at = slot(min(i0 + k * stride, count - 1)) * RG;
      e[k] = *reinterpret_cast<const f2*>(ml + at * 64 + (lane & 31) * 2);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[k][j] = parts[at * (8 * R) + j * 64];
    }
  };
  // (these, too)
  const int bos = min(max(p.c.qsl[piece.b], 0), p.T);
  const int rows = (min(max(p.c.qsl[piece.b + 1], bos), p.T) - bos) * p.H;
  fetch(start);
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f4{0, 0, 0, 0};
  float top = -INFINITY, sum = 0.0f;
  for (int i = tid >> 5; i < count; i += 8)
    top = fmaxf(top, ml[slot(i) * RG * 64 + (tid & 31) * 2]);
  tops[tid >> 5][tid & 31] = top;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 8; ++k) top = fmaxf(top, tops[k][lane & 31]);
  for (int i0 = start; i0 < count; i0 += U * stride) {
    if (i0 != start) fetch(i0);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i0 + k * stride >= count) break;
      const float by = e[k][0] == -INFINITY ? 0.0f : exp2f(e[k][0] - top);
      sum += by * e[k][1];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int d = 0; d < 4; ++d) acc[j][d] += by * v[k][j][d];
    }
  }
  const int row = piece.row_tile * 32 * RG + rg * 32 + (lane & 31);
  const int tok = row / p.H, head = row - tok * p.H;
  char* dst = p.out + int64_t(bos + tok) * p.s_out_tok + head * p.s_out_head;
  // four dimensions of each half from `at` on
  auto write = [&](const f4& o, int at, float by) {
    if constexpr (BF16)
      *reinterpret_cast<u2*>(dst + at * 2) = u2{
          pack_bf16(o[0] * by, o[1] * by), pack_bf16(o[2] * by, o[3] * by)};
    else
      *reinterpret_cast<f4*>(dst + at * 4) =
          f4{o[0] * by, o[1] * by, o[2] * by, o[3] * by};
  };
  if (!few) {
    sums[wave][lane] = sum;
#pragma unroll
    for (int j = 0; j < 4; ++j) box[wave][j][lane] = acc[j];
    __syncthreads();
    sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kJoinWaves; ++k) sum += sums[k][lane];
  }
  if (row >= rows) return;
  const float by = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
  if (few) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      write(acc[j], 32 * u + acc_row(4 * j, half), by);
  } else {
    f4 o = box[0][wave][lane];
#pragma unroll
    for (int k = 1; k < kJoinWaves; ++k)
#pragma unroll
      for (int d = 0; d < 4; ++d) o[d] += box[k][wave][lane][d];
    write(o, 32 * u + acc_row(4 * wave, half), by);
  }
  if (p.lse && half == 0 && u == 0 && (few || wave == 0))
    p.lse[int64_t(bos + tok) * p.s_lse_tok + head * p.s_lse_head] =
        sum == 0.0f ? -INFINITY : (top + log2f(sum)) / kLog2e;
}

template <bool BF16, int R, int P, int RG>
int launch(const LatentParams& p, hipStream_t stream) {
  using Z = Shape<BF16, R, P, RG>;
  static_assert(Z::LDS + 256 <= 160 * 1024, "LDS");
  const hipError_t e = hipFuncSetAttribute(
      reinterpret_cast<const void*>(
          &kda_latent_attention_kernel<BF16, R, P, RG>),
      hipFuncAttributeMaxDynamicSharedMemorySize, Z::LDS);
  if (e != hipSuccess) return int(e);
  launch_kernel(kda_latent_attention_kernel<BF16, R, P, RG>, dim3(p.workers),
                dim3(Z::THREADS), Z::LDS, stream, p);
  launch_kernel(kda_latent_join_kernel<BF16, R, RG>,
                dim3(p.workers, R / 32, RG), dim3(64 * kJoinWaves), 0, stream,
                p);
  return int(hipGetLastError());
}

template <bool BF16, int R, int P>
int launch_groups(const LatentParams& p, hipStream_t stream) {
  if (p.group == 1) return launch<BF16, R, P, 1>(p, stream);
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

int latent_groups(int64_t T, int64_t B, int64_t H) {
  // as many rows as an average request has, so that its tokens are read once
  const int64_t rows = B > 0 ? (T + B - 1) / B * H : H;
  if (rows <= 32) return 1;
  return 2;
}

int latent_workers(int64_t T, int64_t B, int64_t H, int64_t tokens, int group) {
  // no more than the steps that tables of `tokens` places allow
  const int64_t tiles = T * H / (32 * group) + B;
  const int64_t steps = (tokens + kTile - 1) / kTile + kStart;
  return tiles > kLatentWorkers || steps > kLatentWorkers ||
                 tiles * steps > kLatentWorkers
             ? kLatentWorkers
             : int(tiles * steps);
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
