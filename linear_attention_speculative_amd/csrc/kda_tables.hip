// Index arrays of one serving step on gfx950, from request lengths: token
// offsets, block allocation, state slots, and the position and cache slot of
// every token.
//
// Two exclusive prefix sums over the batch (tokens, new blocks) order
// everything: blocks are handed out in batch order, so no atomic decides who
// gets which, and every run gives the same tables.  The request kernel is one
// workgroup (a step has at most some thousand requests; a second workgroup
// would have to wait for the first one's sums): each thread takes one request
// of a tile, or two of a batch of more, all loads of a kind under way
// together, and reads its lengths before any row is written, so that the held
// counts may be updated in place.  What bounds it is the chain of a few
// dependent loads.  The new blocks are written by all threads, each finding
// the request of a block by binary search: a prompt's many blocks would
// otherwise be a chain in one thread.  The token kernel then has one thread
// per token; a workgroup keeps the token offsets in LDS and each thread finds
// its request by a binary search there.
//
// Request kernel, 7 requests and 2000: 3.4 and 10.6 us (one request a thread
// and its blocks in a loop: 4.1 and 13.1); token kernel 1.9 and 5.8 us.
#include "kda_serving.hpp"

namespace kda {
namespace {

constexpr int kTokThreads = 256;    // token kernel
constexpr int kMaxStaged = 8192;    // offsets kept in LDS (32 KiB)

struct Request {
  int row;         // -1: outside the tables
  uint32_t c, q;   // computed tokens, tokens of the step (c + q < 2^32)
  int held, need;  // blocks before the step, and after it
  __device__ int fresh() const { return max(need - held, 0); }
};

// Request b, or an empty one behind the batch.  Loads are unconditional (of
// some valid place where there is nothing to read), so that those of several
// requests stand together.
__device__ __forceinline__ Request load_request(const TablesParams& p,
                                                int b) {
  Request r{-1, 0, 0, 0, 0};
  const bool in = b < p.B;
  const int at = in ? b : p.B - 1;
  const int q = p.query_lens[at];
  const int row = p.req_idx ? p.req_idx[at] : at;
  r.q = in ? uint32_t(max(q, 0)) : 0;
  if (p.rows == 0) return r;
  const bool ok = in && row >= 0 && row < p.rows;
  const int c = p.computed[ok ? row : 0], held = p.held[ok ? row : 0];
  if (ok) {
    r.row = row;
    r.c = uint32_t(max(c, 0));
    r.held = min(max(held, 0), p.width);
    r.need = int(min((r.c + r.q) / uint32_t(p.block) + 1, uint32_t(p.width)));
  }
  return r;
}

// Block i, at most that of the request's next token, of a request whose new
// blocks start at free_blocks[first].
__device__ __forceinline__ int block_of(const TablesParams& p,
                                        const Request& r, int64_t first,
                                        uint32_t i) {
  const int64_t f = first + (int64_t(i) - r.held);
  const bool old = int64_t(i) < r.held;
  const bool ok = r.row >= 0 && i < uint32_t(p.width) &&
                  (old || f < p.num_free);
  const int32_t* at = old ? p.table + r.row * p.s_tab_row + i * p.s_tab_col
                          : p.free_blocks + f;
  const int v = *(ok ? at : p.query_lens);      // (any valid place)
  return ok ? v : p.null_id;
}

// Inclusive prefix sum over a wave.
__device__ __forceinline__ int64_t wave_scan(int64_t v, int lane) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int64_t o = __shfl_up(v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// Exclusive prefix sums of two numbers over the workgroup, and their totals.
template <int NT>
__device__ __forceinline__ void block_scan(int64_t (&v)[2], int64_t (&total)[2],
                                           int64_t (*red)[2]) {
  constexpr int kWaves = NT / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int64_t upto[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) upto[i] = wave_scan(v[i], lane);
  __syncthreads();                       // the last call's red is read
  if (lane == 63) {
    red[w][0] = upto[0];
    red[w][1] = upto[1];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // each wave sums the waves' totals for itself
    const int64_t s = wave_scan(red[lane & (kWaves - 1)][i], lane);
    total[i] = __shfl(s, kWaves - 1);
    const int64_t before = __shfl(s, max(w - 1, 0));
    v[i] = upto[i] - v[i] + (w > 0 ? before : 0);
  }
}

// One tile of K requests a thread at a time, in batch order.
template <int NT, int K>
__global__ void __launch_bounds__(NT)
    kda_request_tables_kernel(TablesParams p) {
  constexpr int kTile = K * NT;
  __shared__ int64_t red[NT / 64][2];
  __shared__ int64_t first[kTile];       // of the request's new blocks
  __shared__ int32_t row[kTile], held[kTile];
  const int tid = threadIdx.x;
  int64_t done[2] = {0, 0};              // tokens, new blocks of earlier tiles
  for (int b0 = 0; b0 < p.B; b0 += kTile) {
    Request r[K];
#pragma unroll
    for (int j = 0; j < K; ++j) r[j] = load_request(p, b0 + tid * K + j);
    int64_t at[2] = {0, 0}, total[2];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      at[0] += r[j].q;
      at[1] += r[j].fresh();
    }
    block_scan<NT>(at, total, red);
#pragma unroll
    for (int i = 0; i < 2; ++i) at[i] += done[i];
    int src[K], dst[K];
    int64_t tok[K];
    int64_t blk = at[1];
    tok[0] = at[0];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      if (j > 0) tok[j] = tok[j - 1] + r[j - 1].q;
      src[j] = block_of(p, r[j], blk, r[j].c / uint32_t(p.block));
      dst[j] = block_of(p, r[j], blk, (r[j].c + r[j].q) / uint32_t(p.block));
      first[tid * K + j] = blk;
      row[tid * K + j] = r[j].row;
      held[tid * K + j] = r[j].held;
      blk += r[j].fresh();
    }
    blk = at[1];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int b = b0 + tid * K + j;
      if (b < p.B) {
        p.qsl[b] = int(min(tok[j], int64_t(p.cap)));
        p.slots[b] = src[j];
        p.initial[b] = r[j].c > 0 ? src[j] : p.null_id;
        p.final_slots[b] = dst[j];
        if (r[j].row >= 0)
          p.new_held[r[j].row] =
              r[j].held + int(min(int64_t(r[j].fresh()),
                                  max(p.num_free - blk, int64_t(0))));
      }
      blk += r[j].fresh();
    }
    __syncthreads();                     // the tile's requests are in LDS
    const int n = min(p.B - b0, kTile);
    for (int64_t f = done[1] + tid; f < done[1] + total[1];
         f += NT) {
      int lo = 0, hi = n;                // the last request with first <= f
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (first[m] <= f)
          lo = m;
        else
          hi = m;
      }
      p.table[row[lo] * p.s_tab_row +
              (held[lo] + (f - first[lo])) * p.s_tab_col] =
          f < p.num_free ? p.free_blocks[f] : p.null_id;
    }
    done[0] += total[0];
    done[1] += total[1];
    __syncthreads();                     // the tile in LDS has been read
  }
  if (tid == 0) {
    p.qsl[p.B] = int(min(done[0], int64_t(p.cap)));
    p.allocated[0] = int(min(done[1], int64_t(0x7fffffff)));
  }
}

// Number of the request of token t: the last b with off[b] <= t.
__device__ __forceinline__ int request_of(const int32_t* off, int B, int t) {
  int lo = 0, hi = B;          // off[lo] <= t < off[hi]
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (off[m] <= t)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

__global__ void __launch_bounds__(kTokThreads)
    kda_token_tables_kernel(TablesParams p) {
  __shared__ int32_t staged[kMaxStaged];
  const int32_t total = p.qsl[p.B];
  const int32_t* off = p.qsl;
  const int t0 = blockIdx.x * kTokThreads, t = t0 + threadIdx.x;
  if (t0 < total && p.B <= kMaxStaged) {
    for (int i = threadIdx.x; i < p.B; i += kTokThreads) staged[i] = p.qsl[i];
    __syncthreads();
    off = staged;
  }
  if (t >= p.cap) return;
  int pos = 0;
  int64_t slot = -1;
  if (t < total) {
    const int b = request_of(off, p.B, t);
    const int row = p.req_idx ? p.req_idx[b] : b;
    const bool ok = row >= 0 && row < p.rows;
    const uint32_t c = ok ? uint32_t(max(p.computed[row], 0)) : 0;
    const uint32_t at = c + uint32_t(t - off[b]);
    pos = int(at);
    const uint32_t blk = at / uint32_t(p.block);
    if (ok && blk < uint32_t(p.width)) {
      const int id = p.table[row * p.s_tab_row + blk * p.s_tab_col];
      if (id > p.null_id)
        slot = int64_t(id) * p.block + (at - blk * uint32_t(p.block));
    }
  }
  p.positions[t] = pos;
  p.slot_mapping[t] = slot;
}

}  // namespace

int launch_step_tables(const TablesParams& p, hipStream_t stream) {
  // few waves for few requests (their barriers are quicker: 3.4 us, 4.9 with
  // 1024 threads), two requests a thread where one would take a second tile
  if (p.B <= 256)
    launch_kernel(kda_request_tables_kernel<256, 1>, dim3(1), dim3(256), 0,
                  stream, p);
  else if (p.B <= 1024)
    launch_kernel(kda_request_tables_kernel<1024, 1>, dim3(1), dim3(1024), 0,
                  stream, p);
  else
    launch_kernel(kda_request_tables_kernel<1024, 2>, dim3(1), dim3(1024), 0,
                  stream, p);
  if (p.cap > 0)
    launch_kernel(kda_token_tables_kernel,
                  dim3((p.cap - 1) / kTokThreads + 1), dim3(kTokThreads), 0,
                  stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
