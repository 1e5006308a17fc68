// Index arrays of one serving step on gfx950, from request lengths: token
// offsets, block allocation, state slots, and the position and cache slot of
// every token.
//
// Two exclusive prefix sums over the batch (tokens, new blocks) order
// everything: blocks are handed out in batch order, so no atomic decides who
// gets which, and every run gives the same tables.  The request kernel is one
// workgroup (a step has at most some thousand requests; a second workgroup
// would have to wait for the first one's sums): each thread takes one request
// of a tile, reads its lengths before it writes its row, so that the held
// counts may be updated in place.  The token kernel then has one thread per
// token; a workgroup keeps the token offsets in LDS and each thread finds its
// request by a binary search there.
#include "kda_serving.hpp"

namespace kda {
namespace {

constexpr int kTabThreads = 1024;   // request kernel
constexpr int kTokThreads = 256;    // token kernel
constexpr int kMaxStaged = 8192;    // offsets kept in LDS (32 KiB)

struct Request {
  int row;         // -1: outside the tables
  uint32_t c, q;   // computed tokens, tokens of the step (c + q < 2^32)
  int held, need;  // blocks before the step, and after it
  __device__ int fresh() const { return max(need - held, 0); }
};

__device__ __forceinline__ Request load_request(const TablesParams& p,
                                                int b) {
  Request r;
  const int row = p.req_idx ? p.req_idx[b] : b;
  r.q = uint32_t(max(p.query_lens[b], 0));
  r.row = row >= 0 && row < p.rows ? row : -1;
  r.c = r.row < 0 ? 0 : uint32_t(max(p.computed[r.row], 0));
  r.held = r.row < 0 ? 0 : min(max(p.held[r.row], 0), p.width);
  r.need = r.row < 0 ? 0
                     : int(min((r.c + r.q) / uint32_t(p.block) + 1,
                               uint32_t(p.width)));
  return r;
}

// Block i of a request whose new blocks start at free_blocks[first].
__device__ __forceinline__ int block_of(const TablesParams& p,
                                        const Request& r, int64_t first,
                                        uint32_t i) {
  const int32_t* at = nullptr;
  if (r.row >= 0 && i < uint32_t(p.width)) {
    const int64_t f = first + (int(i) - r.held);
    if (int(i) < r.held || int(i) >= r.need)
      at = p.table + r.row * p.s_tab_row + i * p.s_tab_col;
    else if (f < p.num_free)
      at = p.free_blocks + f;
  }
  return at ? *at : p.null_id;
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

// Inclusive prefix sum over the workgroup; the total is then in
// red[kTabThreads / 64 - 1] until the next call.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* red) {
  constexpr int kWaves = kTabThreads / 64;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  v = wave_scan(v, lane);
  __syncthreads();                       // the last call's red is read
  if (lane == 63) red[w] = v;
  __syncthreads();
  if (w == 0) {
    const int64_t s = wave_scan(lane < kWaves ? red[lane] : 0, lane);
    if (lane < kWaves) red[lane] = s;
  }
  __syncthreads();
  return w > 0 ? v + red[w - 1] : v;
}

__device__ __forceinline__ void store_request(const TablesParams& p, int b,
                                              const Request& r, int64_t tok,
                                              int64_t first) {
  p.qsl[b] = int(min(tok, int64_t(p.cap)));
  const int src = block_of(p, r, first, r.c / uint32_t(p.block));
  p.slots[b] = src;
  p.initial[b] = r.c > 0 ? src : p.null_id;
  p.final_slots[b] = block_of(p, r, first, (r.c + r.q) / uint32_t(p.block));
  if (r.row < 0) return;
  const int fresh = r.fresh();
  for (int j = 0; j < fresh; ++j) {
    const int64_t f = first + j;
    p.table[r.row * p.s_tab_row + int64_t(r.held + j) * p.s_tab_col] =
        f < p.num_free ? p.free_blocks[f] : p.null_id;
  }
  const int64_t left = max(p.num_free - first, int64_t(0));
  p.new_held[r.row] = r.held + int(min(int64_t(fresh), left));
}

__global__ void __launch_bounds__(kTabThreads)
    kda_request_tables_kernel(TablesParams p) {
  __shared__ int64_t red[kTabThreads / 64];
  int64_t tok0 = 0, blk0 = 0;
  for (int b0 = 0; b0 < p.B; b0 += kTabThreads) {
    const int b = b0 + threadIdx.x;
    Request r{-1, 0, 0, 0, 0};
    if (b < p.B) r = load_request(p, b);
    const int64_t tok = tok0 + block_scan(r.q, red) - r.q;
    tok0 += red[kTabThreads / 64 - 1];
    const int64_t blk = blk0 + block_scan(r.fresh(), red) - r.fresh();
    blk0 += red[kTabThreads / 64 - 1];
    if (b < p.B) store_request(p, b, r, tok, blk);
  }
  if (threadIdx.x == 0) {
    p.qsl[p.B] = int(min(tok0, int64_t(p.cap)));
    p.allocated[0] = int(min(blk0, int64_t(0x7fffffff)));
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
  launch_kernel(kda_request_tables_kernel, dim3(1), dim3(kTabThreads), 0,
                stream, p);
  if (p.cap > 0)
    launch_kernel(kda_token_tables_kernel,
                  dim3((p.cap - 1) / kTokThreads + 1), dim3(kTokThreads), 0,
                  stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
