// The life of cache blocks on gfx950: copies over all pools of a model, forks
// of requests, counting references and listing free blocks, compaction.
//
// Copies are the work: one launch moves the blocks of every pair and pool, a
// workgroup a chunk of one block, 16 bytes a load where the pool allows it.
// The rest is integer bookkeeping in which no order of atomics shows: lists
// are in rising order, ranks come from prefix sums over blocks.  A prefix sum
// over N blocks is two launches (a count of each 4096, then every workgroup
// sums the counts before its own), since N passes what one CU scans quickly.
//
// What bounds them: copies move 584 MB (64 forks, 32 heads of two layers and a
// latent cache) in 91 us, at 6.4 TB/s, part of the reads from the last-level
// cache.  The bookkeeping of 8192 blocks and 512 rows of 40 entries takes 15 us
// (free lists, half of it the pass over the table in one workgroup) and 10 + 5
// us (compaction, the table in a launch of its own).  32 rows of the table under
// way in place of 8 take longer: so does their code to arrive.  Forks take 4 to
// 5 us.
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr int kThreads = 256;

// ---- copies -------------------------------------------------------------------

constexpr int kCopyChunk = 32768;   // bytes of a workgroup's piece

template <class T>
__device__ __forceinline__ void copy_piece(const char* src, char* dst,
                                           int64_t bytes) {
  constexpr int U = 4;              // loads under way together
  const int64_t n = bytes / int64_t(sizeof(T));
  const T* s = reinterpret_cast<const T*>(src);
  T* d = reinterpret_cast<T*>(dst);
  int64_t i = threadIdx.x;
  for (; i + (U - 1) * kThreads < n; i += U * kThreads) {
    T v[U];
#pragma unroll
    for (int k = 0; k < U; ++k) v[k] = s[i + k * kThreads];
#pragma unroll
    for (int k = 0; k < U; ++k) d[i + k * kThreads] = v[k];
  }
  for (; i < n; i += kThreads) d[i] = s[i];
}

__global__ void __launch_bounds__(kThreads)
    kda_copy_blocks_kernel(CopyParams p) {
  const int layer = blockIdx.y;
  const int64_t base = p.tables[layer];
  const int64_t stride = p.tables[p.L + layer];
  const int64_t bytes = p.tables[2 * p.L + layer];
  const int pairs = p.num_pairs ? min(max(p.num_pairs[0], 0), p.P) : p.P;
  const int64_t pieces = (bytes + kCopyChunk - 1) / kCopyChunk;
  char* pool = global_addr<char>(base);
  const bool wide = ((base | stride | bytes) & 15) == 0;
  const bool words = ((base | stride | bytes) & 3) == 0;
  for (int64_t i = blockIdx.x; i < pairs * pieces; i += gridDim.x) {
    const int pair = int(i / pieces);
    const int src = p.pairs[2 * pair], dst = p.pairs[2 * pair + 1];
    if (src <= p.null_id || src >= p.N || dst <= p.null_id || dst >= p.N ||
        src == dst)
      continue;
    const int64_t at = (i - pair * pieces) * kCopyChunk;
    const int64_t n = min(bytes - at, int64_t(kCopyChunk));
    const char* s = pool + src * stride + at;
    char* d = pool + dst * stride + at;
    if (wide)
      copy_piece<u4>(s, d, n);
    else if (words)
      copy_piece<uint32_t>(s, d, n);
    else
      copy_piece<char>(s, d, n);
  }
}

// ---- forks ----------------------------------------------------------------------

// Parent and child rows of fork f; false for one that does nothing.
__device__ __forceinline__ bool fork_rows(const ForkParams& p, int f, int* a,
                                          int* b) {
  *a = p.parents[f];
  *b = p.children[f];
  return *a >= 0 && *a < p.rows && *b >= 0 && *b < p.rows && *a != *b &&
         p.width > 0;
}

// Whether fork f needs a block of its own: the next token's lies in the table.
// (No fork's child is a parent, so the lengths read here stay.)
__device__ __forceinline__ bool fork_takes(const ForkParams& p, int f) {
  int a, b;
  return fork_rows(p, f, &a, &b) && max(p.computed[a], 0) / p.block < p.width;
}

// One workgroup a fork; a fork's rank among those that need a block gives the
// free one that it takes.
__global__ void __launch_bounds__(kThreads) kda_fork_kernel(ForkParams p) {
  __shared__ int red[kThreads / 64];
  const int f = blockIdx.x, tid = threadIdx.x;
  if (p.F == 0) {                            // (a count of none is written)
    if (tid == 0) p.allocated[0] = 0;
    return;
  }
  int a, b, n = 0;
  for (int i = tid; i < f; i += kThreads) n += fork_takes(p, i);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) n += __shfl_xor(n, s);
  if ((tid & 63) == 0) red[tid >> 6] = n;
  __syncthreads();
  int rank = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 64; ++k) rank += red[k];
  if (f == p.F - 1 && tid == 0) p.allocated[0] = rank + fork_takes(p, f);
  const bool ok = fork_rows(p, f, &a, &b);
  if (!ok) {
    if (tid < 2) p.pairs[2 * f + tid] = p.null_id;
    return;
  }
  const int c = max(p.computed[a], 0);
  const int last = c / p.block;              // the block of the next token
  const int32_t* from = p.table + a * p.s_tab_row;
  int32_t* to = p.table + b * p.s_tab_row;
  for (int i = tid; i < min(last, p.width); i += kThreads)
    to[i * p.s_tab_col] = from[i * p.s_tab_col];
  if (tid > 0) return;
  const bool fits = last < p.width && rank < p.num_free;
  const int id = fits ? p.free_blocks[rank] : p.null_id;
  if (last < p.width) to[last * p.s_tab_col] = id;
  // a parent that does not hold that block has nothing to copy
  const bool held = last < p.width && last < p.held[a];
  const int src = held ? from[last * p.s_tab_col] : p.null_id;
  const bool copy = src > p.null_id && id > p.null_id;
  p.pairs[2 * f] = copy ? src : p.null_id;
  p.pairs[2 * f + 1] = copy ? id : p.null_id;
  p.computed[b] = c;
  p.held[b] = min(last + 1, p.width);
}

// ---- references and free blocks ---------------------------------------------------

__global__ void __launch_bounds__(kThreads) kda_free_start_kernel(FreeParams p) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < p.N) p.refs[i] = p.pinned ? max(p.pinned[i], 0) : 0;
}

__global__ void __launch_bounds__(kThreads) kda_free_count_kernel(FreeParams p) {
  const int row = blockIdx.x;
  int released = 0;                          // (a row may be named twice)
  for (int i = threadIdx.x; i < p.R; i += kThreads)
    released |= p.released[i] == row;
  released = __syncthreads_or(released);
  const int n = released ? 0 : min(max(p.held[row], 0), p.width);
  __syncthreads();                           // (new_held may be held itself)
  if (threadIdx.x == 0) p.new_held[row] = n;
  const int32_t* t = p.table + row * p.s_tab_row;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int id = t[i * p.s_tab_col];
    if (id > p.null_id && id < p.N) atomicAdd(&p.refs[id], 1);
  }
}

// Whether block i is live, as 0 or 1; blocks up to the null one count for
// nothing.
__device__ __forceinline__ int is_live(const int32_t* refs, int64_t i,
                                       int64_t N, int null_id) {
  return i > null_id && i < N && refs[i] > 0;
}

// Live blocks of each 4096.
__global__ void __launch_bounds__(kThreads)
    kda_live_count_kernel(const int32_t* refs, int32_t* counts, int64_t N,
                          int null_id) {
  __shared__ int red[kThreads / 64];
  int n = 0;
  for (int k = 0; k < kBlockChunk / kThreads; ++k)
    n += is_live(refs, int64_t(blockIdx.x) * kBlockChunk + k * kThreads +
                           threadIdx.x, N, null_id);
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) n += __shfl_xor(n, s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = n;
  __syncthreads();
  if (threadIdx.x == 0) {
    int all = 0;
    for (int k = 0; k < kThreads / 64; ++k) all += red[k];
    counts[blockIdx.x] = all;
  }
}

// Sum of `n` counts, the same in every thread.
__device__ __forceinline__ int sum_counts(const int32_t* counts, int n,
                                          int* red) {
  int v = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) v += counts[i];
#pragma unroll
  for (int s = 32; s > 0; s >>= 1) v += __shfl_xor(v, s);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  int all = 0;
  for (int k = 0; k < kThreads / 64; ++k) all += red[k];
  return all;
}

// Exclusive rank among the live blocks of a row of kThreads, and their count.
__device__ __forceinline__ int live_rank(int live, int* total, int* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint64_t m = __ballot(live);
  __syncthreads();
  if (lane == 0) red[w] = __popcll(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int k = 0; k < kThreads / 64; ++k) {
    before += k < w ? red[k] : 0;
    all += red[k];
  }
  *total = all;
  return before + __popcll(m & ((uint64_t(1) << lane) - 1));
}

__global__ void __launch_bounds__(kThreads) kda_free_list_kernel(FreeParams p) {
  __shared__ int red[kThreads / 64];
  const int chunks = gridDim.x;
  const int total = sum_counts(p.counts, chunks, red);
  int rank = sum_counts(p.counts, blockIdx.x, red);
  const int64_t first = int64_t(p.null_id) + 1;
  const int free = int(max(p.N - first, int64_t(0))) - total;
  if (blockIdx.x == 0 && threadIdx.x == 0) p.num_free[0] = free;
  for (int k = 0; k < kBlockChunk / kThreads; ++k) {
    const int64_t i = int64_t(blockIdx.x) * kBlockChunk + k * kThreads +
                      threadIdx.x;
    int n;
    const int live = is_live(p.refs, i, p.N, p.null_id);
    const int r = rank + live_rank(live, &n, red);
    rank += n;
    if (i >= p.N) continue;
    if (i >= first && !live) p.free_blocks[i - first - r] = int(i);
    // null ids behind the last free block
    if (i >= free) p.free_blocks[i] = p.null_id;
  }
}

// ---- compaction ----------------------------------------------------------------------

// The i-th live block above null + live (in rising order) moves to the i-th
// free one up to there.
__global__ void __launch_bounds__(kThreads)
    kda_compact_plan_kernel(CompactBlocksParams p) {
  __shared__ int red[kThreads / 64];
  const int chunks = gridDim.x;
  const int total = sum_counts(p.counts, chunks, red);
  int rank = sum_counts(p.counts, blockIdx.x, red);
  const int64_t first = int64_t(p.null_id) + 1, end = first + total;
  // live blocks in front of `end`, which lies inside a chunk
  const int cut = int(end / kBlockChunk);
  int low = sum_counts(p.counts, min(cut, chunks), red);
  for (int k = 0; k < kBlockChunk / kThreads; ++k) {
    const int64_t i = int64_t(cut) * kBlockChunk + k * kThreads +
                      threadIdx.x;
    int n;
    live_rank(i < end && is_live(p.refs, i, p.N, p.null_id), &n, red);
    low += n;
  }
  const int moves = total - low;
  if (blockIdx.x == 0 && threadIdx.x == 0)
    p.num_pairs[0] = min(moves, p.max_pairs);
  for (int k = 0; k < kBlockChunk / kThreads; ++k) {
    const int64_t i = int64_t(blockIdx.x) * kBlockChunk + k * kThreads +
                      threadIdx.x;
    int n;
    const int live = is_live(p.refs, i, p.N, p.null_id);
    const int r = rank + live_rank(live, &n, red);
    rank += n;
    if (i >= p.N) continue;
    if (i >= end && live) {
      const int at = r - low;
      p.moved[i] = at;
      if (at < p.max_pairs) p.pairs[2 * at] = int(i);
    } else if (i >= first && i < end && !live) {
      const int at = int(i - first) - r;
      if (at < p.max_pairs) p.pairs[2 * at + 1] = int(i);
    }
    for (int64_t j = i; j < p.max_pairs; j += p.N)
      if (j >= moves) p.pairs[2 * j] = p.pairs[2 * j + 1] = p.null_id;
  }
}

// Reference counts at their new places.
__global__ void __launch_bounds__(kThreads)
    kda_compact_refs_kernel(CompactBlocksParams p) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.N) return;
  p.new_refs[i] = p.refs[i];
}

__global__ void __launch_bounds__(kThreads)
    kda_compact_move_refs_kernel(CompactBlocksParams p) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i >= p.num_pairs[0]) return;
  const int src = p.pairs[2 * i], dst = p.pairs[2 * i + 1];
  p.new_refs[dst] = p.new_refs[src];
  p.new_refs[src] = 0;
}

__global__ void __launch_bounds__(kThreads)
    kda_compact_table_kernel(CompactBlocksParams p) {
  const int row = blockIdx.x;
  const int n = min(max(p.held[row], 0), p.width);
  const int32_t* from = p.table + row * p.s_tab_row;
  int32_t* to = p.new_table + row * p.s_new_row;
  const int total = p.num_pairs[0];
  // moved blocks are at least the first pair's; an id that no reference counts
  // has nothing in `moved`, so its entry is held against the pair it names
  const int lowest = total > 0 ? p.pairs[0] : 0x7fffffff;
  for (int i = threadIdx.x; i < p.width; i += kThreads) {
    int id = from[i * p.s_tab_col];
    if (i < n && id >= lowest && id < p.N) {
      const int at = p.moved[id];
      if (at >= 0 && at < total && p.pairs[2 * at] == id)
        id = p.pairs[2 * at + 1];
    }
    to[i * p.s_new_col] = id;
  }
}

// ---- the same in one workgroup ---------------------------------------------------

// Pools of up to kSmallBlocks blocks take one launch or two in place of four or
// five: all counts and lists fit LDS.  The table is read in rounds of kRound rows
// by 64 columns (each_entry), 0.7 to 1.9 us each:
// - free lists count it in that launch for up to kFreeRounds rounds, else in
//   four launches (8192 blocks, 512 rows of 40, 4 rounds: 13 us, 17 in four;
//   16384 blocks, 1024 rows of 64, 8 rounds: 27, 19; 4096 rows of 16: 77, 21);
// - compaction rewrites it in that launch for one round, else in a second one
//   with a workgroup a row (5 rows of 6: 4.7 us, 5.0 in two; 64 rows of 64:
//   8.3, 8.4; 512 rows of 8: 18.8, 11.2; 4096 rows of 16: 89, 22, and 23 in
//   five).
constexpr int kSmallBlocks = 16384;
constexpr int kMany = 1024;        // threads
constexpr int kAtOnce = 8;         // rows that a wave has under way
constexpr int kRound = kAtOnce * kMany / 64;
constexpr int kFreeRounds = 4;
constexpr int kSmallRows = kFreeRounds * kRound;
__host__ __device__ constexpr int64_t rounds_of(int64_t rows, int64_t width) {
  return (rows + kRound - 1) / kRound * ((width + 63) / 64);
}

// Exclusive prefix sum over the workgroup's threads, and the total.
__device__ __forceinline__ int scan_many(int v, int* total, int* red) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  int upto = v;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const int o = __shfl_up(upto, s);
    if (lane >= s) upto += o;
  }
  __syncthreads();
  if (lane == 63) red[w] = upto;
  __syncthreads();
  int before = 0, all = 0;
  for (int k = 0; k < kMany / 64; ++k) {
    before += k < w ? red[k] : 0;
    all += red[k];
  }
  *total = all;
  return before + upto - v;
}

// Every entry of a table, a wave a row, kAtOnce rows under way together.
template <class Load, class Use>
__device__ __forceinline__ void each_entry(int rows, int width, Load load,
                                           Use use) {
  constexpr int U = kAtOnce, kWaves = kMany / 64;
  const int lane = threadIdx.x & 63, w = uniform(threadIdx.x >> 6);
  for (int r0 = w; r0 < rows; r0 += U * kWaves)
    for (int j = lane; j < width; j += 64) {
      int id[U];
#pragma unroll
      for (int k = 0; k < U; ++k)
        id[k] = load(min(r0 + k * kWaves, rows - 1), j);
#pragma unroll
      for (int k = 0; k < U; ++k)
        if (r0 + k * kWaves < rows) use(r0 + k * kWaves, j, id[k]);
    }
}

__global__ void __launch_bounds__(kMany) kda_free_small_kernel(FreeParams p) {
  extern __shared__ __align__(16) int32_t refs[];   // [N], then held [rows]
  __shared__ int red[kMany / 64];
  const int tid = threadIdx.x, N = int(p.N);
  int32_t* held = refs + N;
  for (int i = tid; i < N; i += kMany)
    refs[i] = p.pinned ? max(p.pinned[i], 0) : 0;
  for (int i = tid; i < p.rows; i += kMany)
    held[i] = min(max(p.held[i], 0), p.width);
  __syncthreads();
  for (int i = tid; i < p.R; i += kMany) {
    const int row = p.released[i];
    if (row >= 0 && row < p.rows) held[row] = 0;
  }
  __syncthreads();
  for (int i = tid; i < p.rows; i += kMany) p.new_held[i] = held[i];
  if (p.width > 0)
    each_entry(
        p.rows, p.width,
        [&](int r, int j) {
          return j < held[r] ? p.table[r * p.s_tab_row + j * p.s_tab_col]
                             : p.null_id;
        },
        [&](int, int, int id) {
          if (id > p.null_id && id < N) atomicAdd(&refs[id], 1);
        });
  __syncthreads();
  for (int i = tid; i < N; i += kMany) p.refs[i] = refs[i];
  // each thread lists the free ones among its own run of blocks
  const int run = (N + kMany - 1) / kMany, lo = min(tid * run, N),
            hi = min(lo + run, N);
  int n = 0, total;
  for (int i = lo; i < hi; ++i) n += i > p.null_id && refs[i] <= 0;
  int at = scan_many(n, &total, red);
  for (int i = lo; i < hi; ++i)
    if (i > p.null_id && refs[i] <= 0) p.free_blocks[at++] = i;
  for (int i = total + tid; i < N; i += kMany) p.free_blocks[i] = p.null_id;
  if (tid == 0) p.num_free[0] = total;
}

__global__ void __launch_bounds__(kMany)
    kda_compact_small_kernel(CompactBlocksParams p) {
  extern __shared__ __align__(16) int32_t refs[];   // [N], then lists
  __shared__ int red[kMany / 64];
  const int tid = threadIdx.x, N = int(p.N);
  const bool inside = rounds_of(p.rows, p.width) <= 1;
  uint16_t* src = reinterpret_cast<uint16_t*>(refs + N);   // [N / 2 + 1]
  uint16_t* dst = src + N / 2 + 1;
  uint16_t* map = dst + N / 2 + 1;                         // [N]
  int32_t* held = refs + 2 * N + 1;                        // [rows]
  if (inside)
    for (int i = tid; i < min(p.rows, kRound); i += kMany) held[i] = p.held[i];
  for (int i = tid; i < N; i += kMany) {
    refs[i] = p.refs[i];
    map[i] = uint16_t(i);
  }
  __syncthreads();
  const int run = (N + kMany - 1) / kMany, lo = min(tid * run, N),
            hi = min(lo + run, N);
  auto live = [&](int i) { return i > p.null_id && refs[i] > 0; };
  int n = 0, total, moves;
  for (int i = lo; i < hi; ++i) n += live(i);
  const int rank = scan_many(n, &total, red);
  const int first = p.null_id + 1, end = first + total;
  n = 0;
  for (int i = max(lo, end); i < hi; ++i) n += live(i);
  int from = scan_many(n, &moves, red);      // moves: live ones from end on
  int free = lo > first ? lo - first - rank : 0;
  for (int i = lo; i < hi; ++i) {
    if (i >= end && live(i)) src[from++] = uint16_t(i);
    if (i >= first && i < end && !live(i)) dst[free++] = uint16_t(i);
  }
  __syncthreads();
  moves = min(moves, p.max_pairs);
  for (int64_t i = tid; i < p.max_pairs; i += kMany) {
    const bool in = i < moves;
    const int a = in ? src[i] : p.null_id, b = in ? dst[i] : p.null_id;
    p.pairs[2 * i] = a;
    p.pairs[2 * i + 1] = b;
    if (in) {
      map[a] = uint16_t(b);
      if (!inside) p.moved[a] = int(i);
      refs[b] = refs[a];
      refs[a] = 0;
    }
  }
  if (tid == 0) p.num_pairs[0] = moves;
  __syncthreads();
  for (int i = tid; i < N; i += kMany) p.new_refs[i] = refs[i];
  if (inside && p.width > 0)
    each_entry(
        p.rows, p.width,
        [&](int r, int j) { return p.table[r * p.s_tab_row + j * p.s_tab_col]; },
        [&](int r, int j, int id) {
          if (j < held[r] && id > p.null_id && id < N) id = map[id];
          p.new_table[r * p.s_new_row + j * p.s_new_col] = id;
        });
}

}  // namespace

int launch_copy_blocks(const CopyParams& p, int64_t pieces,
                       hipStream_t stream) {
  // pieces: an upper bound of one pool's; workgroups go through them in steps
  // of the grid, some 16 to a CU
  const int64_t most = 4096 / p.L + 1;
  const dim3 grid(uint32_t(pieces < most ? pieces : most), p.L);
  launch_kernel(kda_copy_blocks_kernel, grid, dim3(kThreads), 0, stream, p);
  return int(hipGetLastError());
}
int64_t copy_pieces(int64_t bytes) {
  return (bytes + kCopyChunk - 1) / kCopyChunk;
}

int launch_fork_blocks(const ForkParams& p, hipStream_t stream) {
  launch_kernel(kda_fork_kernel, dim3(p.F > 0 ? p.F : 1), dim3(kThreads), 0,
                stream, p);
  return int(hipGetLastError());
}

namespace {
dim3 grid_of(int64_t n) {
  return dim3(uint32_t((n + kThreads - 1) / kThreads));
}
template <class F>
hipError_t more_lds(F kernel) {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                             hipFuncAttributeMaxDynamicSharedMemorySize,
                             (kSmallBlocks * 2 + 1 + kSmallRows) * 4);
}
dim3 chunks_of(int64_t N) {
  return dim3(uint32_t((N + kBlockChunk - 1) / kBlockChunk));
}
}  // namespace

int launch_free_blocks(const FreeParams& p, hipStream_t stream) {
  if (p.N <= kSmallBlocks && rounds_of(p.rows, p.width) <= kFreeRounds &&
      p.rows <= kSmallRows) {
    const hipError_t e = more_lds(kda_free_small_kernel);
    if (e != hipSuccess) return int(e);
    launch_kernel(kda_free_small_kernel, dim3(1), dim3(kMany),
                  uint32_t(p.N + p.rows) * 4, stream, p);
    return int(hipGetLastError());
  }
  launch_kernel(kda_free_start_kernel, grid_of(p.N), dim3(kThreads), 0, stream,
                p);
  if (p.rows > 0)
    launch_kernel(kda_free_count_kernel, dim3(p.rows), dim3(kThreads), 0,
                  stream, p);
  launch_kernel(kda_live_count_kernel, chunks_of(p.N), dim3(kThreads), 0,
                stream, static_cast<const int32_t*>(p.refs), p.counts, p.N,
                p.null_id);
  launch_kernel(kda_free_list_kernel, chunks_of(p.N), dim3(kThreads), 0,
                stream, p);
  return int(hipGetLastError());
}

int launch_compact_blocks(const CompactBlocksParams& p, hipStream_t stream) {
  if (p.N <= kSmallBlocks) {
    const hipError_t e = more_lds(kda_compact_small_kernel);
    if (e != hipSuccess) return int(e);
    launch_kernel(kda_compact_small_kernel, dim3(1), dim3(kMany),
                  uint32_t(p.N * 2 + 1 + kRound) * 4, stream, p);
    if (rounds_of(p.rows, p.width) > 1)
      launch_kernel(kda_compact_table_kernel, dim3(p.rows), dim3(kThreads), 0,
                    stream, p);
    return int(hipGetLastError());
  }
  launch_kernel(kda_live_count_kernel, chunks_of(p.N), dim3(kThreads), 0,
                stream, p.refs, p.counts, p.N, p.null_id);
  launch_kernel(kda_compact_plan_kernel, chunks_of(p.N), dim3(kThreads), 0,
                stream, p);
  if (p.new_refs != p.refs)
    launch_kernel(kda_compact_refs_kernel, grid_of(p.N), dim3(kThreads), 0,
                  stream, p);
  if (p.max_pairs > 0)
    launch_kernel(kda_compact_move_refs_kernel, grid_of(p.max_pairs),
                  dim3(kThreads), 0, stream, p);
  if (p.rows > 0 && p.width > 0)
    launch_kernel(kda_compact_table_kernel, dim3(p.rows), dim3(kThreads), 0,
                  stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
