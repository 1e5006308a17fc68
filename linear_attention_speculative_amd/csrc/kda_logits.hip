// Changes of logits in front of the sampling on gfx950: biases, penalties for
// repeated tokens and grammar masks, in place.
//
//   y = x + bias;  seen token: y > 0 ? y / r : y r;  count > 0: y - f count - p;
//   not allowed: -inf.
//
// `count` is how often a token was produced: the history behind the prompt, and
// in a draft window the drafts up to the row.  Nothing is kept between calls.
// One workgroup takes a request: it counts the tokens of its history in a table
// in LDS that is addressed by the token (integer atomics: no order changes a
// count), with each token's last bias, lists the places in use, and changes
// their entries in all rows of the window, four under way in each thread.  What
// bounds that is memory: an entry costs a line of it.  Requests with more
// tokens than the table takes go through the vocabulary in slices, a word of
// LDS a token, by workgroups of their own.  The masks are a kernel of their own
// behind it, 16 bytes at a time (in one kernel with the rest, the rows under a
// mask held up their workgroup: 640 rows of 131072 bf16, a quarter of them
// masked, 118 us).  Those rows, with 1500 tokens of history, now take 50 us in
// the table's kernel (91 MB of lines, 1.8 TB/s: one workgroup of 1024 threads a
// request and CU, in phases of counting, listing and changing, of which the
// largest has three times the mean's entries) and 19 us in the masks' (88 MB at
// 4.6 TB/s); a request's single row 6 and 4.  The same batch with 8000 tokens of
// history each, in slices, takes 202 us a call.
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr int kThreads = 1024;
constexpr int kMaskThreads = 256;
constexpr int64_t kMaskRows = 65535;
constexpr int kPlaces = 8192;      // of the table
constexpr int kMost = 6144;        // tokens that it takes
constexpr int kSlice = 4096;       // tokens of a pass without it
constexpr int kPool = 256;         // workgroups of such passes
constexpr int kRows = 64;          // rows of a window whose data is in LDS
// a token of the prompt, one that a row's draft may add, and its count
constexpr uint32_t kSeen = 1u << 31, kListed = 1u << 30, kCount = kListed - 1;

struct Change {
  float r, f, p;
  const int32_t* tokens;           // the request's biases
  const float* values;
  int n;
};

// `w`: seen and count; `e`: a bias's place in the list, plus one.
__device__ __forceinline__ float change(const Change& c, float y, uint32_t w,
                                        uint32_t e) {
  if (e) y += c.values[e - 1];
  if (w) y = y > 0.0f ? y / c.r : y * c.r;
  if (w & kCount) y = y - c.f * float(w & kCount) - c.p;
  return y;
}

// Mask words of a mask row, or null.
__device__ __forceinline__ const int32_t* mask_at(const LogitsParams& p,
                                                  int mr) {
  return mr >= 0 && mr < p.num_masks ? p.mask + mr * p.s_mask : nullptr;
}

// Rows [first, m1) of a window, with what the LDS holds of them.
struct Rows {
  const int32_t* draft;            // draft[m - first]; null: none
  const int32_t* mask_row;         // as well, of given mask rows
  int first, count;
};

// Changes `touched` listed tokens in all rows: token_of(i) and word_of(i) of
// the i-th one, bias_of(i) as change() takes it.
template <bool BF16, class Token, class Word, class Bias>
__device__ __forceinline__ void change_listed(const LogitsParams& p,
                                              const Change& c, const Rows& r,
                                              int touched, Token token_of,
                                              Word word_of, Bias bias_of) {
  typedef typename Act<BF16>::T E;
  constexpr int U = 4;
  const int64_t items = int64_t(touched) * r.count;
  for (int64_t i0 = threadIdx.x; i0 < items; i0 += U * kThreads) {
    E* x[U];
    float y[U];
    uint32_t w[U], e[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      x[k] = nullptr;
      const int64_t i = i0 + k * kThreads;
      if (i >= items) continue;
      const int at = int(i / r.count), j = int(i - int64_t(at) * r.count);
      const int token = token_of(at);
      const int32_t* mask =
          p.mask ? mask_at(p, p.mask_rows ? r.mask_row[j] : r.first + j)
                 : nullptr;
      // (what a mask hides stays as it is)
      if (mask && !((uint32_t(mask[token >> 5]) >> (token & 31)) & 1))
        continue;
      w[k] = word_of(at) & ~kListed;
      if (r.draft)
        for (int d = 1; d <= j; ++d) w[k] += r.draft[d] == token;
      e[k] = bias_of(at);
      if (!(w[k] | e[k])) continue;          // (a later row's draft)
      x[k] = static_cast<E*>(p.logits) + (r.first + j) * p.s_row + token;
      y[k] = ld_elem(x[k], 0, BF16);
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (x[k]) st_elem(x[k], 0, change(c, y[k], w[k], e[k]), BF16);
  }
}

// A request's window, history and parameters.
struct Request {
  int start, end;                  // rows of its window
  const int32_t* history;
  int known, prompt;
  bool drafts;
  Change c;
  // (`known` is 0 where no penalty needs it)
  __device__ __forceinline__ Request(const LogitsParams& p, int b)
      : start(b), end(b + 1), history(nullptr), known(0), prompt(0),
        c{1.0f, 0.0f, 0.0f, nullptr, nullptr, 0} {
    if (p.qsl) {
      start = min(max(p.qsl[b], 0), p.M);
      end = min(max(p.qsl[b + 1], start), p.M);
    }
    if (p.tokens) {
      const int row = p.req_idx ? p.req_idx[b] : b;
      if (row >= 0 && row < p.rows) {
        history = p.tokens + row * p.s_tok;
        known = min(max(p.known[row], 0), p.L);
        prompt = p.prompt[row];
      }
    }
    if (p.rep) c.r = p.rep[b];
    if (p.freq) c.f = p.freq[b];
    if (p.pres) c.p = p.pres[b];
    if (!(c.r > 0.0f)) c.r = 1.0f;           // (NaN, too)
    if (c.f != c.f) c.f = 0.0f;
    if (c.p != c.p) c.p = 0.0f;
    if (p.bias_start) {
      const int lo = min(max(p.bias_start[b], 0), p.num_bias);
      c.n = min(max(p.bias_start[b + 1], lo), p.num_bias) - lo;
      c.tokens = p.bias_tokens + lo;
      c.values = p.bias_values + lo;
    }
    const bool counts = c.r != 1.0f || c.f != 0.0f || c.p != 0.0f;
    if (!counts) known = 0;
    drafts = counts && p.draft;
  }
  // Whether nothing changes, and whether the table takes its tokens.
  __device__ __forceinline__ bool idle() const {
    return start >= end || (known == 0 && !drafts && c.n == 0);
  }
  __device__ __forceinline__ bool fits() const {
    return int64_t(known) + c.n + (drafts ? end - start : 0) <= kMost;
  }
};

// A window of many rows is shared by several workgroups: part `z` of `parts`,
// with the rows' data in LDS where it fits.
__device__ __forceinline__ Rows part_of(const LogitsParams& p,
                                        const Request& q, int z, int parts,
                                        int32_t* row_draft,
                                        int32_t* row_mask) {
  const int per = (q.end - q.start + parts - 1) / parts;
  const int first = min(q.start + z * per, q.end);
  Rows r{q.drafts ? p.draft + first : nullptr, nullptr, first,
         min(q.end - first, per)};
  if (p.mask && p.mask_rows) {
    r.mask_row = p.mask_rows + first;
    if (r.count <= kRows) {
      if (int(threadIdx.x) < r.count)
        row_mask[threadIdx.x] = r.mask_row[threadIdx.x];
      r.mask_row = row_mask;
    }
  }
  if (q.drafts && r.count <= kRows) {
    if (int(threadIdx.x) < r.count)
      row_draft[threadIdx.x] = p.draft[first + threadIdx.x];
    r.draft = row_draft;
  }
  return r;
}

// What a workgroup has in LDS besides the table or the slice.
struct Small {
  int touched, found[kThreads / 64];
  int32_t row_draft[kRows], row_mask[kRows];
  uint16_t over[kThreads];
};

// Request b, part z of its window, by the table if it takes its tokens.
template <bool BF16>
__device__ __forceinline__ void adjust_by_table(const LogitsParams& p, int b,
                                                int z, uint32_t* lds,
                                                Small& sm) {
  const int tid = threadIdx.x;
  const Request q(p, b);
  if (q.idle() || !q.fits()) return;
  const Rows r = part_of(p, q, z, p.parts, sm.row_draft, sm.row_mask);
  if (r.count <= 0) return;
  int& touched = sm.touched;
  const Change& c = q.c;
  const int first = r.first, end = first + r.count;

  uint32_t* key = lds;                       // a token plus one; 0: free
  uint32_t* word = lds + kPlaces;
  uint16_t* list = reinterpret_cast<uint16_t*>(lds + 2 * kPlaces);
  uint32_t* biased = lds + 2 * kPlaces + kPlaces / 2;
  for (int i = tid; i < kPlaces / 4; i += kThreads) {
    reinterpret_cast<u4*>(key)[i] = u4{0, 0, 0, 0};
    reinterpret_cast<u4*>(word)[i] = u4{0, 0, 0, 0};
    if (p.bias_start) reinterpret_cast<u4*>(biased)[i] = u4{0, 0, 0, 0};
  }
  if (tid == 0) touched = 0;
  __syncthreads();
  // the place of a token, taken for it if it is new; at most kMost tokens
  // come, so there is always a free one
  auto place_of = [&](int token) -> int {
    if (uint32_t(token) >= uint32_t(p.V)) return -1;
    const uint32_t k = uint32_t(token) + 1;
    uint32_t at = (k * 2654435761u) >> 19;
    while (true) {
      const uint32_t had = atomicCAS(&key[at], 0u, k);
      if (had == 0) list[atomicAdd(&touched, 1)] = uint16_t(at);
      if (had == 0 || had == k) return int(at);
      at = (at + 1) % kPlaces;
    }
  };
  for (int i = tid; i < q.known; i += kThreads) {
    const int at = place_of(q.history[i]);
    if (at < 0) continue;
    if (i < q.prompt)
      atomicOr(&word[at], kSeen);
    else
      atomicAdd(&word[at], 1u);
  }
  if (q.drafts)
    for (int i = q.start + 1 + tid; i < end; i += kThreads) {
      const int at = place_of(p.draft[i]);
      if (at >= 0 && i <= first) atomicAdd(&word[at], 1u);
    }
  for (int i = tid; i < c.n; i += kThreads) {
    const int at = place_of(c.tokens[i]);
    if (at >= 0) atomicMax(&biased[at], uint32_t(i) + 1);
  }
  __syncthreads();
  change_listed<BF16>(
      p, c, r, touched, [&](int i) { return int(key[list[i]]) - 1; },
      [&](int i) { return word[list[i]]; },
      [&](int i) { return c.n > 0 ? biased[list[i]] : 0u; });
}

// Requests that the table does not take: each of `count` workgroups looks all
// requests over and lists them, and the items (request, part of its window,
// slice of the vocabulary) go round the workgroups.
template <bool BF16>
__device__ __forceinline__ void adjust_by_slices(const LogitsParams& p,
                                                 int number, int count,
                                                 uint32_t* lds, Small& sm) {
  uint32_t* words = lds;
  uint32_t* biased = lds + kSlice;
  uint16_t* list = reinterpret_cast<uint16_t*>(lds + 2 * kSlice);
  int& touched = sm.touched;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slices = (p.V + kSlice - 1) / kSlice, each = slices * p.parts;
  // (few requests: an item each, whether the table takes it or not, without
  // the list, which costs a second look at the request)
  const bool few = int64_t(p.B) * each <= count;
  int64_t next = number;                     // this workgroup's next item
  int64_t done = 0;                          // items of the requests before b0
  for (int b0 = 0; b0 < p.B; b0 += kThreads) {
    int all = p.B;
    if (!few) {
      bool mine = false;
      if (b0 + tid < p.B) {
        const Request q(p, b0 + tid);
        mine = !q.idle() && !q.fits();
      }
      const uint64_t m = __ballot(mine);
      __syncthreads();                       // the last list is done
      if (lane == 0) sm.found[wave] = __popcll(m);
      __syncthreads();
      int at = __popcll(m & ((uint64_t(1) << lane) - 1));
      all = 0;
      for (int k = 0; k < kThreads / 64; ++k) {
        at += k < wave ? sm.found[k] : 0;
        all += sm.found[k];
      }
      if (mine) sm.over[at] = uint16_t(tid);
      __syncthreads();
    }
    const int64_t end_item = done + int64_t(all) * each;
    for (; next < end_item; next += count) {
      const int in = int(next - done);       // (of 1024 requests: 2^24 at most)
      const int k = in / each, item = in - k * each;
      const int z = item / slices, v0 = (item - z * slices) * kSlice;
      const int nv = min(p.V - v0, kSlice);
      const Request q(p, b0 + (few ? k : sm.over[k]));
      if (few && (q.idle() || q.fits())) continue;
      __syncthreads();                       // the last item is done
      const Rows r = part_of(p, q, z, p.parts, sm.row_draft,
                             sm.row_mask);
      if (r.count <= 0) continue;
      const Change& c = q.c;
      const int first = r.first, end = first + r.count;
      for (int i = tid; i < kSlice / 4; i += kThreads) {
        reinterpret_cast<u4*>(words)[i] = u4{0, 0, 0, 0};
        reinterpret_cast<u4*>(biased)[i] = u4{0, 0, 0, 0};
      }
      if (tid == 0) touched = 0;
      __syncthreads();
      for (int i = tid; i < q.known; i += kThreads) {
        const uint32_t at = uint32_t(q.history[i]) - uint32_t(v0);
        if (at >= uint32_t(nv)) continue;
        if (i < q.prompt)
          atomicOr(&words[at], kSeen);
        else
          atomicAdd(&words[at], 1u);
      }
      if (q.drafts)
        for (int i = q.start + 1 + tid; i < end; i += kThreads) {
          const uint32_t at = uint32_t(p.draft[i]) - uint32_t(v0);
          if (at >= uint32_t(nv)) continue;
          if (i <= first)
            atomicAdd(&words[at], 1u);
          else
            atomicOr(&words[at], kListed);
        }
      for (int i = tid; i < c.n; i += kThreads) {
        const uint32_t at = uint32_t(c.tokens[i]) - uint32_t(v0);
        if (at < uint32_t(nv)) atomicMax(&biased[at], uint32_t(i) + 1);
      }
      __syncthreads();
      for (int i = tid; i < nv; i += kThreads)
        if (words[i] | biased[i]) list[atomicAdd(&touched, 1)] = uint16_t(i);
      __syncthreads();
      change_listed<BF16>(
          p, c, r, touched, [&](int i) { return v0 + list[i]; },
          [&](int i) { return words[list[i]]; },
          [&](int i) { return biased[list[i]]; });
    }
    done = end_item;
  }
}

// Workgroups [0, B) x parts: a part of a request each.  Those behind them take
// what the table does not.
template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    kda_adjust_logits_kernel(LogitsParams p) {
  extern __shared__ __align__(16) uint32_t lds[];
  __shared__ Small sm;
  const int x = blockIdx.x - p.B;
  if (x < 0)
    adjust_by_table<BF16>(p, blockIdx.x, blockIdx.y, lds, sm);
  else
    adjust_by_slices<BF16>(p, x * p.parts + blockIdx.y,
                           (gridDim.x - p.B) * p.parts, lds, sm);
}

// Entries that a row's mask does not allow, after the changes.
template <bool BF16>
__global__ void __launch_bounds__(kMaskThreads)
    kda_mask_logits_kernel(LogitsParams p) {
  constexpr int G = BF16 ? 8 : 4;            // entries of 16 bytes
  constexpr int U = 4, kMaskChunk = U * kMaskThreads * G;
  constexpr uint32_t all = (1u << G) - 1;
  typedef typename Act<BF16>::T E;
  const int m = p.mask_from + blockIdx.y, v0 = blockIdx.x * kMaskChunk;
  if (p.qsl && (m < p.qsl[0] || m >= p.qsl[p.B])) return;
  const int32_t* mask = mask_at(p, p.mask_rows ? p.mask_rows[m] : m);
  if (!mask) return;
  E* x = static_cast<E*>(p.logits) + m * p.s_row;
  const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0;
  uint32_t out[U];
  u4 v[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = v0 + (k * kMaskThreads + int(threadIdx.x)) * G;
    out[k] = i < p.V ? ~(uint32_t(mask[i >> 5]) >> (i & 31)) & all : 0u;
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = v0 + (k * kMaskThreads + int(threadIdx.x)) * G;
    v[k] = u4{0, 0, 0, 0};
    if (out[k] && out[k] != all && wide && i + G <= p.V)
      v[k] = *reinterpret_cast<const u4*>(x + i);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = v0 + (k * kMaskThreads + int(threadIdx.x)) * G;
    if (!out[k]) continue;
    if (wide && i + G <= p.V) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          const uint32_t lo = (out[k] >> (2 * j)) & 1,
                         hi = (out[k] >> (2 * j + 1)) & 1;
          const uint32_t part = ((0u - lo) & 0xffffu) | (0u - hi) << 16;
          v[k][j] = (v[k][j] & ~part) | (0xff80ff80u & part);
        } else {
          if ((out[k] >> j) & 1) v[k][j] = 0xff800000u;
        }
      }
      *reinterpret_cast<u4*>(x + i) = v[k];
    } else {
      for (int j = 0; j < G && i + j < p.V; ++j)
        if ((out[k] >> j) & 1) st_elem(x, i + j, -INFINITY, BF16);
    }
  }
}

}  // namespace

namespace {
template <bool BF16>
int launch(const LogitsParams& p, hipStream_t stream) {
  if (p.rep || p.freq || p.pres || p.bias_start) {
    // a workgroup takes some 16 rows of an average window
    const int64_t rows = (int64_t(p.M) / p.B + 15) / 16;
    LogitsParams q = p;
    q.parts = rows < 1 ? 1 : rows > 64 ? 64 : int32_t(rows);
    // Lengths are on the GPU.  Where the longest history, all biases and all
    // drafts fit the table no request exceeds it; else there are workgroups for
    // those that do, one a CU (256 requests of 3000 tokens in rows of 3001: 53
    // us; in rows of 8192 and more: 53 us, 404 with 32 workgroups a request)
    int64_t pool = 0;
    if (int64_t(p.L) + p.num_bias + p.M > kMost) {
      const int64_t items = int64_t(p.B) * q.parts *
                            ((p.V + kSlice - 1) / kSlice);
      pool = ((items < kPool ? items : kPool) + q.parts - 1) / q.parts;
    }
    constexpr int lds = (3 * kPlaces + kPlaces / 2) * 4;
    static_assert(lds - kPlaces * 4 >= (2 * kSlice + kSlice / 2) * 4 &&
                  lds + sizeof(Small) <= 160 * 1024, "LDS");
    const auto kernel = kda_adjust_logits_kernel<BF16>;
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kernel),
        hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return int(e);
    launch_kernel(kernel, dim3(uint32_t(p.B + pool), q.parts), dim3(kThreads),
                  p.bias_start ? lds : lds - kPlaces * 4, stream, q);
  }
  if (p.mask) {
    constexpr int kMaskChunk = 4 * kMaskThreads * (BF16 ? 8 : 4);
    LogitsParams q = p;
    // (rows in launches of what a grid takes)
    for (int64_t m = 0; m < p.M; m += kMaskRows) {
      q.mask_from = int32_t(m);
      const int64_t n = p.M - m < kMaskRows ? p.M - m : kMaskRows;
      launch_kernel(kda_mask_logits_kernel<BF16>,
                    dim3((p.V - 1) / kMaskChunk + 1, uint32_t(n)),
                    dim3(kMaskThreads), 0, stream, q);
    }
  }
  return int(hipGetLastError());
}
}  // namespace

int launch_adjust_logits(const LogitsParams& p, bool bf16,
                         hipStream_t stream) {
  return bf16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

}  // namespace kda
