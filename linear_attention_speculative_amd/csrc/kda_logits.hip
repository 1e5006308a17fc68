// Changes of logits in front of the sampling on gfx950: biases, penalties for
// repeated tokens and grammar masks, in place.
//
//   y = x + bias;  seen token: y > 0 ? y / r : y r;  count > 0: y - f count - p;
//   not allowed: -inf.
//
// `count` is how often a token was produced: the history behind the prompt,
// and in a draft window the drafts up to the row.  Nothing is kept between
// calls: one workgroup takes a request and a slice of the vocabulary, counts
// the slice's tokens of the history in LDS (integer atomics: no order changes
// a count) and goes through the rows of the request's window, one more draft
// counted for each.  Only entries that change are read and written: a row
// without a mask costs the entries of its history, a masked one its writes.
//
// One word of LDS a token: a bias, the prompt's tokens and the count.  The
// bias itself is looked up in the request's list when a token has one, from
// the end (the last of several counts).
#include "kda_cache.hpp"
#include "kda_mma.hpp"

namespace kda {
namespace {

constexpr int kSlice = 8192;       // tokens of a workgroup
constexpr int kThreads = 512;
constexpr uint32_t kSeen = 1u << 31, kBiased = 1u << 30, kCount = kBiased - 1;

struct Change {
  float r, f, p;
  const int32_t* tokens;           // the request's biases
  const float* values;
  int n;
};

__device__ __forceinline__ float bias_of(const Change& c, int token) {
  for (int i = c.n - 1; i >= 0; --i)
    if (c.tokens[i] == token) return c.values[i];
  return 0.0f;
}

__device__ __forceinline__ float change(const Change& c, float y, uint32_t w,
                                        int token) {
  if (w & kBiased) y += bias_of(c, token);
  if (w & (kSeen | kCount)) y = y > 0.0f ? y / c.r : y * c.r;
  if (w & kCount) y = y - c.f * float(w & kCount) - c.p;
  return y;
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads)
    kda_adjust_logits_kernel(LogitsParams p) {
  constexpr int G = BF16 ? 8 : 4;            // entries of 16 bytes
  typedef typename Act<BF16>::T E;
  __shared__ __align__(16) uint32_t words[kSlice];
  const int tid = threadIdx.x, b = blockIdx.y;
  const int v0 = blockIdx.x * kSlice, nv = min(p.V - v0, kSlice);
  int m0 = b, m1 = b + 1;
  if (p.qsl) {
    m0 = min(max(p.qsl[b], 0), p.M);
    m1 = min(max(p.qsl[b + 1], m0), p.M);
  }
  // a window of many rows is shared: rows [first, m1) are this workgroup's
  const int per = (m1 - m0 + int(gridDim.z) - 1) / int(gridDim.z);
  const int first = m0 + int(blockIdx.z) * per;
  const int start = m0;
  m1 = min(m1, first + per);
  if (first >= m1) return;

  Change c{1.0f, 0.0f, 0.0f, nullptr, nullptr, 0};
  if (p.rep) c.r = p.rep[b];
  if (p.freq) c.f = p.freq[b];
  if (p.pres) c.p = p.pres[b];
  if (!(c.r > 0.0f)) c.r = 1.0f;             // (NaN, too)
  if (c.f != c.f) c.f = 0.0f;
  if (c.p != c.p) c.p = 0.0f;
  if (p.bias_start) {
    const int lo = min(max(p.bias_start[b], 0), p.num_bias);
    c.n = min(max(p.bias_start[b + 1], lo), p.num_bias) - lo;
    c.tokens = p.bias_tokens + lo;
    c.values = p.bias_values + lo;
  }
  const bool counts = c.r != 1.0f || c.f != 0.0f || c.p != 0.0f;
  const bool any = counts || c.n > 0;
  if (!any && !p.mask) return;

  if (any) {
    for (int i = tid; i < kSlice / 4; i += kThreads)
      reinterpret_cast<u4*>(words)[i] = u4{0, 0, 0, 0};
    __syncthreads();
    if (counts && p.tokens) {
      const int row = p.req_idx ? p.req_idx[b] : b;
      if (row >= 0 && row < p.rows) {
        const int32_t* t = p.tokens + row * p.s_tok;
        const int known = min(max(p.known[row], 0), p.L);
        const int prompt = p.prompt[row];
        for (int i = tid; i < known; i += kThreads) {
          const uint32_t at = uint32_t(t[i]) - uint32_t(v0);
          if (at < uint32_t(nv)) {
            if (i < prompt)
              atomicOr(&words[at], kSeen);
            else
              atomicAdd(&words[at], 1u);
          }
        }
      }
    }
    for (int i = tid; i < c.n; i += kThreads) {
      const uint32_t at = uint32_t(c.tokens[i]) - uint32_t(v0);
      if (at < uint32_t(nv)) atomicOr(&words[at], kBiased);
    }
    if (counts && p.draft)
      for (int i = start + 1 + tid; i <= first; i += kThreads) {
        const uint32_t at = uint32_t(p.draft[i]) - uint32_t(v0);
        if (at < uint32_t(nv)) atomicAdd(&words[at], 1u);
      }
    __syncthreads();
  }

  for (int m = first; m < m1; ++m) {
    if (m > first && counts && p.draft) {
      __syncthreads();
      const uint32_t at = uint32_t(p.draft[m]) - uint32_t(v0);
      if (tid == 0 && at < uint32_t(nv)) ++words[at];
      __syncthreads();
    }
    E* x = static_cast<E*>(p.logits) + m * p.s_row + v0;
    const int32_t* mask = nullptr;
    if (p.mask) {
      const int mr = p.mask_rows ? p.mask_rows[m] : m;
      if (mr >= 0 && mr < p.num_masks)
        mask = p.mask + mr * p.s_mask + v0 / 32;
    }
    if (!any && !mask) continue;
    const bool wide = reinterpret_cast<uintptr_t>(x) % 16 == 0;
    for (int i = tid * G; i < nv; i += kThreads * G) {
      uint32_t w[G], changed = 0;
#pragma unroll
      for (int k = 0; k < G; ++k) w[k] = 0;
      if (any) {
#pragma unroll
        for (int k = 0; k < G; k += 4) {
          const u4 q = *reinterpret_cast<const u4*>(words + i + k);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[k + j] = q[j];
        }
#pragma unroll
        for (int k = 0; k < G; ++k) changed |= w[k] ? 1u << k : 0u;
      }
      constexpr uint32_t all = (1u << G) - 1;
      uint32_t out = 0;                      // entries that are masked
      if (mask) out = ~(uint32_t(mask[i >> 5]) >> (i & 31)) & all;
      if (!(changed | out)) continue;
      changed &= ~out;
      if (wide && i + G <= nv) {
        u4 v = {0, 0, 0, 0};
        if (out != all) v = *reinterpret_cast<const u4*>(x + i);
#pragma unroll
        for (int k = 0; k < G; ++k) {
          float y = BF16 ? bf16_to_f32(uint16_t(v[k / 2] >> (k % 2 * 16)))
                         : __uint_as_float(v[BF16 ? 0 : k]);
          if ((changed >> k) & 1) y = change(c, y, w[k], v0 + i + k);
          if ((out >> k) & 1) y = -INFINITY;
          if (!(((changed | out) >> k) & 1)) continue;
          if constexpr (BF16)
            v[k / 2] = (v[k / 2] & (0xffff0000u >> (k % 2 * 16))) |
                       (uint32_t(f32_to_bf16(y)) << (k % 2 * 16));
          else
            v[k] = __float_as_uint(y);
        }
        *reinterpret_cast<u4*>(x + i) = v;
      } else {
        for (int k = 0; k < G && i + k < nv; ++k) {
          if ((out >> k) & 1)
            st_elem(x, i + k, -INFINITY, BF16);
          else if ((changed >> k) & 1)
            st_elem(x, i + k,
                    change(c, ld_elem(x, i + k, BF16), words[i + k],
                           v0 + i + k),
                    BF16);
        }
      }
    }
  }
}

}  // namespace

int64_t logits_slices(int64_t V) { return (V + kSlice - 1) / kSlice; }

int launch_adjust_logits(const LogitsParams& p, bool bf16,
                         hipStream_t stream) {
  // a workgroup takes some 16 rows of an average window
  const int64_t z = (int64_t(p.M) / p.B + 15) / 16;
  const dim3 grid(uint32_t(logits_slices(p.V)), p.B,
                  uint32_t(z < 1 ? 1 : z > 64 ? 64 : z));
  if (bf16)
    launch_kernel(kda_adjust_logits_kernel<true>, grid, dim3(kThreads), 0,
                  stream, p);
  else
    launch_kernel(kda_adjust_logits_kernel<false>, grid, dim3(kThreads), 0,
                  stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
