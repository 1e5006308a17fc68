// KDA layer over prompts for gfx950, in the chunked form: chunks of C = 32
// tokens turn the token-by-token recurrence into matrix products.
//
// Inside a chunk, with G_t the sum of the log-decays up to token t (per
// channel), k_t and q_t normalised, and S_0 the state before the chunk:
//   A_tj = sum_k k_tk k_jk e^(G_tk - G_jk)  (j < t)
//   B_tj = sum_k q_tk k_jk e^(G_tk - G_jk)  (j <= t)
//   T    = (I + diag(beta) A)^-1 diag(beta)
//   c    = T (V - (k e^G) S_0^T)            corrections of all 32 tokens
//   O    = (q e^G) S_0^T + B c
//   S_C  = S_0 diag(e^G_C) + c^T (k e^(G_C - G))
// Only the last three lines need S_0.  So two kernels:
//
//   kda_prefill_chunk_kernel: one workgroup per (chunk, head), all chunks at
//   once: convolution, norms, gates, A, B, T and the scaled k and q, written
//   to the workspace in the order in which the second kernel's lanes hold
//   matrix operands (one 16-byte load per lane and operand).
//
//   kda_prefill_state_kernel: one wave per (request, head, 16 state rows),
//   chunk after chunk.  The rows v of the state never mix, so a wave keeps
//   its 16 rows for all channels in 4 D/16 registers per lane, never in LDS:
//   the result layout of one product (column on lane % 16, four rows per lane
//   group) serves as the right operand of the next one if the summed index is
//   taken in the order 4 g + e (e < 4), 16 + 4 g + e - 4, g = lane / 16, on
//   both sides.  LDS holds what the waves of a workgroup share, the operands
//   of the next chunks, brought by waves that do nothing else: issuing a load
//   to LDS takes a wave some 50 cycles, which the others then do not spend.
//
// What bounds them, on 8192 tokens of 32 heads of D = 128 (bf16): the chunk
// kernel, 230 us, its vector arithmetic and memory (0.27 GB read and 0.6 GB
// written: 175 us at a copy's rate); the state kernel, 415 us, the length of
// one chunk's chain of products, 1.6 us times 256 chunks, with one wave to
// each SIMD that has any.  16 prompts of 16000 tokens together: 439 and 308 us.
//
// Decays never divide: every exponent above is a sum over tokens between j
// and t, so each factor is at most 1, however strong the gates.  Within 16
// tokens products e^(G_t - G_j) are carried from j to t by multiplication;
// the block of later rows and earlier columns splits at its border into two
// factors of at most 1 each, which a matrix product takes.
//
// Rounding: states, sums and the triangular inverse are fp32.  The operands
// of the second kernel's products are pairs of fp16 (x = hi + lo, 22 bits)
// under a power-of-two scale, three products each, which loses 2^-22 of a
// term: fp32-like, at a third of the fp16 matrix rate instead of the
// sixteenth that fp32 operands have.  k e^G and the like are at most 1 and
// take fixed scales; each column of S, with its V, r and c, has a scale of
// its own that follows its largest element: errors go by the largest value
// that a column of S, or its V, has within a chunk.  Of a column that a chunk
// decays to e^G of itself, with G below some -20, and that no V joins, the
// corrections that remain (e^G or less each) keep fewer bits, down to none.
// The products behind bf16 outputs are as exact: an output is what two terms
// leave, and where the delta rule replaces what the state held, it can be far
// smaller than they are.  (With the high halves alone, 2^-11 of each term, the
// two kernels took 223 and 364 us, and outputs were off by many bf16 steps.)
#include "kda_serving.hpp"

namespace kda {
namespace {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h4 __attribute__((ext_vector_type(4)));

constexpr int C = kChunk;
constexpr int kSub = 16;             // tokens of a sub-block
constexpr float kUnit = 4096.0f;     // scale of operands of at most 1
constexpr float kLate = 32.0f;       // scale of k e^(G_C - G)
constexpr int kFrag = 1024;          // bytes of one operand (64 lanes x 16)

// Workspace of one (chunk slot, head): byte offsets of its operands.
template <int D>
struct Work {
  static constexpr int KS = D >= 32 ? D / 32 : 1;  // channel steps of 32
  static constexpr int MT = D / 16;                // state row tiles
  static constexpr int kd = 0;                     // [2][KS] hi, lo
  static constexpr int ke = kd + 2 * KS * 2 * kFrag;   // [MT] hi, lo
  static constexpr int t = ke + MT * 2 * kFrag;        // [2] hi, lo
  static constexpr int v = t + 2 * 2 * kFrag;          // [2][MT] fp32
  static constexpr int gam = v + 2 * MT * kFrag;       // [D] fp32
  static constexpr int qd = gam + (D * 4 + kFrag - 1) / kFrag * kFrag;
  static constexpr int b = qd + 2 * KS * 2 * kFrag;    // q e^G, then B: [2]
  static constexpr int size = b + 2 * 2 * kFrag;       // hi, lo
};

struct Split {
  h8 hi, lo;
};

// Both halves are taken from one fp32 value.  It is made opaque first: where
// the compiler sees the product that x comes from, it may round that product
// to fp16 once, without the fp32 step, for one half and not for the other,
// and in a tie hi + lo is then a whole fp16 step off.
__device__ __forceinline__ Split split8(float (&x)[8]) {
  Split s;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    asm("" : "+v"(x[e]));
    s.hi[e] = _Float16(x[e]);
    s.lo[e] = _Float16(x[e] - float(s.hi[e]));
  }
  return s;
}

__device__ __forceinline__ void store_frag(char* at, int lane, h8 v) {
  *reinterpret_cast<h8*>(at + lane * 16) = v;
}

template <int D, bool BF16>
struct Pair;   // two neighbouring channels of an activation row
template <int D>
struct Pair<D, true> {
  typedef uint32_t T;
  static __device__ __forceinline__ float lo(T x) {
    return __uint_as_float(x << 16);
  }
  static __device__ __forceinline__ float hi(T x) {
    return __uint_as_float(x & 0xffff0000u);
  }
};
template <int D>
struct Pair<D, false> {
  typedef float2 T;
  static __device__ __forceinline__ float lo(T x) { return x.x; }
  static __device__ __forceinline__ float hi(T x) { return x.y; }
};

// Two workgroups fit a CU's LDS at D = 128; 512 threads each keep four waves
// on every SIMD (8192 tokens of 32 heads: 12% faster than with 256).
template <int D>
struct ChunkCfg {
  static constexpr int NT = D >= 32 ? 512 : 256;
  static constexpr int NW = NT / 64;
  static constexpr int CP = D / 2;               // channel pairs
  static constexpr int TG = NT / CP;             // token groups
  static constexpr int NTK = C / TG;             // tokens per thread
  static constexpr int RS = D + 4;               // padded row, floats
  static constexpr int AS = C + 4;
};

template <int D>
struct ChunkSmem {
  using F = ChunkCfg<D>;
  // With P_t and Q_t the products of a sub-block's decays up to token t and
  // behind it, P_end those of the whole sub-block:
  float k[C][F::RS];    // k, then k P
  float q[C][F::RS];    // q, then q P
  float z[C][F::RS];    // decays, then k Q
  float end[2][D];      // P_end
  float rend[2][D];     // 1 / P_end
  float a[C][F::AS];
  float b[C][F::AS];
  float t[C][F::AS];
  float beta[C];
  int before, all, task;
};

// Bounds of request b in the token rows, whatever the offsets hold.
__device__ __forceinline__ int2 token_range(const PrefillParams& p, int b) {
  const int bos = min(max(p.qsl[b], 0), p.T);
  return make_int2(bos, min(max(p.qsl[b + 1], bos), p.T));
}

// First chunk slot of request b.  Slots of different requests are disjoint:
// the next request starts at least ceil(length / C) later.
__device__ __forceinline__ int first_slot(int bos, int b) {
  return bos / C + b;
}

// 1 / sqrt(sum + eps) of N tokens' q and k rows, each spread in pairs over
// CP consecutive lanes.  The 2 N sums are reduced together, each lane ending
// with one of them, so that the root is taken once per row and handed back.
template <int CP, int N>
__device__ __forceinline__ void row_norms(const float (&q)[N][2],
                                          const float (&k)[N][2],
                                          float (&nq)[N], float (&nk)[N]) {
  float s[2 * N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    s[i] = q[i][0] * q[i][0] + q[i][1] * q[i][1];
    s[N + i] = k[i][0] * k[i][0] + k[i][1] * k[i][1];
  }
  if constexpr (CP >= 16) {
    constexpr int E = 16 / (2 * N);      // lanes that end with one sum
    float v = transpose_sum<16, 2 * N>(s, threadIdx.x & 15);
    if constexpr (CP >= 32)
      v += __int_as_float(
          __builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F));
    if constexpr (CP >= 64) v += __shfl_xor(v, 32);
    v = __builtin_amdgcn_rsqf(v + kNormEps);
    const int base = threadIdx.x & 48;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      nq[i] = __shfl(v, base + i * E);
      nk[i] = __shfl(v, base + (N + i) * E);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      nq[i] = __builtin_amdgcn_rsqf(group_sum<CP>(s[i]) + kNormEps);
      nk[i] = __builtin_amdgcn_rsqf(group_sum<CP>(s[N + i]) + kNormEps);
    }
  }
}

// The request that holds a chunk slot, or -1: the last one whose first slot is
// not behind it, found by every wave for itself, 64 candidates at a time.
__device__ __forceinline__ int request_of_slot(const PrefillParams& p,
                                               int slot, int lane) {
  int lo = 0, n = p.y.B;       // candidates lo .. lo + n - 1
  while (n > 1) {
    const int step = (n + 63) / 64;
    const int i = lane * step;
    const bool in = i < n && first_slot(token_range(p, lo + i).x, lo + i) <=
                                 slot;
    // (offsets that run backwards give some candidate, checked below)
    const int k = max(int(__popcll(__ballot(in))) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  const int2 r = token_range(p, lo);
  const int f = first_slot(r.x, lo);
  return slot >= f && slot < f + (r.y - r.x + C - 1) / C ? uniform(lo) : -1;
}

// Place of request b in the order of falling lengths (ties by number), written
// to the order that the state kernel takes its requests in: its workgroups
// then start with the longest ones, and the short ones fill the gaps.  Empty
// requests have no place; order[-1] counts the others.  The first workgroup
// writes the count even where it holds no request (b = -1), so that a batch
// of empty requests leaves 0 there and not what the workspace held.
template <int D>
__device__ __forceinline__ void rank_request(const PrefillParams& p, int b,
                                             ChunkSmem<D>& m) {
  const int2 mine = b < 0 ? make_int2(0, 0) : token_range(p, b);
  const int len = mine.y - mine.x;
  // counted by waves: one LDS atomic each (by lanes, all on one address, they
  // took 5 us)
  int before = 0, all = 0;
  for (int i0 = threadIdx.x & ~63; i0 < p.y.B; i0 += ChunkCfg<D>::NT) {
    const int i = i0 + int(threadIdx.x & 63);
    const bool in = i < p.y.B;
    const int2 r = token_range(p, in ? i : 0);
    const int n = r.y - r.x;
    before += __popcll(__ballot(in && (n > len || (n == len && i < b))));
    all += __popcll(__ballot(in && n > 0));
  }
  __syncthreads();           // the counters are cleared
  if ((threadIdx.x & 63) == 0) {
    atomicAdd(&m.before, before);
    atomicAdd(&m.all, all);
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (b >= 0) p.order[m.before] = b;
    if (blockIdx.x == 0) p.order[-1] = m.all;
  }
}

template <int D, bool BF16>
__global__ void __launch_bounds__(ChunkCfg<D>::NT)
    __attribute__((amdgpu_waves_per_eu(4, 4)))
    kda_prefill_chunk_kernel(PrefillParams p) {
  using F = ChunkCfg<D>;
  using W = Work<D>;
  using P2 = Pair<D, BF16>;
  typedef typename Act<BF16>::T T;
  extern __shared__ __align__(16) char smem[];
  ChunkSmem<D>& m = *reinterpret_cast<ChunkSmem<D>*>(smem);
  const LayerParams& y = p.y;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int slot = blockIdx.x / y.H, h = blockIdx.x - slot * y.H;

  if (tid == 0) m.before = m.all = m.task = 0;
  const int b = request_of_slot(p, slot, lane);
  if (b < 0) {
    if (blockIdx.x == 0) rank_request<D>(p, -1, m);
    return;
  }
  const int2 range = token_range(p, b);
  const int first = (slot - first_slot(range.x, b)) * C;   // in the request
  // (offsets that run backwards can give slot 0 to a later chunk)
  if (h == 0 && (first == 0 || slot == 0))
    rank_request<D>(p, first == 0 ? b : -1, m);
  if (!live_slot(y, y.slots[b])) return;
  const int t0 = range.x + first, n = min(C, range.y - t0);
  char* work = p.work + (int64_t(slot) * y.H + h) * W::size;

  // ---- activations: convolution, norms, gates ----
  // a wave holds whole rows at D = 128: its token rows are scalar addresses
  const int cp = tid % F::CP;
  const int tg = F::CP == 64 ? uniform(tid / F::CP) : tid / F::CP;
  const int64_t HD = int64_t(y.H) * D, ch = int64_t(h) * D + 2 * cp;
  const bool conv = !(y.flags & kNoConv);
  // Every row index is clamped into the request: the loads then stand in one
  // block, all in flight together.  What comes of rows behind the request is
  // dropped at the end (no row before them uses it).
  const int tk = tg * F::NTK;
  typename P2::T raw[3][F::NTK + 3], rawg[F::NTK];
  const T* xcol = static_cast<const T*>(y.mixed_qkv) + ch;
  const T* gcol = static_cast<const T*>(y.raw_gate) + ch;
#pragma unroll
  for (int i = 0; i < F::NTK + 3; ++i) {
    const int64_t row = t0 + min(max(tk + i - 3, -first), n - 1);
#pragma unroll
    for (int part = 0; part < 3; ++part)
      raw[part][i] = *reinterpret_cast<const typename P2::T*>(
          xcol + row * y.s_x + part * HD);
    if (i >= 3)
      rawg[i - 3] = *reinterpret_cast<const typename P2::T*>(gcol +
                                                             row * y.s_g);
  }
  float w[3][2][kConvWidth];
  if (conv) {
    if (y.flags & kWRow) {
      // four taps of a channel in one load
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int64_t o = (part * HD + ch + e) * kConvWidth;
          if (y.flags & kWBf16) {
            const uint2 u = *reinterpret_cast<const uint2*>(
                static_cast<const uint16_t*>(y.conv_weight) + o);
            w[part][e][0] = __uint_as_float(u.x << 16);
            w[part][e][1] = __uint_as_float(u.x & 0xffff0000u);
            w[part][e][2] = __uint_as_float(u.y << 16);
            w[part][e][3] = __uint_as_float(u.y & 0xffff0000u);
          } else {
            const f4 u = *reinterpret_cast<const f4*>(
                static_cast<const float*>(y.conv_weight) + o);
#pragma unroll
            for (int i = 0; i < 4; ++i) w[part][e][i] = u[i];
          }
        }
    } else {
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < kConvWidth; ++i)
            w[part][e][i] = ld_elem(
                y.conv_weight,
                (part * HD + ch + e) * y.s_w_chan + i * y.s_w_tap,
                y.flags & kWBf16);
    }
  }
  float val[3][F::NTK][2];
  const bool head = first == 0 && tk < 3;   // the window reaches the history
  const int src = p.initial ? p.initial[b] : -1;
#pragma unroll
  for (int part = 0; part < 3; ++part) {
    float x[F::NTK + 3][2];
#pragma unroll
    for (int i = 0; i < F::NTK + 3; ++i) {
      x[i][0] = P2::lo(raw[part][i]);
      x[i][1] = P2::hi(raw[part][i]);
    }
    if (conv) {
      if (head) {
        const bool from = live_slot(y, src);
        const T* cs = static_cast<const T*>(y.conv_state) +
                      (part * HD + ch) * y.s_cs_chan;
        if (from) cs += src * y.s_cs_slot + history_at(y, b) * y.s_cs_tok;
#pragma unroll
        for (int i = 0; i < 3; ++i)
          if (tk + i < 3) {
            x[i][0] = from ? Act<BF16>::f(cs[(tk + i) * y.s_cs_tok]) : 0.0f;
            x[i][1] = from ? Act<BF16>::f(cs[y.s_cs_chan +
                                             (tk + i) * y.s_cs_tok])
                           : 0.0f;
          }
      }
#pragma unroll
      for (int i = 0; i < F::NTK; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float acc = w[part][e][0] * x[i][e];
          acc = __builtin_fmaf(w[part][e][1], x[i + 1][e], acc);
          acc = __builtin_fmaf(w[part][e][2], x[i + 2][e], acc);
          acc = __builtin_fmaf(w[part][e][3], x[i + 3][e], acc);
          val[part][i][e] = silu_(acc);
        }
    } else {
#pragma unroll
      for (int i = 0; i < F::NTK; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) val[part][i][e] = x[i + 3][e];
    }
  }
  const float A = exp_(y.A_log[h]);
  const float2 bias = *reinterpret_cast<const float2*>(y.dt_bias + ch);
  float gate[F::NTK][2];
#pragma unroll
  for (int i = 0; i < F::NTK; ++i) {
    gate[i][0] = P2::lo(rawg[i]) + bias.x;
    gate[i][1] = P2::hi(rawg[i]) + bias.y;
  }
  if (y.flags & kLowerBound) {
#pragma unroll
    for (int i = 0; i < F::NTK; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        gate[i][e] = layer_gate(gate[i][e], A, true, y.lb);
  } else {
#pragma unroll
    for (int i = 0; i < F::NTK; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        gate[i][e] = layer_gate(gate[i][e], A, false, 0.0f);
  }
  // |q|^2 and |k|^2 of the thread's tokens over the lanes of their row
  float nq[F::NTK], nk[F::NTK];
  row_norms<F::CP, F::NTK>(val[0], val[1], nq, nk);
  // rows behind the request vanish: k = q = v = 0, decay 1
  if (n < C) {
#pragma unroll
    for (int i = 0; i < F::NTK; ++i)
      if (tk + i >= n) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          val[0][i][e] = val[1][i][e] = val[2][i][e] = gate[i][e] = 0.0f;
        nq[i] = nk[i] = 0.0f;
      }
  }
#pragma unroll
  for (int i = 0; i < F::NTK; ++i) {
    const int t = tk + i;
    const float fq = nq[i] * (1.0f / sqrtf(float(D)));
    *reinterpret_cast<float2*>(&m.q[t][2 * cp]) =
        make_float2(val[0][i][0] * fq, val[0][i][1] * fq);
    *reinterpret_cast<float2*>(&m.k[t][2 * cp]) =
        make_float2(val[1][i][0] * nk[i], val[1][i][1] * nk[i]);
    *reinterpret_cast<float2*>(&m.z[t][2 * cp]) =
        make_float2(exp_(gate[i][0]), exp_(gate[i][1]));
  }
  // V as the second kernel's accumulators hold it
  char* vf = work + W::v;
  if constexpr (F::NTK >= 4) {
#pragma unroll
    for (int i = 0; i < F::NTK; i += 4)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = tk + i, d = 2 * cp + e;
        *reinterpret_cast<f4*>(
            vf + ((t / kSub * W::MT + d / 16) * 64 + (t % kSub) / 4 * 16 +
                  d % 16) * 16) = f4{val[2][i][e], val[2][i + 1][e],
                                     val[2][i + 2][e], val[2][i + 3][e]};
      }
  } else {
#pragma unroll
    for (int i = 0; i < F::NTK; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int t = tk + i, d = 2 * cp + e;
        reinterpret_cast<float*>(
            vf)[((t / kSub * W::MT + d / 16) * 64 + (t % kSub) / 4 * 16 +
                 d % 16) * 4 + t % 4] = val[2][i][e];
      }
  }
  if (tid < C)
    m.beta[tid] =
        tid < n ? sigmoid_(Act<BF16>::f(static_cast<const T*>(
                      y.raw_beta)[int64_t(t0 + tid) * y.s_beta + h]))
                : 0.0f;
  __syncthreads();

  // ---- products of decays from the sub-block's start, and to its end ----
  // a thread's channel, sub-block and, at 512 threads, half of its tokens
  constexpr int HV = F::NT >= 4 * D && 2 * D % 64 == 0 ? 2 : 1;
  constexpr int TK = kSub / HV;
  const int pc = tid % D, pb = tid / D % 2;
  const int half = HV == 2 ? uniform(tid / (2 * D)) : 0;   // of whole waves
  const int t1 = half * TK;
  const bool scans = tid < 2 * D * HV;
  float pre[TK], suf[TK], full = 1.0f;
  if (scans) {
    float d[kSub];
#pragma unroll
    for (int i = 0; i < kSub; ++i) d[i] = m.z[pb * kSub + i][pc];
    // products over the thread's tokens and, from there on, over the others
    const auto scan = [&](auto first) {
      constexpr int t0 = decltype(first)::value;
      float f = 1.0f, l = 1.0f;
#pragma unroll
      for (int i = 0; i < t0; ++i) f *= d[i];
#pragma unroll
      for (int i = 0; i < TK; ++i) pre[i] = f *= d[t0 + i];
#pragma unroll
      for (int i = kSub - 1; i >= t0 + TK; --i) l *= d[i];
      full = f * l;
#pragma unroll
      for (int i = TK - 1; i >= 0; --i) {
        suf[i] = l;
        l *= d[t0 + i];
      }
    };
    if (half == 0)
      scan(std::integral_constant<int, 0>{});
    else
      scan(std::integral_constant<int, HV == 2 ? TK : 0>{});
  }
  // Within a sub-block, e^(G_i - G_j) = (P_i / P_end) Q_j as long as no P
  // leaves the fp32 range (down to 1e-37: 16 tokens of log-decay -5 each stay
  // inside): A and B are then fp32 matrix products.  Where a channel decays
  // further, the sub-blocks are done by carrying k_j e^(G_i - G_j) from row to
  // row, which takes any decay (all chunks of 8192 tokens and 32 heads: 290 us
  // for the kernel in place of 232).
  const bool deep = __syncthreads_or(!(full >= 1e-37f));
  if (deep) {
    // waves 2 sb + half; a lane takes four columns j and D/32 channels
    if (wave < 4) {
      constexpr int CH = D >= 32 ? D / 32 : 1;
      const int sb = wave >> 1, cl = lane & 31;
      const int jg = (wave & 1) ? 1 + (lane >> 5) : 3 * (lane >> 5);
      const int r0 = sb * kSub;
      const bool on = cl * CH < D;
      const int c0 = on ? cl * CH : 0;
      float kd[4][CH] = {};
#pragma unroll 1
      for (int i = 0; i < kSub; ++i) {
        float ai[CH], ki[CH], qi[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          ai[e] = m.z[r0 + i][c0 + e];
          ki[e] = on ? m.k[r0 + i][c0 + e] : 0.0f;
          qi[e] = on ? m.q[r0 + i][c0 + e] : 0.0f;
        }
        float sum[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[j] = sum[4 + j] = 0.0f;
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            kd[j][e] = i == 4 * jg + j ? ki[e] : kd[j][e] * ai[e];
            sum[j] = __builtin_fmaf(ki[e], kd[j][e], sum[j]);
            sum[4 + j] = __builtin_fmaf(qi[e], kd[j][e], sum[4 + j]);
          }
        }
        float tot = transpose_sum<16, 8>(sum, lane & 15);
        tot += __int_as_float(
            __builtin_amdgcn_ds_swizzle(__float_as_int(tot), 0x401F));
        const int v = (lane & 15) >> 1, j = 4 * jg + (v & 3);
        if ((lane & 17) == 0) {
          if (v >= 4)
            m.b[r0 + i][r0 + j] = tot;
          else
            m.a[r0 + i][r0 + j] = i > j ? tot : 0.0f;
        }
      }
    }
    __syncthreads();
  }
  if (scans) {
    // the column's k, q and decays make way for k P, q P and k Q
#pragma unroll
    for (int i = 0; i < TK; ++i) {
      const int t = pb * kSub + t1 + i;
      const float kv = m.k[t][pc];
      m.k[t][pc] = kv * pre[i];
      m.q[t][pc] *= pre[i];
      m.z[t][pc] = kv * suf[i];
    }
    if (t1 == 0) {
      m.end[pb][pc] = full;
      m.rend[pb][pc] = rcp_(full);
    }
  }
  __syncthreads();

  const int col = lane & 15, g = lane >> 4;
  // One 16 x 16 block of A (rows k P) or B (rows q P) as a matrix product: a
  // diagonal block (divided by P_end), or the one of rows 16.. and columns
  // ..15, whose decays split at its border into two factors of at most 1.
  // Lanes take the summed channels in the order 16 u + 4 g + i.
  auto block = [&](const float (*rows)[F::RS], float (*dst)[F::AS], int r0,
                   int c0, bool strict) {
    const bool diag = r0 == c0;
    f4 acc = {0, 0, 0, 0}, acc2 = {0, 0, 0, 0};
#pragma unroll
    for (int u = 0; u < D / 16; ++u) {
      const int c = 16 * u + 4 * g;
      f4 x = *reinterpret_cast<const f4*>(&rows[r0 + col][c]);
      const f4 z = *reinterpret_cast<const f4*>(&m.z[c0 + col][c]);
      if (diag)
        x *= *reinterpret_cast<const f4*>(&m.rend[r0 / kSub][c]);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i], z[i], acc, 0, 0, 0);
        acc2 = __builtin_amdgcn_mfma_f32_16x16x4f32(x[i + 1], z[i + 1], acc2,
                                                    0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * g + i;
      const bool in = !diag || (strict ? r > col : r >= col);
      dst[r0 + r][c0 + col] = in ? acc[i] + acc2[i] : 0.0f;
    }
  };
#pragma unroll 1
  for (int i = wave; i < (deep ? 2 : 6); i += F::NW) {
    const int r0 = i == 4 || i == 5 ? 0 : kSub;       // off, off, 1, 1, 0, 0
    if (i & 1)
      block(m.q, m.b, r0, i < 2 ? 0 : r0, false);
    else
      block(m.k, m.a, r0, i < 2 ? 0 : r0, true);
  }
  __syncthreads();

  if (wave == 0) {
    // T: the two diagonal inverses by substitution (lane = column), then the
    // block below them, -X2 (beta A21) X1, by products
    const int blk = (lane >> 4) & 1, r0 = blk * kSub;
    float x[kSub];
    f4 row[4] = {}, next[4];
    float bt = m.beta[r0];
#pragma unroll
    for (int i = 0; i < kSub; ++i) {
      // the next row travels while this one is used
      const float bn = i + 1 < kSub ? m.beta[r0 + i + 1] : 0.0f;
#pragma unroll
      for (int j = 0; j < (i + 4) / 4; ++j)
        if (i + 1 < kSub)
          next[j] = *reinterpret_cast<const f4*>(&m.a[r0 + i + 1][r0 + 4 * j]);
      float acc = 0.0f, acc2 = 0.0f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        float& s = j % 2 ? acc2 : acc;
        s = __builtin_fmaf(row[j / 4][j % 4], x[j], s);
      }
      x[i] = (i == col ? 1.0f : 0.0f) - bt * (acc + acc2);
      // finish this row here: otherwise every row of A is loaded up front,
      // into 120 registers
      asm volatile("" : "+v"(x[i]) : : "memory");
      bt = bn;
#pragma unroll
      for (int j = 0; j < 4; ++j) row[j] = next[j];
    }
    // lanes 32.. repeat lanes ..31 and write the same values
    const float scale = blk ? 1.0f : m.beta[col];
#pragma unroll
    for (int i = 0; i < kSub; ++i) m.t[r0 + i][r0 + col] = x[i] * scale;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
    f4 yv = {0, 0, 0, 0}, z = {0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
      yv = __builtin_amdgcn_mfma_f32_16x16x4f32(
          m.beta[kSub + col] * m.a[kSub + col][4 * s + g], m.t[4 * s + g][col],
          yv, 0, 0, 0);
#pragma unroll
    for (int s = 0; s < 4; ++s)       // summed index 4 g + s on both sides
      z = __builtin_amdgcn_mfma_f32_16x16x4f32(
          m.t[kSub + col][kSub + 4 * g + s], yv[s], z, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) m.t[kSub + 4 * g + i][col] = -z[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup", "local");
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = kUnit * m.t[r * kSub + col][4 * g + e];
        v[4 + e] = r == 0 ? 0.0f
                          : kUnit * m.t[kSub + col][kSub + 4 * g + e] *
                                m.beta[kSub + 4 * g + e];
      }
      const Split s = split8(v);
      store_frag(work + W::t + 2 * r * kFrag, lane, s.hi);
      store_frag(work + W::t + (2 * r + 1) * kFrag, lane, s.lo);
    }
  } else if (wave == 1) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[e] = kUnit * m.b[r * kSub + col][4 * g + e];
        v[4 + e] = r == 0 ? 0.0f : kUnit * m.b[kSub + col][kSub + 4 * g + e];
      }
      const Split s = split8(v);
      store_frag(work + W::b + 2 * r * kFrag, lane, s.hi);
      store_frag(work + W::b + (2 * r + 1) * kFrag, lane, s.lo);
    }
  }
  // scaled k and q, handed out as the waves become free
  constexpr int NKD = 2 * W::KS;
  for (;;) {
    int task = 0;
    if (lane == 0) task = atomicAdd(&m.task, 1);
    task = uniform(task);
    if (task >= NKD + W::MT) break;
    float x[8], z[8];
    if (task < NKD) {
      const int r = task / W::KS, s = task - r * W::KS, t = r * kSub + col;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = 32 * s + (e < 4 ? 4 * g + e : 16 + 4 * g + e - 4);
        x[e] = z[e] = 0.0f;
        if (c < D) {
          const float d = r ? kUnit * m.end[0][c] : kUnit;
          x[e] = m.k[t][c] * d;
          z[e] = m.q[t][c] * d;
        }
      }
      const Split a = split8(x), q = split8(z);
      store_frag(work + W::kd + 2 * task * kFrag, lane, a.hi);
      store_frag(work + W::kd + (2 * task + 1) * kFrag, lane, a.lo);
      store_frag(work + W::qd + 2 * task * kFrag, lane, q.hi);
      store_frag(work + W::qd + (2 * task + 1) * kFrag, lane, q.lo);
    } else {
      const int mt = task - NKD, c = 16 * mt + col;
      const float late = m.end[1][c];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int t = e < 4 ? 4 * g + e : kSub + 4 * g + e - 4;
        x[e] = kLate * m.z[t][c] * (e < 4 ? late : 1.0f);
      }
      const Split a = split8(x);
      store_frag(work + W::ke + 2 * mt * kFrag, lane, a.hi);
      store_frag(work + W::ke + (2 * mt + 1) * kFrag, lane, a.lo);
    }
  }
  if (tid < D)
    reinterpret_cast<float*>(work + W::gam)[tid] =
        m.end[0][tid] * m.end[1][tid];
}

// ---- second kernel ----------------------------------------------------------

__device__ __forceinline__ f4 mfma(h8 a, h8 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Largest value over the four lanes that share a column.
__device__ __forceinline__ float column_max(float v) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const float w = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t x = __float_as_uint(w);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// hi and lo of eight scaled values.  hi is made opaque before it is widened
// again: left visible, the compiler recomputes it with a fused instruction of
// half the rate.
__device__ __forceinline__ Split split_wide(const float (&x)[8]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  u4 hi, lo;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const h2 h = {_Float16(x[2 * e]), _Float16(x[2 * e + 1])};
    uint32_t u = __builtin_bit_cast(uint32_t, h);
    asm("" : "+v"(u));
    hi[e] = u;
    const h2 k = __builtin_bit_cast(h2, u);
    const h2 l = {_Float16(x[2 * e] - float(k[0])),
                  _Float16(x[2 * e + 1] - float(k[1]))};
    lo[e] = __builtin_bit_cast(uint32_t, l);
  }
  return Split{__builtin_bit_cast(h8, hi), __builtin_bit_cast(h8, lo)};
}

__device__ __forceinline__ float max_abs(const f4& a, float m) {
  return fmaxf(fmaxf(fmaxf(fabsf(a[0]), fabsf(a[1])),
                     fmaxf(fabsf(a[2]), fabsf(a[3]))), m);
}

// One wave's load of 64 x 16 bytes from global memory straight into LDS, in
// lane order (no register holds the data, so any number may be in flight).
// The completion is waited for by hand (wait_vm): the compiler does not see
// these loads and keeps no count of them.  (m0 is a reserved register, which
// the compiler sets anew before each use of its own.)
__device__ __forceinline__ void load_lds(const char* base, uint32_t off,
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

// LDS of the state kernel: BUFS buffers of one chunk's operands (in workspace
// order without V, then each wave's two V operands, whose place takes the
// chunk's outputs on their way to memory).
template <int D, bool O32, int WAVES, int PROD, int BUFS>
struct Stage {
  using W = Work<D>;
  static constexpr int shared_frags = (W::size - 2 * W::MT * kFrag) /
                                      kFrag;
  static constexpr int frags = shared_frags + 2 * WAVES;
  static constexpr int per_loader = (frags + PROD - 1) / PROD;
  static constexpr int bytes = frags * kFrag;
  static constexpr int out_row = O32 ? 64 : 48;   // bytes of 16 outputs
  static constexpr int lds = BUFS * bytes;
  static_assert(C * out_row <= 2 * kFrag, "outputs in V's place");
  // LDS offset of a workspace offset behind V
  static constexpr int behind(int off) { return off - 2 * W::MT * kFrag; }
};

template <int D, bool O32, int WAVES, int PROD, int BUFS>
__global__ void __launch_bounds__(64 * (WAVES + PROD))
    kda_prefill_state_kernel(PrefillParams p, int act_bf16) {
  using W = Work<D>;
  using G = Stage<D, O32, WAVES, PROD, BUFS>;
  constexpr bool kLean = WAVES + PROD > 8;
  constexpr int kStores = O32 ? 2 : 1;         // output stores of a chunk
  extern __shared__ __align__(16) char smem[];
  const LayerParams& y = p.y;
  const int lane = threadIdx.x & 63, col = lane & 15, g = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  // workgroup -> (request, longest first; head; tiles): the workgroups of a
  // head on one XCD (blocks i, i + 8, ..), whose L2 then serves its operands
  // to all of them
  constexpr int TB = W::MT / WAVES;            // workgroups of a head
  const int grp = blockIdx.x / (8 * TB), in = blockIdx.x - grp * (8 * TB);
  const int item = grp * 8 + in % 8;
  const int vt0 = in / 8 * WAVES, vt = vt0 + wave;
  const int rank = item / y.H, h = item - rank * y.H;
  if (rank >= y.B || rank >= p.order[-1]) return;
  const int b = p.order[rank];
  // offsets that run backwards leave places of the order unwritten
  if (b < 0 || b >= y.B) return;
  const int2 range = token_range(p, b);
  const int L = range.y - range.x;
  const int dst = y.slots[b];
  if (!live_slot(y, dst)) {
    if (wave < WAVES)
      for (int t = g; t < L; t += 4)
        st_elem(y.out,
                (range.x + t) * y.s_out + int64_t(h) * D + vt * 16 + col, 0.0f,
                !O32);
    return;
  }
  const int64_t step = int64_t(y.H) * W::size;
  const char* work =
      p.work +
      (int64_t(first_slot(range.x, b)) * y.H + h) * W::size;
  const uint32_t lds0 = uint32_t(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) char*)smem));
  const int chunks = (L + C - 1) / C;
  // One loader's share of a chunk's operands: every loader issues the same
  // number of loads (the last ones again where they do not divide), and
  // chunks behind the last one are the last one again, so that the number of
  // loads under way is known at every wait.
  auto stage = [&](int chunk) {
    const char* from_work = work + min(chunk, chunks - 1) * step;
    const int buf = chunk % BUFS, id = wave - WAVES;
#pragma unroll
    for (int i = 0; i < G::per_loader; ++i) {
      const int f = min(i * PROD + id, G::frags - 1);
      int off;
      if (f < G::shared_frags) {
        off = f * kFrag;
        if (off >= W::v) off += 2 * W::MT * kFrag;
      } else {
        const int v = f - G::shared_frags;     // [wave][row tile]
        off = W::v + ((v & 1) * W::MT + vt0 + (v >> 1)) * kFrag;
      }
      load_lds(from_work, off + lane * 16,
               lds0 + buf * G::bytes + f * kFrag);
    }
  };

  // Barrier n of the loop: chunk n's operands are in LDS, and chunk n - 1's
  // buffer has been read.  After it, chunk n + BUFS - 1 is loaded there.
  if (wave >= WAVES) {
#pragma unroll 1
    for (int n = 0; n < BUFS - 1; ++n) stage(n);
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
      wait_vm<(BUFS - 2) * G::per_loader>();
      __builtin_amdgcn_s_barrier();
      stage(n + BUFS - 1);
    }
    wait_vm<0>();     // no load may land after the workgroup's end
    return;
  }

  const int src = p.initial ? p.initial[b] : -1;
  const bool from = live_slot(y, src);
  f4 S[W::MT];      // S[m][i]: row v = col, channel 16 m + 4 g + i
  const int64_t so = (int64_t(h) * D + vt * 16 + col) * D + 4 * g;
#pragma unroll
  for (int m = 0; m < W::MT; ++m) {
    S[m] = f4{0, 0, 0, 0};
    if (from)
      S[m] = *reinterpret_cast<const f4*>(y.state + src * y.s_slot + so +
                                          16 * m);
  }
  // a wave's outputs pass through its tile in LDS: 16 bytes a lane go out,
  // in place of single elements of eight rows
  constexpr int EO = O32 ? 4 : 2, LPR = EO;    // lanes per row of 16 bytes
  char* tile = smem + (G::shared_frags + 2 * wave) * kFrag;
  const int orow = lane / LPR, ocol = lane % LPR;
  char* oat = static_cast<char*>(y.out) +
              ((range.x + orow) * y.s_out + int64_t(h) * D + vt * 16) * EO +
              ocol * 16;

  // S, V, r and c of a column share a power-of-two scale sig, chosen so that
  // the largest of S and V lies in [2^9, 2^10) and left alone while it stays
  // in [2^4, 2^10]: |r| <= |V| + |S column| <= 2^10 (1 + sqrt 128) < 65504,
  // and what the low halves cannot hold is under 2^-28 of the largest.
  float sig = 1.0f, inv = 1.0f;
#pragma unroll 1
  for (int n = 0; n < chunks; ++n) {
    const int t0 = n * C;
    lds_barrier();
    const int buf = n % BUFS;
    const char* sm = smem + buf * G::bytes + lane * 16;
    auto op = [&](int off) {
      return *reinterpret_cast<const h8*>(sm + off);
    };

    h8 kh[2 * W::KS], kl[2 * W::KS], qh[2 * W::KS], ql[2 * W::KS];
    f4 r[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r[i] = *reinterpret_cast<const f4*>(
          sm + (G::shared_frags + 2 * wave + i) * kFrag);
    const auto load_kq = [&](int j) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int a = i * W::KS + j;
        kh[a] = op(W::kd + 2 * a * kFrag);
        kl[a] = op(W::kd + (2 * a + 1) * kFrag);
        qh[a] = op(G::behind(W::qd + 2 * a * kFrag));
        ql[a] = op(G::behind(W::qd + (2 * a + 1) * kFrag));
      }
    };
    // many waves to a SIMD cover each other's loads and have no registers to
    // hold operands ahead of their use
    if constexpr (!kLean) {
#pragma unroll
      for (int j = 0; j < W::KS; ++j) load_kq(j);
      __builtin_amdgcn_sched_barrier(0);
    }
    // scale
    float top = 0.0f;
#pragma unroll
    for (int m = 0; m < W::MT; ++m) top = max_abs(S[m], top);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[i] *= sig;
      top = max_abs(r[i], top);
    }
    uint64_t low = __ballot(top < 16.0f);
    low &= low >> 32;
    low &= low >> 16;                     // all four lanes of a column
    if (__ballot(top > 1024.0f) | (low & 0xffff)) {
      // V once more, unscaled: under the scale of a column that had vanished
      // it may be infinite
      float ts = 0.0f, tv = 0.0f;
#pragma unroll
      for (int m = 0; m < W::MT; ++m) ts = max_abs(S[m], ts);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        r[i] = *reinterpret_cast<const f4*>(
            sm + (G::shared_frags + 2 * wave + i) * kFrag);
        tv = max_abs(r[i], tv);
      }
      ts = column_max(ts);
      tv = column_max(tv);
      // biased exponents under the scale of now
      const int es = int(__float_as_uint(sig) >> 23);
      const int e_s = max(int(__float_as_uint(ts) >> 23), 1);
      const int e_v = max(int(__float_as_uint(tv) >> 23), 1);
      const int e = max(ts > 0.0f ? e_s : -999,
                        tv > 0.0f ? e_v + es - 127 : -999);
      int d = 127 + 9 - e;
      if ((e >= 127 + 4 && e < 127 + 10) || e == -999 || e_s == 255 ||
          e_v == 255)
        d = 0;
      // sig stays in 2^-125 .. 2^110 (below 2^-118 only for a state past the
      // largest fp32 number), so d is in -235 .. 235: up in two factors, and
      // far down to where S is nothing beside V
      d = min(max(d, 2 - es), 237 - es);
      const float f =
          __uint_as_float(uint32_t(max(127 + min(d, 127), 0)) << 23);
      const float f2 = __uint_as_float(uint32_t(max(d, 127)) << 23);
      sig = __uint_as_float(uint32_t(es + d) << 23);
      inv = __uint_as_float(uint32_t(254 - es - d) << 23);
#pragma unroll
      for (int m = 0; m < W::MT; ++m) S[m] = S[m] * f * f2;
#pragma unroll
      for (int i = 0; i < 2; ++i) r[i] *= sig;
    }
    // S as the right operand: two 16-channel tiles make one step of 32
    f4 pr[2] = {}, pl[2] = {}, o[2] = {};
#pragma unroll
    for (int j = 0; j < W::KS; ++j) {
      if constexpr (kLean) load_kq(j);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int m = 2 * j + (e >> 2);
        x[e] = m < W::MT ? S[m < W::MT ? m : 0][e & 3] : 0.0f;
      }
      const Split s = split_wide(x);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int a = i * W::KS + j;
        pr[i] = mfma(kh[a], s.hi, pr[i]);
        pl[i] = mfma(kl[a], s.hi, pl[i]);
        o[i] = mfma(qh[a], s.hi, o[i]);
        pl[i] = mfma(kh[a], s.lo, pl[i]);
        o[i] = mfma(ql[a], s.hi, o[i]);
        o[i] = mfma(qh[a], s.lo, o[i]);
      }
      if constexpr (kLean) __builtin_amdgcn_sched_barrier(0);
    }
    // operands of the second half, on their way during the next products
    h8 th[2], tl[2], bh[2], bl[2], eh[W::MT], el[W::MT];
    f4 gam[W::MT];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      th[i] = op(W::t + 2 * i * kFrag);
      tl[i] = op(W::t + (2 * i + 1) * kFrag);
    }
#pragma unroll
    for (int m = 0; m < W::MT; ++m)
      gam[m] = *reinterpret_cast<const f4*>(
          smem + buf * G::bytes + G::behind(W::gam) + (16 * m + 4 * g) * 4);
    const auto load_ke = [&](int m) {
      eh[m] = op(W::ke + 2 * m * kFrag);
      el[m] = op(W::ke + (2 * m + 1) * kFrag);
    };
    if constexpr (!kLean) {
#pragma unroll
      for (int m = 0; m < W::MT; ++m) load_ke(m);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bh[i] = op(G::behind(W::b + 2 * i * kFrag));
      bl[i] = op(G::behind(W::b + (2 * i + 1) * kFrag));
    }
    if constexpr (!kLean) __builtin_amdgcn_sched_barrier(0);
    // r = V - (k e^G) S, c = T r; c is kept at sig / kLate, so that the update
    // (k e^(G_C - G) carries kLate) adds up at sig: a split that leaves both
    // operands' low halves above fp16's smallest steps
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = r[e >> 2][e & 3] -
             (pr[e >> 2][e & 3] + pl[e >> 2][e & 3]) * (1.0f / kUnit);
    const Split rs = split_wide(x);
    f4 cr[2], cl[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      cr[i] = mfma(th[i], rs.hi, f4{0, 0, 0, 0});
      cl[i] = mfma(tl[i], rs.hi, f4{0, 0, 0, 0});
      cl[i] = mfma(th[i], rs.lo, cl[i]);
    }
#pragma unroll
    for (int m = 0; m < W::MT; ++m) S[m] *= gam[m];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      x[e] = (cr[e >> 2][e & 3] + cl[e >> 2][e & 3]) *
             (1.0f / (kUnit * kLate));
    const Split cs = split_wide(x);
    // outputs
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[i] *= 1.0f / kLate;                 // from kUnit sig, as B c is
      o[i] = mfma(bh[i], cs.hi, o[i]);
      o[i] = mfma(bl[i], cs.hi, o[i]);
      o[i] = mfma(bh[i], cs.lo, o[i]);
    }
    // the state behind the chunk
#pragma unroll
    for (int m = 0; m < W::MT; ++m) {
      if constexpr (kLean) load_ke(m);
      S[m] = mfma(eh[m], cs.hi, S[m]);
      S[m] = mfma(el[m], cs.hi, S[m]);
      S[m] = mfma(eh[m], cs.lo, S[m]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float v = o[i][e] * (inv * (kLate / kUnit));
        char* at = tile + buf * G::bytes + (16 * i + 4 * g + e) * G::out_row +
                   col * EO;
        if constexpr (O32)
          *reinterpret_cast<float*>(at) = v;
        else
          *reinterpret_cast<__bf16*>(at) = __bf16(v);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
#pragma unroll
    for (int i = 0; i < kStores; ++i) {
      const int row = orow + i * (64 / LPR);
      const f4 v = *reinterpret_cast<const f4*>(
          tile + buf * G::bytes + row * G::out_row + ocol * 16);
      if (t0 + row < L)
        *reinterpret_cast<f4*>(oat + int64_t(i) * (64 / LPR) * y.s_out * EO) =
            v;
    }
    oat += C * y.s_out * EO;
  }
  float* to = y.state + dst * y.s_slot + so;
#pragma unroll
  for (int m = 0; m < W::MT; ++m)
    *reinterpret_cast<f4*>(to + 16 * m) = S[m] * inv;

  if (vt == 0 && !(y.flags & kNoConv)) {
    // the newest three raw inputs of the head's channels; each lane reads a
    // channel's history before it writes the channel (the slots may be one)
    const int at = history_at(y, b);
    for (int j = lane; j < 3 * D; j += 64) {
      const int part = j / D;
      const int64_t c = part * (int64_t(y.H) * D) + int64_t(h) * D +
                        (j - part * D);
      uint32_t v[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int t = L - 3 + i;
        v[i] = 0;
        if (t >= 0) {
          const int64_t e = int64_t(range.x + t) * y.s_x + c;
          v[i] = act_bf16 ? static_cast<const uint16_t*>(y.mixed_qkv)[e]
                          : static_cast<const uint32_t*>(y.mixed_qkv)[e];
        } else if (from) {
          const int64_t e = src * y.s_cs_slot + c * y.s_cs_chan +
                            (at + t + 3) * y.s_cs_tok;
          v[i] = act_bf16 ? static_cast<const uint16_t*>(y.conv_state)[e]
                          : static_cast<const uint32_t*>(y.conv_state)[e];
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int64_t e = dst * y.s_cs_slot + c * y.s_cs_chan +
                          i * y.s_cs_tok;
        if (act_bf16)
          static_cast<uint16_t*>(y.conv_state)[e] = uint16_t(v[i]);
        else
          static_cast<uint32_t*>(y.conv_state)[e] = v[i];
      }
    }
  }
}

template <int D, bool O32, int WAVES, int PROD, int BUFS>
int launch_state(const PrefillParams& p, bool act_bf16, hipStream_t stream) {
  const size_t lds = Stage<D, O32, WAVES, PROD, BUFS>::lds;
  static_assert(Stage<D, O32, WAVES, PROD, BUFS>::lds <= 160 * 1024, "LDS");
  auto kernel = kda_prefill_state_kernel<D, O32, WAVES, PROD, BUFS>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(kernel),
        hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return int(e);
  }
  const int64_t groups = (int64_t(p.y.B) * p.y.H + 7) / 8;
  const int64_t blocks = groups * 8 * (Work<D>::MT / WAVES);
  if (blocks > 0x7fffffff) return int(hipErrorInvalidValue);
  launch_kernel(kernel, dim3(uint32_t(blocks)), dim3(64 * (WAVES + PROD)),
                lds, stream, p, int(act_bf16));
  return int(hipGetLastError());
}

template <int D, bool BF16, bool O32>
int launch_prefill_dim(const PrefillParams& p, hipStream_t stream) {
  const int64_t wgs = int64_t(p.n_slots) * p.y.H;
  if (wgs > 0x7fffffff) return int(hipErrorInvalidValue);
  const size_t lds = sizeof(ChunkSmem<D>);
  auto chunk = kda_prefill_chunk_kernel<D, BF16>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(
        reinterpret_cast<const void*>(chunk),
        hipFuncAttributeMaxDynamicSharedMemorySize, int(lds));
    if (e != hipSuccess) return int(e);
  }
  launch_kernel(chunk, dim3(uint32_t(wgs)), dim3(ChunkCfg<D>::NT), lds, stream,
                p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return int(e);
  constexpr int MT = Work<D>::MT;
  // Waves that share a workgroup's operands: as few as keep all workgroups
  // resident at once (a chunk of D = 128 takes 2.1 us with two waves on every
  // CU, 2.4 to 2.7 with four, 3.4 to 4.8 with eight), else as many as there
  // are, which load and hold each operand once.  (fp32 outputs have no variant
  // of eight.)
  const int64_t items = int64_t(p.y.B) * p.y.H;
  if constexpr (MT > 4 && !O32)
    if (items * (MT / 4) > 256)
      return launch_state<D, O32, 8, 4, 2>(p, BF16, stream);
  if constexpr (MT > 2)
    if (items * (MT / 2) > 256)
      return launch_state<D, O32, 4, 4, 2>(p, BF16, stream);
  return launch_state<D, O32, (MT < 2 ? MT : 2), 4, (D == 128 ? 2 : 3)>(
      p, BF16, stream);
}

template <int D>
int launch_prefill_types(const PrefillParams& p, bool act_bf16,
                         hipStream_t stream) {
  const bool o32 = !(p.y.flags & kOutBf16);
  if (act_bf16)
    return o32 ? launch_prefill_dim<D, true, true>(p, stream)
               : launch_prefill_dim<D, true, false>(p, stream);
  return launch_prefill_dim<D, false, true>(p, stream);
}

}  // namespace

int64_t prefill_slot_bytes(int D) {
  switch (D) {
    case 16: return Work<16>::size;
    case 32: return Work<32>::size;
    case 64: return Work<64>::size;
    case 128: return Work<128>::size;
    default: return 0;
  }
}

int launch_prefill(const PrefillParams& p, int D, bool act_bf16,
                   hipStream_t stream) {
  switch (D) {
    case 16: return launch_prefill_types<16>(p, act_bf16, stream);
    case 32: return launch_prefill_types<32>(p, act_bf16, stream);
    case 64: return launch_prefill_types<64>(p, act_bf16, stream);
    case 128: return launch_prefill_types<128>(p, act_bf16, stream);
    default: return int(hipErrorInvalidValue);
  }
}

}  // namespace kda
