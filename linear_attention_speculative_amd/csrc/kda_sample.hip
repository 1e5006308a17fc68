// Sampling from logits on gfx950: temperature, top-k, min-p and top-p, the
// token from a given uniform number, and the acceptance of draft windows.
//
// For a row x with maximum m: w_i = 2^-d_i, d_i = (m - x_i) log2(e) / T, held
// as integers round(w 2^s) with s <= 46 and sums below 2^62.  All three
// filters keep a prefix of the order (x falling, index rising), so the kept
// set is one threshold pair (value, index); the token is the lowest kept index
// whose running weight passes u times the whole.  Integer sums make the result
// independent of the order in which lanes add; the weights come from fp64
// arithmetic, which a token at the border of two sums of 10^5 terms needs.
//
// A full sort is avoided.  What reads the logits is split over many workgroups
// (one alone gets some 40 GB/s of a row); what orders a row is one wave's or
// one workgroup's:
//
//   kda_group_max_kernel reads the logits once (the floor: HBM) and leaves the
//   maximum of every group of 512.
//   kda_row_sums_kernel, only for rows that need it: with top-p alone the
//   weights by bins of 1/32 octave of d, with more for top-k than groups that
//   hold any logit counts by bins, without either the weights of each group.
//   plan_row, one wave a row, then decides which logits matter.  Greedy rows
//   end here.  With top-k <= groups, the k-th largest group maximum bounds the
//   k-th largest value from below; with larger k the bin at the border of the
//   counts does.  Top-p alone needs only the bin that holds its border, and so
//   finds the threshold pair however many logits are kept.
//   kda_gather_kernel lists those logits, reading again only groups whose
//   maximum reaches the bound.
//   kda_list_kernel, one workgroup a row, sorts the list, cuts it and takes the
//   token.  What no list holds (thousands of ties, or of top-k) it leaves to a
//   radix search of any size.
//   kda_kept_sums_kernel, only for rows that kept more than a list: the kept
//   weights of each group; pick_token, one wave a row, the token from them.
//
// plan_row and pick_token have kernels of their own, except where a batch has
// so few workgroups that launches count: there one wave of the last workgroup
// to finish a row's sums does their work (launch_rows).
//
// In all, 640 of 1024 window rows of 131072 bf16 logits with mixed parameters:
// 28 us for the maxima (6 TB/s), 55 sums and plans (fp64 weights of the rows
// with top-p alone), 16 lists, 33 sorts, 26 kept sums and picks, 5 acceptance.
#include "kda_serving.hpp"

namespace kda {
namespace {

constexpr int kGroup = 512;          // logits of a group
constexpr int kMaxGroups = 2048;     // V up to 2^20
constexpr int kMaxThreads = 256;     // split kernels
constexpr int kPerWg = 4 * 4;        // their groups per workgroup
constexpr int kRowThreads = 512;     // list kernel
constexpr int kWaves = kRowThreads / 64;
constexpr int kList = 4096;          // entries of the sorted list
constexpr int kBins = 2048;
// items per thread of the row kernel: bins and groups, list entries, half bins
constexpr int kPer2k = kBins / kRowThreads;
constexpr int kPerList = kList / kRowThreads;
constexpr int kPer1k = 1024 / kRowThreads;
static_assert(kBins == kMaxGroups && kPer1k >= 1, "sizes");
constexpr int kSteps = 256;          // of an octave, in the table of weights

// The request of row m, or -1 for a row outside every request.
__device__ __forceinline__ int request_of_row(const SampleParams& p, int m,
                                              int lane) {
  if (p.qsl == nullptr) return m < p.B ? m : -1;
  if (p.B == 0 || m < p.qsl[0] || m >= p.qsl[p.B]) return -1;
  int lo = 0, n = p.B;
  while (n > 1) {      // last b with qsl[b] <= m, 64 candidates at a time
    const int step = (n + 63) / 64;
    const int i = lane * step;
    const bool in = i < n && p.qsl[lo + i] <= m;
    const int k = max(int(__popcll(__ballot(in))) - 1, 0) * step;
    lo += k;
    n = min(step, n - k);
  }
  lo = uniform(lo);
  return p.qsl[lo] <= m && m < p.qsl[lo + 1] ? lo : -1;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v = fmaxf(v, __shfl_xor(v, s));
  return v;
}

// Eight consecutive logits of an aligned row as one or two 16-byte loads.
template <bool BF16>
__device__ __forceinline__ void load8(const char* row, int i, float (&x)[8]) {
  if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + 2 * int64_t(i));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f4 v = *reinterpret_cast<const f4*>(row + 4 * int64_t(i) + 16 * h);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[4 * h + e] = v[e];
    }
  }
}

// A group's logits over the lanes of a wave: element e of lane l is logit
// first + 8 l + e (aligned rows) or first + 64 e + l; index(e) tells which.
// Behind the row's end -inf, and -inf for NaN.
template <bool BF16, bool VEC>
struct Group {
  float x[8];
  int first;
  __device__ __forceinline__ int index(int e) const {
    const int lane = threadIdx.x & 63;
    return VEC ? first + 8 * lane + e : first + 64 * e + lane;
  }
  __device__ __forceinline__ void load(const char* row, int g, int V) {
    typedef typename Act<BF16>::T T;
    first = g * kGroup;
    const int lane = threadIdx.x & 63;
    if (first + kGroup <= V) {
      if constexpr (VEC) {
        load8<BF16>(row, first + 8 * lane, x);
      } else {
        const T* at = reinterpret_cast<const T*>(row) + first + lane;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = Act<BF16>::f(at[64 * e]);
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = min(index(e), V - 1);
        x[e] = Act<BF16>::f(reinterpret_cast<const T*>(row)[i]);
        if (index(e) >= V) x[e] = -__builtin_inff();
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!(x[e] == x[e])) x[e] = -__builtin_inff();
  }
};

// fp32 as an unsigned number of the same order, and back.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);      // -0 counts as 0
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
constexpr uint32_t kLowestKey = 0x00800000u;       // the least above -inf's

// The least key from kLowestKey to `top` whose value satisfies `test`, which
// `top` does and every value above one that does: by every wave for itself,
// 64 candidates at a time.
template <class Test>
__device__ __forceinline__ uint32_t least_key(uint32_t top, Test test) {
  uint32_t lo = kLowestKey, hi = top;
  while (lo < hi) {
    const uint32_t step = (hi - lo) / 64 + 1;
    const uint64_t at = uint64_t(lo) + uint64_t(threadIdx.x & 63) * step;
    const uint64_t in =
        __ballot(at >= hi || test(unordered(uint32_t(at < hi ? at : hi))));
    // some candidate is at or past hi, or test holds from none of them to hi
    const int f = in ? int(__ffsll((unsigned long long)in)) - 1 : 64;
    const uint64_t first = uint64_t(lo) + uint64_t(f) * step;
    if (f > 0) lo += uint32_t(f - 1) * step + 1;
    hi = first < hi ? uint32_t(first) : hi;
  }
  return uint32_t(uniform(int(hi)));
}

struct RowSmem {
  union {
    // ordered(x) << 32 | ~index.  A sort of at most half of them uses the
    // upper half as its second buffer, which then holds their weights.
    uint64_t key[kList];
    uint32_t count[kBins];
    uint64_t mass[kBins];
    uint64_t group[kMaxGroups];
  };
  float gmax[kMaxGroups];
  double table[kSteps];         // 2^(-j/256)
  uint64_t red[kWaves];
  int found, pick;
  uint64_t before, value;
};

__device__ __forceinline__ void fill_table(double* table) {
  for (int i = threadIdx.x; i < kSteps; i += blockDim.x)
    table[i] = exp2(double(i) * (-1.0 / kSteps));
}

__device__ __forceinline__ double uniform_double(double v) {
  return __hiloint2double(uniform(__double2hiint(v)),
                          uniform(__double2loint(v)));
}

// Weight of a logit as an integer, from its distance to the maximum in steps
// of 1/256 octave: a table for the nearest whole step, the exponential's series
// up to the fourth power for the rest (the fifth is under 2^-54 of the weight;
// without the fourth, weights are up to ten units low), the octave by the
// exponent field, and an addition whose last binary place is 1 to round.
struct Weights {
  const double* table;
  double m, c;                  // maximum; steps per unit
  double most, d_min_p;         // clamp; steps that min-p allows
  int s;                        // binary places
  __device__ __forceinline__ void init(const double* tab, float top, float T,
                                       float min_p, int places) {
    table = tab;
    m = top;
    s = places;
    c = kSteps * 1.4426950408889634074 / double(T);
    if (top == __builtin_inff()) {      // itself: 0 steps; all others: `most`
      m = 0x1p128;
      c = 0x1p900;
    }
    most = double((places + 2) * kSteps);           // weighs 2^-2 places: 0
    d_min_p = min_p > 0.0f ? -kSteps * log2(double(fminf(min_p, 1.0f)))
                           : __builtin_inf();
    // one value for all lanes: in scalar registers
    m = uniform_double(m);
    c = uniform_double(c);
    most = uniform_double(most);
    d_min_p = uniform_double(d_min_p);
  }
  // Steps below the maximum (`most` for -inf and whatever the weights cannot
  // tell from 0).
  __device__ __forceinline__ double steps(float x) const {
    return fmax(fmin((m - double(x)) * c, most), 0.0);
  }
  // the nearest whole step
  __device__ __forceinline__ int nearest(double d) const {
    return __double2loint(d + 0x1.8p52);
  }
  __device__ __forceinline__ uint64_t whole(double d) const {
    const double r = d + 0x1.8p52;
    const int e = __double2loint(r);
    const double f = d - (r - 0x1.8p52);
    constexpr double l = -0.6931471805599453094 / kSteps;
    double q = fma(f, l * l * l * l / 24.0, l * l * l / 6.0);
    q = fma(f, q, l * l / 2.0);
    q = fma(f, q, l);
    q = fma(f, q, 1.0) * table[e & (kSteps - 1)];
    const int64_t u = __double_as_longlong(q) +
                      (int64_t(s - e / kSteps) << 52);
    return uint64_t(__double_as_longlong(__longlong_as_double(u) + 0x1p52)) &
           ((uint64_t(1) << 52) - 1);
  }
  __device__ __forceinline__ uint64_t of(float x) const {
    return whole(steps(x));
  }
  // within min-p (a -inf never is)
  __device__ __forceinline__ bool allows(float x, double d) const {
    return d <= d_min_p && x > -__builtin_inff();
  }
  // 1/32 octave bins
  __device__ __forceinline__ int bin(double d) const {
    return min(nearest(d) >> 3, kBins - 1);
  }
};

// The parameters of a row's request, NaN and absent ones off.
struct Params {
  float T, top_p, min_p, u;
  int k;
  bool greedy, need_k, need_p;
  __device__ __forceinline__ Params(const SampleParams& p, int b, int m) {
    // five loads under way together, of some valid place for what is absent
    const float* any = p.uniform + m;
    const float t = *(p.temperature ? p.temperature + b : any);
    const int n = *(p.top_k ? p.top_k + b : reinterpret_cast<const int*>(any));
    const float tp = *(p.top_p ? p.top_p + b : any);
    const float mp = *(p.min_p ? p.min_p + b : any);
    const float uu = *any;
    T = p.temperature && t == t ? t : 1.0f;
    k = p.top_k ? n : 0;
    top_p = p.top_p && tp < 1.0f ? tp : 1.0f;
    min_p = p.min_p && mp > 0.0f ? mp : 0.0f;
    u = uu > 0.0f ? fminf(uu, 0x1.fffffep-1f) : 0.0f;
    greedy = T <= 0.0f || k == 1 || top_p <= 0.0f;
    need_k = k > 0 && k < p.V;
    need_p = top_p < 1.0f;
  }
};

// What is left to do for a row, and what the kernels tell each other.
enum Mode : int32_t {
  kDecided,      // nothing
  kGather,       // list the keys first <= key < last, then take it from there
  kSearch,       // too many for a list
  kKept,         // sum the weights that the threshold pair keeps, then pick
  kSummed        // pick; the sums are there
};
struct Plan {
  Mode mode;
  float top;                 // the row's maximum
  uint32_t min_key;          // least key that min-p allows
  uint32_t first, last;
  uint32_t n;                // keys found; kList at most are in the list
  uint64_t mass, before;     // top-p alone: weights of all, and above `last`
  uint32_t key;              // threshold pair
  int32_t index;
  uint32_t arrived[2];       // workgroups that have done the row's sums, and
                             // its kept sums
};

// Workspace of a row: maxima of its groups, sums (bins or groups), the list,
// and its plan.
struct Work {
  float* gmax;
  uint64_t* sums;         // [kBins]: bins, or weights of groups
  uint64_t* list;         // [kList]: ordered(x) << 32 | ~index
  Plan* plan;
  __device__ __host__ static int64_t maxima(int64_t M, int64_t G) {
    return (M * G * 4 + 255) / 256 * 256;
  }
  __device__ __host__ static int64_t bytes(int64_t M, int64_t G) {
    return maxima(M, G) + M * int64_t(kBins + kList) * 8 +
           (M * int64_t(sizeof(Plan)) + 255) / 256 * 256;
  }
  __device__ __forceinline__ Work(const SampleParams& p, int m, int G) {
    char* at = p.work + maxima(p.M, G);
    gmax = reinterpret_cast<float*>(p.work) + int64_t(m) * G;
    sums = reinterpret_cast<uint64_t*>(at) + int64_t(m) * kBins;
    at += int64_t(p.M) * kBins * 8;
    list = reinterpret_cast<uint64_t*>(at) + int64_t(m) * kList;
    at += int64_t(p.M) * kList * 8;
    plan = reinterpret_cast<Plan*>(at) + m;
  }
};

// Whether this workgroup is the last of `parts` of a row to get here.  It then
// may read what the others wrote before: each counts itself with a release of
// what its threads wrote (the barrier hands that to the first thread), and the
// count it finds acquires what the others released.  Every wave also waits for
// its stores to end before the barrier, so that the release finds them in the
// L2 whatever the order in which a CU's waves reach it.  A release writes back
// an XCD's L2, so this is for few workgroups (launch_rows).
__device__ __forceinline__ bool last_of(uint32_t* arrived, int parts) {
  __shared__ int last;
  asm volatile("s_waitcnt vmcnt(0)" : : : "memory");
  __syncthreads();
  if (threadIdx.x == 0)
    last = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_ACQ_REL,
                                  __HIP_MEMORY_SCOPE_AGENT) ==
           uint32_t(parts - 1);
  __syncthreads();
  return last != 0;
}

// The groups of a row that a workgroup of the split kernels takes.
struct Part {
  int m, first, end;
  bool chosen;     // one of them, not always on the same XCD
  __device__ __forceinline__ Part(int G, int per_row, int per_wg = kPerWg) {
    m = blockIdx.x / per_row;
    const int part = blockIdx.x - m * per_row;
    first = part * per_wg;
    end = min(first + per_wg, G);
    chosen = part == m % per_row;
  }
};

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
    kda_group_max_kernel(SampleParams p, int G, int per_row) {
  const Part part(G, per_row);
  const int m = part.m;
  if (p.qsl && (m < p.qsl[0] || m >= p.qsl[p.B])) return;
  const char* row = static_cast<const char*>(p.logits) +
                    m * p.s_row * (BF16 ? 2 : 4);
  const Work out(p, m, G);
  if (part.chosen && threadIdx.x == 0)
    out.plan->arrived[0] = out.plan->arrived[1] = 0;
  // the row's bins, cleared for the next kernel
  for (int i = (blockIdx.x - m * per_row) * kMaxThreads + threadIdx.x;
       i < kBins; i += per_row * kMaxThreads)
    out.sums[i] = 0;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int g0 = part.first + wave * (kPerWg / 4);
  Group<BF16, VEC> v[kPerWg / 4];
#pragma unroll
  for (int i = 0; i < kPerWg / 4; ++i) v[i].load(row, min(g0 + i, G - 1), p.V);
#pragma unroll
  for (int i = 0; i < kPerWg / 4; ++i) {
    float t = v[i].x[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) t = fmaxf(t, v[i].x[e]);
    t = wave_max(t);
    if (lane == 0 && g0 + i < part.end) out.gmax[g0 + i] = t;
  }
}

// f(x) for the logits of a wave's group that keep(x, index) takes.  The lanes
// first gather them in `buf` (512 floats of the wave's own): with few kept,
// one dense pass in place of eight sparse ones through f's fp64 arithmetic.
template <bool BF16, bool VEC, class Keep, class F>
__device__ __forceinline__ void each_kept(const Group<BF16, VEC>& v,
                                          float* buf, Keep keep, F f) {
  const int lane = threadIdx.x & 63;
  uint64_t in[8];
  int n = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    in[e] = __ballot(keep(v.x[e], v.index(e)));
    n += __popcll(in[e]);
  }
  if (n > kGroup / 4 * 3) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (keep(v.x[e], v.index(e))) f(v.x[e]);
    return;
  }
  uint32_t at = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t mine = __builtin_amdgcn_mbcnt_hi(
        uint32_t(in[e] >> 32),
        __builtin_amdgcn_mbcnt_lo(uint32_t(in[e]), at));
    if (keep(v.x[e], v.index(e))) buf[mine] = v.x[e];
    at += __popcll(in[e]);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
  for (int i = lane; i < n; i += 64) f(buf[i]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
}

// Threshold pair: a logit is kept if it is larger than `key`'s value, or equal
// and at an index of at most `index`.
struct Threshold {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool keeps(float x, int i) const {
    const float at = unordered(key);
    return x > at || (x == at && i <= index);
  }
};

template <bool BF16, bool VEC>
struct Row {
  const char* at;
  int V, G;
  RowSmem& sm;
  // f(x, index) for the logits of the groups that `use(g)` takes; -inf is left
  // out.
  template <class Use, class F>
  __device__ __forceinline__ void each(Use use, F f) const {
    each_group(use, [&](const Group<BF16, VEC>& v) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (v.x[e] > -__builtin_inff()) f(v.x[e], v.index(e));
    });
  }
  // f(group), a group to a wave.
  template <class Use, class F>
  __device__ __forceinline__ void each_group(Use use, F f) const {
    each_batch(use, [&](const Group<BF16, VEC>(&v)[kAhead], int n) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (j >= n) break;
        f(v[j]);
      }
    });
  }
  // f(groups, count): the loads of up to kAhead groups at once.
  static constexpr int kAhead = 2;
  template <class Use, class F>
  __device__ __forceinline__ void each_batch(Use use, F f) const {
    const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
#pragma unroll 1
    for (int base = wave; base < G; base += 64 * kWaves) {
      const int mine = base + lane * kWaves;
      uint64_t left = __ballot(mine < G && use(min(mine, G - 1)));
#pragma unroll 1
      while (left) {
        int id[kAhead], n = 0;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          id[j] = j > 0 ? id[j - 1] : 0;
          if (left) {
            id[j] = base + (__ffsll((unsigned long long)left) - 1) * kWaves;
            left &= left - 1;
            ++n;
          }
        }
        Group<BF16, VEC> v[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) v[j].load(at, id[j], V);
        f(v, n);
      }
    }
  }
};

__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) v += __shfl_xor((unsigned long long)v, s);
  return v;
}

// Inclusive prefix sum over a wave.
__device__ __forceinline__ uint64_t wave_scan(uint64_t v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 1; s < 64; s <<= 1) {
    const uint64_t o = __shfl_up((unsigned long long)v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// First of n numbers (at most 64 * 64) whose inclusive prefix sum reaches
// goal(total), or -1, by one wave: by the `own` numbers of each lane, then
// among those of the lane found.
struct Found {
  int at;
  uint64_t before, value, total;
};
// kOwn = n / 64: numbers that an earlier launch left; kOwn = 0: any n, written
// by others of this launch.
template <int kOwn, class Goal>
__device__ __forceinline__ Found find_first(const uint64_t* a, int n,
                                            Goal goal) {
  const int own = kOwn > 0 ? kOwn : (n + 63) / 64;
  const int lane = threadIdx.x & 63;
  uint64_t sum = 0;
  if constexpr (kOwn > 0) {
#pragma unroll
    for (int j = 0; j < kOwn / 2; ++j) {
      const ulonglong2 v =
          reinterpret_cast<const ulonglong2*>(a)[lane * (kOwn / 2) + j];
      sum += v.x + v.y;
    }
  } else {
#pragma unroll 4
    for (int j = 0; j < own; ++j) {
      const int i = lane * own + j;
      const uint64_t v = a[min(i, n - 1)];
      sum += i < n ? v : 0;
    }
  }
  Found f{-1, 0, 0, 0};
  const uint64_t upto = wave_scan(sum);
  f.total = __shfl((unsigned long long)upto, 63);
  const uint64_t target = goal(f.total);
  const uint64_t in = __ballot(upto >= target);
  if (in == 0) return f;
  const int l = __ffsll((unsigned long long)in) - 1;
  const uint64_t base = __shfl((unsigned long long)(upto - sum), l);
  const int first = l * own;
  const uint64_t v =
      lane < own && first + lane < n ? a[first + lane] : 0;
  const uint64_t u = base + wave_scan(v);
  const int i = __ffsll((unsigned long long)__ballot(u >= target)) - 1;
  f.at = first + i;
  f.before = __shfl((unsigned long long)(u - v), i);
  f.value = __shfl((unsigned long long)v, i);
  return f;
}
static_assert(kMaxGroups <= 64 * 64 && kBins <= 64 * 64, "find_first");

// Inclusive prefix sum over the workgroup, and the total.
__device__ __forceinline__ uint64_t row_scan(uint64_t v, uint64_t* red,
                                             uint64_t* total) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  v = wave_scan(v);
  __syncthreads();
  if (lane == 63) red[w] = v;
  __syncthreads();
  uint64_t base = 0, sum = 0;
#pragma unroll
  for (int j = 0; j < kWaves; ++j) {
    base = j == w ? sum : base;
    sum += red[j];
  }
  *total = sum;
  return base + v;
}

// First index i of a(0 .. n - 1) (n <= kPer * kRowThreads) whose inclusive
// prefix sum reaches goal(total of a); sm.found = i (or -1), sm.before = the
// sum before it, sm.value = a(i).  Returns the total.
template <int kPer, class A, class Goal>
__device__ __forceinline__ uint64_t find_prefix(RowSmem& sm, A a, int n,
                                                Goal goal) {
  uint64_t v[kPer], own = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x * kPer + j;
    v[j] = i < n ? uint64_t(a(i)) : 0;
    own += v[j];
  }
  __syncthreads();                    // the last result has been read
  if (threadIdx.x == 0) sm.found = -1;
  uint64_t total;
  uint64_t sum = row_scan(own, sm.red, &total) - own;
  const uint64_t target = goal(total);
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int i = threadIdx.x * kPer + j;
    if (i < n && sum < target && sum + v[j] >= target) {
      sm.found = i;
      sm.before = sum;
      sm.value = v[j];
    }
    sum += v[j];
  }
  __syncthreads();
  return total;
}

// The value of lane l ^ J, without a trip through LDS.
template <int J>
__device__ __forceinline__ uint32_t lane_xor(uint32_t u) {
  const auto mov = [](uint32_t x, auto ctrl) {
    return uint32_t(__builtin_amdgcn_mov_dpp(int(x), decltype(ctrl)::value,
                                             0xF, 0xF, true));
  };
  if constexpr (J == 1) return mov(u, std::integral_constant<int, kQuadXor1>{});
  if constexpr (J == 2) return mov(u, std::integral_constant<int, kQuadXor2>{});
  if constexpr (J == 4)        // l ^ 7, then l ^ 3
    return mov(mov(u, std::integral_constant<int, kRowHalfMirror>{}),
               std::integral_constant<int, 0x1B>{});
  if constexpr (J == 8)        // l ^ 15, then l ^ 7
    return mov(mov(u, std::integral_constant<int, kRowMirror>{}),
               std::integral_constant<int, kRowHalfMirror>{});
  if constexpr (J == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    return threadIdx.x & 16 ? r[0] : r[1];
  }
  if constexpr (J == 32) {
    const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return threadIdx.x & 32 ? r[0] : r[1];
  }
}

// One step of the bitonic network on key i: the larger of the pair goes to
// the lower index in blocks of k whose bit k is clear.
__device__ __forceinline__ uint64_t keep_of(uint64_t own, uint64_t other,
                                            int i, int k, int j) {
  const bool larger = ((i & k) == 0) == ((i & j) == 0);
  return (own > other) == larger ? own : other;
}

template <int J, int P>
__device__ __forceinline__ void lane_step(uint64_t (&v)[P], int k) {
  if (J >= k) return;
#pragma unroll
  for (int r = 0; r < P; ++r) {
    const uint64_t o = uint64_t(lane_xor<J>(uint32_t(v[r] >> 32))) << 32 |
                       lane_xor<J>(uint32_t(v[r]));
    v[r] = keep_of(v[r], o, r * kRowThreads + threadIdx.x, k, J);
  }
}

// Sort of `size` keys (a power of two, at most P * kRowThreads), falling: key
// r * kRowThreads + tid in register r of a thread.  Pairs inside a wave are
// exchanged between lanes, pairs of registers in place, the others through two
// buffers in turn, at one barrier each, or through a alone (b = a) at two.
template <int P>
__device__ __forceinline__ void sort_keys(uint64_t* a, uint64_t* b, int size) {
  const int tid = threadIdx.x;
  uint64_t v[P];
#pragma unroll
  for (int r = 0; r < P; ++r) {
    const int i = r * kRowThreads + tid;
    v[r] = i < size ? a[i] : 0;
  }
  uint64_t* buf = b;
#pragma unroll 1
  for (int k = 2; k <= size; k <<= 1) {
#pragma unroll
    for (int s = P / 2; s >= 1; s >>= 1)
      if (s * kRowThreads < k) {
#pragma unroll
        for (int r = 0; r < P; ++r)
          if ((r & s) == 0) {
            const int i = r * kRowThreads + tid;
            const uint64_t x = v[r], z = v[r + s];
            const bool larger = (i & k) == 0;
            v[r] = (x > z) == larger ? x : z;
            v[r + s] = (x > z) == larger ? z : x;
          }
      }
#pragma unroll 1
    for (int j = min(k >> 1, kRowThreads / 2); j >= 64; j >>= 1) {
#pragma unroll
      for (int r = 0; r < P; ++r) buf[r * kRowThreads + tid] = v[r];
      __syncthreads();
#pragma unroll
      for (int r = 0; r < P; ++r) {
        const int i = r * kRowThreads + tid;
        v[r] = keep_of(v[r], buf[i ^ j], i, k, j);
      }
      if (a == b) __syncthreads();
      buf = buf == a ? b : a;
    }
    lane_step<32>(v, k);
    lane_step<16>(v, k);
    lane_step<8>(v, k);
    lane_step<4>(v, k);
    lane_step<2>(v, k);
    lane_step<1>(v, k);
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < P; ++r) a[r * kRowThreads + tid] = v[r];
  __syncthreads();
}

// Sort of the list's first n keys, falling; zeros follow them.
__device__ __forceinline__ void sort_list(RowSmem& sm, int n) {
  int size = 2;
  while (size < n) size <<= 1;
  for (int i = n + threadIdx.x; i < size; i += kRowThreads) sm.key[i] = 0;
  __syncthreads();
  uint64_t* const upper = sm.key + kList / 2;
  if (size <= kRowThreads)
    sort_keys<1>(sm.key, upper, size);
  else if (size <= 2 * kRowThreads)
    sort_keys<2>(sm.key, upper, size);
  else if (size <= 4 * kRowThreads)
    sort_keys<4>(sm.key, upper, size);
  else
    sort_keys<8>(sm.key, sm.key, size);
  static_assert(kList == 8 * kRowThreads, "sort");
}

// Target of a share of a whole: the least integer >= share * mass, at least 1
// and at most mass.
__device__ __forceinline__ uint64_t share_of(double share, uint64_t mass) {
  const double t = ceil(share * double(mass));
  const uint64_t v = t >= 1.0 ? uint64_t(t) : 1;
  return v < mass ? v : mass;
}

// Sums of v before each element of a wave's group, in the order of indexes.
template <bool VEC>
__device__ __forceinline__ void group_prefix(const uint64_t (&v)[8],
                                             uint64_t (&pre)[8]) {
  if constexpr (VEC) {            // a lane's elements are neighbours
    uint64_t own = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      pre[e] = own;
      own += v[e];
    }
    const uint64_t base = wave_scan(own) - own;
#pragma unroll
    for (int e = 0; e < 8; ++e) pre[e] += base;
  } else {                        // neighbours are in neighbouring lanes
    uint64_t base = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint64_t upto = wave_scan(v[e]);
      pre[e] = base + upto - v[e];
      base += __shfl((unsigned long long)upto, 63);
    }
  }
}

// The least integer > u * mass, at most mass.
__device__ __forceinline__ uint64_t past_share(float u, uint64_t mass) {
  const uint64_t past = uint64_t(double(u) * double(mass)) + 1;
  return past < mass ? past : mass;
}

// The threshold of the first `target` in what(x) among the logits that `thr`
// keeps and whose keys are at least `least`: radix search over the ordered
// keys, 11, 11 and 10 bits a pass, then the last tie's index.
template <bool BF16, bool VEC, class What>
__device__ __forceinline__ Threshold search(const Row<BF16, VEC>& row,
                                            uint32_t least, Threshold thr,
                                            uint64_t target, What what) {
  RowSmem& sm = row.sm;
  const auto used = [&](int g) { return ordered(sm.gmax[g]) >= least; };
  uint32_t prefix = 0, mask = 0;
  uint64_t before = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    __syncthreads();
    for (int i = threadIdx.x; i < bins; i += kRowThreads) sm.mass[i] = 0;
    __syncthreads();
    row.each(used, [&](float x, int i) {
      const uint32_t k = ordered(x);
      if ((k & mask) == prefix && k >= least && thr.keeps(x, i))
        // bins in falling order
        atomicAdd((unsigned long long*)&sm
                      .mass[bins - 1 - ((k >> shift) & (bins - 1))],
                  (unsigned long long)what(x));
    });
    __syncthreads();
    find_prefix<kPer2k>(sm, [&](int i) { return sm.mass[i]; }, bins,
                   [&](uint64_t) { return target - before; });
    before += sm.before;
    prefix |= uint32_t(bins - 1 - max(sm.found, 0)) << shift;
    mask |= uint32_t(bins - 1) << shift;
  }
  // ties: each counts the same; the index of the last one kept
  const uint64_t one = what(unordered(prefix));
  const uint64_t left = target - before;
  const uint64_t rank = one > 0 ? (left + one - 1) / one : 1;
  __syncthreads();
  for (int i = threadIdx.x; i < row.G; i += kRowThreads) sm.group[i] = 0;
  __syncthreads();
  row.each(used, [&](float x, int i) {
    if (ordered(x) == prefix && thr.keeps(x, i))
      atomicAdd((unsigned long long*)&sm.group[i / kGroup], 1ull);
  });
  __syncthreads();
  find_prefix<kPer2k>(sm, [&](int i) { return sm.group[i]; }, row.G,
                      [&](uint64_t) { return rank; });
  const int g = sm.found;
  const uint64_t seen = sm.before;
  if (threadIdx.x == 0) sm.pick = row.V - 1;
  __syncthreads();
  if (g >= 0 && threadIdx.x < 64) {
    Group<BF16, VEC> v;
    v.load(row.at, g, row.V);
    uint64_t tie[8], pre[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      tie[e] = ordered(v.x[e]) == prefix && thr.keeps(v.x[e], v.index(e));
    group_prefix<VEC>(tie, pre);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (tie[e] && seen + pre[e] + 1 == rank) sm.pick = v.index(e);
  }
  __syncthreads();
  const Threshold t{prefix, sm.pick};
  __syncthreads();
  return t;
}

// Row maximum from the groups' maxima, by every wave for itself.
__device__ __forceinline__ float row_max(const float* gmax, int G) {
  float top = -__builtin_inff();
  for (int g = threadIdx.x & 63; g < G; g += 64) top = fmaxf(top, gmax[g]);
  return wave_max(top);
}

// Groups whose maximum has a key of at least `least`.
__device__ __forceinline__ int live_groups(const float* gmax, int G,
                                           uint32_t least) {
  const int lane = threadIdx.x & 63;
  int n = 0;
  for (int g = lane; g - lane < G; g += 64)
    n += __popcll(__ballot(g < G && ordered(gmax[min(g, G - 1)]) >= least));
  return n;
}

// Key of the k-th largest group maximum (k <= G), bit by bit, by every wave
// for itself.
__device__ __forceinline__ uint32_t kth_key(const float* gmax, int G, int k) {
  constexpr int kRegs = kMaxGroups / 64, kStep = 4;
  const int lane = threadIdx.x & 63;
  uint32_t key[kRegs];
#pragma unroll
  for (int r = 0; r < kRegs; r += kStep) {
    if (r * 64 >= G) break;
#pragma unroll
    for (int i = r; i < r + kStep; ++i) {
      const int g = i * 64 + lane;
      key[i] = g < G ? ordered(gmax[min(g, G - 1)]) : 0;
    }
  }
  uint32_t at = 0;       // the largest key that k maxima reach, two bits a step
#pragma unroll 1
  for (int bit = 30; bit >= 0; bit -= 2) {
    int n[3] = {0, 0, 0};
#pragma unroll
    for (int r = 0; r < kRegs; r += kStep) {
      if (r * 64 >= G) break;
#pragma unroll
      for (int i = r; i < r + kStep; ++i)
#pragma unroll
        for (int d = 0; d < 3; ++d)
          n[d] += __popcll(__ballot(key[i] >= (at | uint32_t(d + 1) << bit)));
    }
    at |= uint32_t((n[0] >= k) + (n[1] >= k) + (n[2] >= k)) << bit;
  }
  return at;
}

// Bins of m - x for counts; kBins for whatever lies behind the last one (or
// cannot be told, below a maximum of +inf).  Those down to `low`, the least
// maximum among the groups that hold a key of at least min_key, take 7/8 of
// them for few and 3/8 for many: of G groups of any 512 independent values
// some G ln G lie at or above it.  Fewer logits to count, and finer bins.
struct CountBins {
  float top, scale;
  static __device__ __forceinline__ bool few(int k, int G) {
    return 2.0f * float(k) <= float(G) * __log2f(float(G));
  }
  __device__ __forceinline__ CountBins(const float* gmax, int G, float top_,
                                       uint32_t min_key, bool few)
      : top(top_) {
    float low = top;
    for (int g = threadIdx.x & 63; g < G; g += 64)
      if (ordered(gmax[g]) >= min_key) low = fminf(low, gmax[g]);
    low = -wave_max(-low);
    scale = float(kBins / 8) * (few ? 7.0f : 3.0f) / fmaxf(top - low, 1e-3f);
  }
  // never falls as x falls
  __device__ __forceinline__ int operator()(float x) const {
    const float f = (top - x) * scale;
    return f < float(kBins) ? int(f) : kBins;
  }
};

// Least key that min-p allows.
__device__ __forceinline__ uint32_t least_allowed(const Params& q,
                                                  const Weights& wt,
                                                  float top) {
  if (!(q.min_p > 0.0f)) return kLowestKey;
  return least_key(ordered(top),
                   [&](float x) { return wt.allows(x, wt.steps(x)); });
}

// What a row needs, by one wave; greedy rows get their token.
template <bool BF16, bool VEC, bool kShared>
__device__ __forceinline__ void plan_row(const SampleParams& p,
                                         const Work& work, const Params& q,
                                         int m, int G, int places) {
  const int lane = threadIdx.x & 63;
  const int k = q.k;
  const float* gmax = work.gmax;
  const float top = row_max(gmax, G);
  Plan plan{};
  plan.top = top;
  plan.last = 0xffffffffu;
  plan.index = p.V;
  if (top == -__builtin_inff() || q.greedy) {
    int token = -1;
    if (top > -__builtin_inff()) {
      // the lowest index of the maximum
      int g = lane;
      while (!__any(g < G && gmax[min(g, G - 1)] == top) && g - lane < G)
        g += 64;
      const uint64_t in = __ballot(g < G && gmax[min(g, G - 1)] == top);
      g = g - lane + __ffsll((unsigned long long)in) - 1;
      Group<BF16, VEC> v;
      v.load(static_cast<const char*>(p.logits) +
                 m * p.s_row * (BF16 ? 2 : 4),
             min(max(g, 0), G - 1), p.V);
      int at = p.V - 1;
#pragma unroll
      for (int e = 7; e >= 0; --e)
        if (v.x[e] == top) at = min(at, v.index(e));
#pragma unroll
      for (int s = 1; s < 64; s <<= 1) at = min(at, __shfl_xor(at, s));
      token = at;
    }
    if (lane == 0) {
      p.tokens[m] = token;
      work.plan->mode = kDecided;
    }
    return;
  }
  // Every condition on a logit's weight is one on its key.
  Weights wt;
  wt.init(nullptr, top, q.T, q.min_p, places);
  const uint32_t min_key = least_allowed(q, wt, top);
  const uint32_t top_key = ordered(top);
  plan.min_key = plan.first = plan.key = min_key;
  plan.mode = kGather;
  if (!q.need_k && !q.need_p) {
    plan.mode = kSummed;
  } else if (!q.need_k) {
    const Found f = find_first<kShared ? 0 : kBins / 64>(
        work.sums, kBins, [&](uint64_t w) { return share_of(q.top_p, w); });
    plan.mass = f.total;
    plan.before = f.before;
    plan.first = max(min_key, least_key(top_key, [&](float x) {
                       return wt.bin(wt.steps(x)) <= f.at;
                     }));
    if (f.at > 0)
      plan.last = least_key(top_key, [&](float x) {
        return wt.bin(wt.steps(x)) < f.at;
      });
  } else {
    // groups that hold any logit, and one that min-p allows
    const int live = live_groups(gmax, G, kLowestKey);
    const int allowed = live_groups(gmax, G, min_key);
    if (k <= allowed) {
      // at least k logits lie at or above the k-th largest group maximum
      plan.first = kth_key(gmax, G, k);
    } else if (k > live) {           // counted before
      const CountBins bins(gmax, G, top, min_key, CountBins::few(k, live));
      const Found f = find_first<kShared ? 0 : kBins / 64>(
          work.sums, kBins, [&](uint64_t) { return uint64_t(k); });
      if (f.at >= 0)
        plan.first = max(min_key, least_key(top_key, [&](float x) {
                           return bins(x) <= f.at;
                         }));
      // (below the last bin may lie any number; min-p may leave few of it)
      const bool many = f.at >= 0 ? f.before + f.value > kList
                                  : allowed * kGroup > kList;
      if (many && !(q.min_p > 0.0f)) plan.mode = kSearch;
    }
    // between the two, min-p likely leaves few: all it allows
  }
  if (lane == 0) *work.plan = plan;
}

// per_wg groups a workgroup, of the rows that need more than their group
// maxima: top-k beyond the number of groups, counts by bins; top-p alone,
// weights by bins (both added to the row's bins); neither, the weight of each
// group.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
    kda_row_sums_kernel(SampleParams p, int G, int per_row, int per_wg,
                        int places, bool plans) {
  __shared__ double table[kSteps];
  __shared__ unsigned long long mass[kBins];
  __shared__ float kept[kMaxThreads / 64][kGroup];
  const Part part(G, per_row, per_wg);
  const int m = part.m;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int b = request_of_row(p, m, lane);
  const Work work(p, m, G);
  if (b < 0) {
    if (plans && part.chosen && threadIdx.x == 0) work.plan->mode = kDecided;
    return;
  }
  const Params q(p, b, m);
  if (q.greedy && !plans) return;
  const bool counts = q.need_k;
  const int live = counts ? live_groups(work.gmax, G, kLowestKey) : G;
  const float top = row_max(work.gmax, G);
  if (q.greedy || (counts && q.k <= live) || top == -__builtin_inff()) {
    if (plans && part.chosen && wave == 0)
      plan_row<BF16, VEC, true>(p, work, q, m, G, places);
    return;
  }
  if (!counts) fill_table(table);
  const bool binned = counts || q.need_p;
  uint32_t* count = reinterpret_cast<uint32_t*>(mass);
  if (binned)
    for (int i = threadIdx.x; i < (counts ? kBins / 2 : kBins);
         i += kMaxThreads)
      mass[i] = 0;
  __syncthreads();
  Weights wt;
  wt.init(table, top, q.T, q.min_p, places);
  const uint32_t min_key = least_allowed(q, wt, top);
  const float least = unordered(min_key);
  const CountBins bins(work.gmax, G, top, min_key, CountBins::few(q.k, live));
  const char* row = static_cast<const char*>(p.logits) +
                    m * p.s_row * (BF16 ? 2 : 4);
#pragma unroll 1
  for (int g = part.first + wave; g < part.end; g += kMaxThreads / 64) {
    // a group whose largest logit min-p drops has nothing to add
    if (work.gmax[g] < least) {
      if (!binned && lane == 0) work.sums[g] = 0;
      continue;
    }
    Group<BF16, VEC> v;
    v.load(row, g, p.V);
    if (counts) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int bin = bins(v.x[e]);
        if (bin < kBins) atomicAdd(&count[bin], 1u);
      }
      continue;
    }
    uint64_t sum = 0;
    const auto in = [&](float x, int) { return x >= least; };
    if (binned) {
      each_kept<BF16, VEC>(v, kept[wave], in, [&](float x) {
        const double d = wt.steps(x);
        const uint64_t w = wt.whole(d);
        if (w > 0) atomicAdd(&mass[wt.bin(d)], (unsigned long long)w);
      });
    } else {
      each_kept<BF16, VEC>(v, kept[wave], in,
                           [&](float x) { sum += wt.of(x); });
      sum = wave_sum64(sum);
      if (lane == 0) work.sums[g] = sum;
    }
  }
  if (binned) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kMaxThreads) {
      const uint64_t add = counts ? count[i] : mass[i];
      if (add > 0)
        atomicAdd((unsigned long long*)&work.sums[i], (unsigned long long)add);
    }
  }
  if (plans && last_of(&work.plan->arrived[0], per_row) && wave == 0)
    plan_row<BF16, VEC, true>(p, work, q, m, G, places);
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(64)
    kda_plan_kernel(SampleParams p, int G, int places) {
  const int m = blockIdx.x;
  const Work work(p, m, G);
  const int b = request_of_row(p, m, threadIdx.x);
  if (b < 0) {
    if (threadIdx.x == 0) work.plan->mode = kDecided;
    return;
  }
  plan_row<BF16, VEC, false>(p, work, Params(p, b, m), m, G, places);
}

// The token whose running weight passes u, by one wave: from the weights of
// the groups and the group that the border falls into.
template <bool BF16, bool VEC>
__device__ __forceinline__ void pick_token(const SampleParams& p,
                                           const Work& work,
                                           const Weights& wt, Threshold thr,
                                           float u, int m, int G) {
  const Found f = find_first<0>(
      work.sums, G, [&](uint64_t w) { return past_share(u, w); });
  const uint64_t target = past_share(u, f.total);
  Group<BF16, VEC> v;
  v.load(static_cast<const char*>(p.logits) + m * p.s_row * (BF16 ? 2 : 4),
         max(f.at, 0), p.V);
  uint64_t w[8], pre[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    w[e] = thr.keeps(v.x[e], v.index(e)) ? wt.of(v.x[e]) : 0;
  group_prefix<VEC>(w, pre);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (f.before + pre[e] < target && f.before + pre[e] + w[e] >= target)
      p.tokens[m] = v.index(e);
}

// The keys first <= key < last of the rows that list them, in any order.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
    kda_gather_kernel(SampleParams p, int G, int per_row) {
  const Part part(G, per_row);
  const int m = part.m;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const Work work(p, m, G);
  const Plan plan = *work.plan;
  if (plan.mode != kGather) return;
  // as floats; without a last key, one that nothing compares with
  const uint32_t last = plan.last;
  const float x_first = unordered(plan.first);
  const float x_last = last == 0xffffffffu ? __builtin_nanf("")
                                           : unordered(last);
  const auto in = [&](float x) { return x >= x_first && !(x >= x_last); };
  constexpr int kOwn = kPerWg / 4;           // groups of a wave
  const int g0 = part.first + wave * kOwn;
  int id[kOwn], groups = 0;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    id[i] = 0;
    const bool use = g0 + i < G && work.gmax[min(g0 + i, G - 1)] >= x_first;
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
      if (use && j == groups) id[j] = g0 + i;
    groups += use;
  }
  if (groups == 0) return;
  const char* row = static_cast<const char*>(p.logits) +
                    m * p.s_row * (BF16 ? 2 : 4);
  Group<BF16, VEC> v[kOwn];
#pragma unroll
  for (int j = 0; j < kOwn; ++j)
    if (j < groups) v[j].load(row, id[j], p.V);
  int own = 0;
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    if (j >= groups) break;
#pragma unroll
    for (int e = 0; e < 8; ++e) own += in(v[j].x[e]);
  }
  // places: one addition for the wave, and the lanes' own by the binary
  // digits of their numbers
  static_assert(8 * kOwn < 64, "digits");
  uint32_t all = 0, at = 0;
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const uint64_t has = __ballot(own >> i & 1);
    all += uint32_t(__popcll(has)) << i;
    at += __builtin_amdgcn_mbcnt_hi(
              uint32_t(has >> 32),
              __builtin_amdgcn_mbcnt_lo(uint32_t(has), 0))
          << i;
  }
  if (all == 0) return;
  uint32_t base = 0;
  if (lane == 0) base = atomicAdd(&work.plan->n, all);
  at += uint32_t(uniform(int(base)));
#pragma unroll
  for (int j = 0; j < kOwn; ++j) {
    if (j >= groups) break;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (in(v[j].x[e])) {
        if (at < kList)
          work.list[at] = uint64_t(ordered(v[j].x[e])) << 32 |
                          (0xffffffffu - uint32_t(v[j].index(e)));
        ++at;
      }
  }
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kRowThreads)
    __attribute__((amdgpu_waves_per_eu(6)))
    kda_list_kernel(SampleParams p, int G, int places) {
  extern __shared__ __align__(16) char smem[];
  RowSmem& sm = *reinterpret_cast<RowSmem*>(smem);
  const int m = blockIdx.x, tid = threadIdx.x;
  const Work work(p, m, G);
  const Plan plan = *work.plan;
  if (plan.mode != kGather && plan.mode != kSearch) return;
  const int b = request_of_row(p, m, tid & 63);
  if (b < 0) return;
  const Params q(p, b, m);
  const int k = q.k;
  fill_table(sm.table);
  Weights wt;
  wt.init(sm.table, plan.top, q.T, q.min_p, places);
  Threshold thr{plan.min_key, p.V};
  if (plan.mode == kGather && plan.n >= 1 && plan.n <= kList) {
    const int n = int(plan.n);
    for (int i = tid; i < n; i += kRowThreads) sm.key[i] = work.list[i];
    sort_list(sm, n);
    int kept = q.need_k ? min(n, k) : n;
    // weights: kept beside a short list, computed at each use for a long one
    const bool stored = n <= kList / 2;
    uint64_t* const w = sm.key + kList / 2;
    if (stored)
      for (int i = tid; i < kept; i += kRowThreads)
        w[i] = wt.of(unordered(uint32_t(sm.key[i] >> 32)));
    const auto weight = [&](int i) {
      return stored ? w[i] : wt.of(unordered(uint32_t(sm.key[i] >> 32)));
    };
    __syncthreads();
    if (q.need_p) {
      find_prefix<kPerList>(sm, weight, kept, [&](uint64_t all) {
        return share_of(q.top_p, q.need_k ? all : plan.mass) - plan.before;
      });
      if (sm.found >= 0) kept = sm.found + 1;
    }
    if (!q.need_k) {
      // the last kept one is the threshold pair
      const uint64_t end = sm.key[kept - 1];
      thr = Threshold{uint32_t(end >> 32), int(0xffffffffu - uint32_t(end))};
    } else {
      // the index whose running weight passes u: by its upper ten bits, then
      // by its lower ten
      uint64_t* bins = reinterpret_cast<uint64_t*>(sm.gmax);
      static_assert(kMaxGroups * kGroup <= 1 << 20 &&
                    sizeof(sm.gmax) >= 1024 * sizeof(uint64_t), "index bits");
      uint64_t target = 0;
      int high = 0;
#pragma unroll 1
      for (int pass = 0; pass < 2; ++pass) {
        __syncthreads();
        for (int i = tid; i < 1024; i += kRowThreads) bins[i] = 0;
        __syncthreads();
        for (int i = tid; i < kept; i += kRowThreads) {
          const int at = int(0xffffffffu - uint32_t(sm.key[i]));
          if (pass == 0 || at >> 10 == high)
            atomicAdd((unsigned long long*)&bins[pass == 0 ? at >> 10
                                                           : at & 1023],
                      (unsigned long long)weight(i));
        }
        __syncthreads();
        find_prefix<kPer1k>(sm, [&](int i) { return bins[i]; }, 1024,
                            [&](uint64_t all) {
                              if (pass == 0) target = past_share(q.u, all);
                              return target;
                            });
        target -= sm.before;
        if (pass == 0) high = max(sm.found, 0);
      }
      if (tid == 0) {
        p.tokens[m] = high << 10 | max(sm.found, 0);
        work.plan->mode = kDecided;
      }
      return;
    }
  } else {
    // ---- no list holds them: thresholds by radix search ----
    const uint32_t min_key = plan.min_key;
    const Row<BF16, VEC> row{static_cast<const char*>(p.logits) +
                                 m * p.s_row * (BF16 ? 2 : 4),
                             p.V, G, sm};
    uint64_t mass = plan.mass;
    for (int g = tid; g < G; g += kRowThreads) sm.gmax[g] = work.gmax[g];
    const auto used = [&](int g) { return ordered(sm.gmax[g]) >= min_key; };
    __syncthreads();
    if (q.need_k) {
      uint64_t n = 0;
      row.each(used, [&](float x, int) { n += ordered(x) >= min_key; });
      row_scan(n, sm.red, &n);
      if (n > uint64_t(k))
        thr = search<BF16, VEC>(row, min_key, thr, uint64_t(k),
                                [](float) { return uint64_t(1); });
      if (q.need_p) {
        uint64_t sum = 0;
        row.each(used, [&](float x, int i) {
          if (ordered(x) >= min_key && thr.keeps(x, i)) sum += wt.of(x);
        });
        row_scan(sum, sm.red, &mass);
      }
    }
    if (q.need_p)
      thr = search<BF16, VEC>(row, min_key, thr, share_of(q.top_p, mass),
                              [&](float x) { return wt.of(x); });
  }
  // the kept weights of each group are left to many workgroups
  if (tid == 0) {
    work.plan->key = thr.key;
    work.plan->index = thr.index;
    work.plan->mode = kKept;
  }
}

// Kept weights of each group of the rows with a threshold pair, and their
// token, or that of a row whose sums are there.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kMaxThreads)
    kda_kept_sums_kernel(SampleParams p, int G, int per_row, int places,
                         bool picks) {
  __shared__ double table[kSteps];
  __shared__ float kept[kMaxThreads / 64][kGroup];
  const Part part(G, per_row);
  const int m = part.m;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const Work work(p, m, G);
  const Mode mode = work.plan->mode;
  if (mode != kKept && !(picks && mode == kSummed && part.chosen)) return;
  const Plan plan = *work.plan;
  const Threshold thr{plan.key, plan.index};
  const int b = request_of_row(p, m, lane);
  if (b < 0) return;
  const Params q(p, b, m);
  fill_table(table);
  __syncthreads();
  Weights wt;
  wt.init(table, plan.top, q.T, q.min_p, places);
  // (the threshold is never below what min-p allows)
  const float least = unordered(thr.key);
  const char* row = static_cast<const char*>(p.logits) +
                    m * p.s_row * (BF16 ? 2 : 4);
  if (mode == kSummed) {
    if (wave == 0) pick_token<BF16, VEC>(p, work, wt, thr, q.u, m, G);
    return;
  }
#pragma unroll 1
  for (int g = part.first + wave; g < part.end; g += kMaxThreads / 64) {
    uint64_t sum = 0;
    if (work.gmax[g] >= least) {
      Group<BF16, VEC> v;
      v.load(row, g, p.V);
      each_kept<BF16, VEC>(
          v, kept[wave], [&](float x, int i) { return thr.keeps(x, i); },
          [&](float x) { sum += wt.of(x); });
      sum = wave_sum64(sum);
    }
    if (lane == 0) work.sums[g] = sum;
  }
  if (picks && last_of(&work.plan->arrived[1], per_row) && wave == 0)
    pick_token<BF16, VEC>(p, work, wt, thr, q.u, m, G);
}

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(64)
    kda_pick_kernel(SampleParams p, int G, int places) {
  __shared__ double table[kSteps];
  const int m = blockIdx.x;
  const Work work(p, m, G);
  const Plan plan = *work.plan;
  if (plan.mode != kKept && plan.mode != kSummed) return;
  const int b = request_of_row(p, m, threadIdx.x);
  if (b < 0) return;
  const Params q(p, b, m);
  fill_table(table);
  __syncthreads();
  Weights wt;
  wt.init(table, plan.top, q.T, q.min_p, places);
  pick_token<BF16, VEC>(p, work, wt, Threshold{plan.key, plan.index}, q.u, m,
                        G);
}

// One thread per request: leading rows whose token is the window's next one.
__global__ void __launch_bounds__(256) kda_accept_kernel(SampleParams p) {
  const int b = blockIdx.x * 256 + threadIdx.x;
  if (b >= p.B) return;
  const int s = min(max(p.qsl[b], 0), p.M);
  const int e = min(max(p.qsl[b + 1], s), p.M);
  int t = s;
  while (t + 1 < e && p.tokens[t] == p.draft[t + 1]) ++t;
  p.accepted[b] = s < e ? t - s + 1 : 0;
  p.next[b] = s < e ? p.tokens[t] : -1;
}

static_assert(sizeof(RowSmem) <= 64 * 1024, "LDS of a launch");

template <bool BF16, bool VEC>
int launch_rows(const SampleParams& p, int G, int places,
                hipStream_t stream) {
  const int per_row = (G + kPerWg - 1) / kPerWg;
  const dim3 parts(uint32_t(p.M) * uint32_t(per_row));
  launch_kernel(kda_group_max_kernel<BF16, VEC>, parts, dim3(kMaxThreads), 0,
                stream, p, G, per_row);
  // Half as many workgroups, each with bins of its own, for the sums of eight
  // a CU and more (times of a call: 640 rows of 131072 with top-k 1000 261 us
  // against 285, 640 of 32000 98 against 106, 128 of 131072 77 against 83; 96
  // of 131072 69 both; with fewer the whole number is quicker: 256 rows of
  // 32000 without filters 33 against 38, 32 of 131072 27 against 35).
  const bool many = int64_t(p.M) * per_row >= 2048;
  // Up to 128 workgroups, a row's last one plans and picks (4 rows of 131072:
  // 22 us a call against 26 without filters, 49 against 51 with top-p; 32 of
  // 32000: 22 against 25, 49 against 48).  More of them wait for each other's
  // releases (16 rows of 131072 with top-p: 55 against 53; 127: 199 against
  // 105).
  const bool last = int64_t(p.M) * per_row <= 128;
  const int sums_wg = many ? 2 * kPerWg : kPerWg;
  const int sums_row = (G + sums_wg - 1) / sums_wg;
  launch_kernel(kda_row_sums_kernel<BF16, VEC>,
                dim3(uint32_t(p.M) * uint32_t(sums_row)), dim3(kMaxThreads), 0,
                stream, p, G, sums_row, sums_wg, places, last);
  if (!last)
    launch_kernel(kda_plan_kernel<BF16, VEC>, dim3(p.M), dim3(64), 0, stream,
                  p, G, places);
  if (p.top_k || p.top_p) {
    launch_kernel(kda_gather_kernel<BF16, VEC>, parts, dim3(kMaxThreads), 0,
                  stream, p, G, per_row);
    launch_kernel(kda_list_kernel<BF16, VEC>, dim3(p.M), dim3(kRowThreads),
                  sizeof(RowSmem), stream, p, G, places);
  }
  launch_kernel(kda_kept_sums_kernel<BF16, VEC>, parts, dim3(kMaxThreads), 0,
                stream, p, G, per_row, places, last);
  if (!last)
    launch_kernel(kda_pick_kernel<BF16, VEC>, dim3(p.M), dim3(64), 0, stream,
                  p, G, places);
  return int(hipGetLastError());
}

}  // namespace

int64_t sample_work_bytes(int64_t M, int64_t V) {
  if (M < 0 || V < 1 || M > 0x7fffffff || V > int64_t(kMaxGroups) * kGroup)
    return 0;
  const int64_t G = (V + kGroup - 1) / kGroup;
  // work items of the launches: 256 per kPerWg groups, 512 per row
  if (M * ((G + kPerWg - 1) / kPerWg) > 0xffffffff / kMaxThreads ||
      M > 0xffffffff / kRowThreads)
    return 0;
  return Work::bytes(M, G) + 256;
}

int launch_sample(const SampleParams& p, bool bf16, hipStream_t stream) {
  const int G = (p.V + kGroup - 1) / kGroup;
  // binary places of a weight: sums of V of them stay below 2^62, and one
  // below 2^51, where adding 2^52 still rounds to whole numbers
  int bits = 0;
  while ((int64_t(1) << bits) < p.V) ++bits;
  const int places = bits < 16 ? 46 : 62 - bits;
  const int elem = bf16 ? 2 : 4;
  const bool vec = reinterpret_cast<uintptr_t>(p.logits) % 16 == 0 &&
                   p.s_row * elem % 16 == 0;
  if (p.M > 0) {
    const int e = bf16 ? (vec ? launch_rows<true, true>(p, G, places, stream)
                              : launch_rows<true, false>(p, G, places, stream))
                       : (vec ? launch_rows<false, true>(p, G, places, stream)
                              : launch_rows<false, false>(p, G, places,
                                                          stream));
    if (e != 0) return e;
  }
  if (p.draft && p.B > 0)
    launch_kernel(kda_accept_kernel, dim3((p.B - 1) / 256 + 1), dim3(256), 0,
                  stream, p);
  return int(hipGetLastError());
}

}  // namespace kda
