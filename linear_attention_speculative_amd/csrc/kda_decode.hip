// Single-token decode of a KDA layer for gfx950: for every (request, head)
// one step of the recurrence, from the request's state slot to its final
// slot, with the short convolution and its history in the same launch.
//
// With a = e^g, k_hat and q normalised (see the verify), the row v of the
// state takes
//   u_v = sum_k S_vk a_k k_hat_k          c_v = beta (v_v - u_v)
//   S'_vk = S_vk a_k + c_v k_hat_k
//   o_v = sum_k S'_vk q_k = sum_k S_vk a_k q_k + c_v (k_hat . q)
// so both dot products come from the tile as it was loaded and the row is
// finished without a second pass.  The norms are applied after the dot
// products: every row group spans all channels, so it forms k.k, q.q and k.q
// beside its rows' sums and no workgroup-wide reduction is needed.
//
// The kernel is a stream: the D x D fp32 tile of a (request, head) is read
// and written once (128 KiB at D = 128), everything else is a few hundred
// bytes.  One workgroup takes one tile, held in registers; its loads are
// issued first, so that the convolution and the gates run under them.
// Workgroups follow the XCD-aware order of the commit: each XCD streams one
// contiguous eighth of the items.  251 requests of 32 heads (1.05 GB read and
// written): 196 us, 5.4 TB/s; one request: 6.2 us, the latency of its loads.
#include "kda_layer.hpp"
#include "kda_serving.hpp"

namespace kda {
namespace {

template <int D>
struct DecodeCfg {
  static constexpr int NT = D >= 128 ? 512 : (D == 64 ? 256 : 64);
  static constexpr int L = D / 4;       // lanes per state row (float4)
  static constexpr int RPP = NT / L;    // rows per pass
  static constexpr int PASSES = D / RPP;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(DecodeCfg<D>::NT)
    kda_decode_kernel(DecodeParams p) {
  using C = DecodeCfg<D>;
  typedef typename Act<BF16>::T T;
  __shared__ __align__(16) float qkv[3][D];
  __shared__ __align__(16) float decay[D];
  const LayerParams& y = p.y;
  const int tid = threadIdx.x;

  // workgroup -> (request, head), each XCD a contiguous eighth
  const int n = gridDim.x, i = blockIdx.x;
  const int per = (n + 7) / 8, full = n % 8 == 0 ? 8 : n % 8;
  const int x = i % 8;
  const int item = x * per - max(0, x - full) + i / 8;
  const int b = item / y.H, h = item - b * y.H;

  const int slot = y.slots[b];
  const int64_t hd = int64_t(h) * D;
  if (!live_slot(y, slot)) {
    for (int d = tid; d < D; d += C::NT)
      st_elem(y.out, b * y.s_out + hd + d, 0.0f, y.flags & kOutBf16);
    return;
  }
  const int fin = p.final_slots ? p.final_slots[b] : slot;
  const bool keep = live_slot(y, fin);

  const int lane = tid % C::L, row0 = tid / C::L;
  const float* src = y.state + slot * y.s_slot + hd * D;
  f4 s[C::PASSES];
#pragma unroll
  for (int r = 0; r < C::PASSES; ++r)
    s[r] = ld_stream(src + (row0 + r * C::RPP) * D + lane * 4);

  const T* xr = static_cast<const T*>(y.mixed_qkv) + b * y.s_x;
  const int64_t HD = int64_t(y.H) * D;
  const bool conv = !(y.flags & kNoConv);
  for (int j = tid; j < 3 * D; j += C::NT) {
    const int part = j / D;
    const int64_t ch = part * HD + hd + (j - part * D);
    const T xn = xr[ch];
    float v = Act<BF16>::f(xn);
    if (conv) {
      T* cs = static_cast<T*>(y.conv_state) + ch * y.s_cs_chan;
      const T* old = cs + slot * y.s_cs_slot + history_at(y, b) * y.s_cs_tok;
      const T h0 = old[0], h1 = old[y.s_cs_tok], h2 = old[2 * y.s_cs_tok];
      const int64_t w = ch * y.s_w_chan;
      const bool wb = y.flags & kWBf16;
      float acc = ld_elem(y.conv_weight, w, wb) * Act<BF16>::f(h0);
      acc += ld_elem(y.conv_weight, w + y.s_w_tap, wb) * Act<BF16>::f(h1);
      acc += ld_elem(y.conv_weight, w + 2 * y.s_w_tap, wb) * Act<BF16>::f(h2);
      acc += ld_elem(y.conv_weight, w + 3 * y.s_w_tap, wb) * v;
      v = silu_(acc);
      if (keep) {   // this thread alone reads and writes the channel
        T* to = cs + fin * y.s_cs_slot;
        to[0] = h1;
        to[y.s_cs_tok] = h2;
        to[2 * y.s_cs_tok] = xn;
      }
    }
    qkv[part][j - part * D] = v;
  }
  const float A = exp_(y.A_log[h]);
  for (int d = tid; d < D; d += C::NT) {
    const float xg =
        Act<BF16>::f(static_cast<const T*>(y.raw_gate)[b * y.s_g + hd + d]) +
        y.dt_bias[hd + d];
    decay[d] = exp_(layer_gate(xg, A, y.flags & kLowerBound, y.lb));
  }
  const float beta = sigmoid_(
      Act<BF16>::f(static_cast<const T*>(y.raw_beta)[b * y.s_beta + h]));
  lds_barrier();

  const f4 q = *reinterpret_cast<const f4*>(&qkv[0][lane * 4]);
  const f4 k = *reinterpret_cast<const f4*>(&qkv[1][lane * 4]);
  const f4 a = *reinterpret_cast<const f4*>(&decay[lane * 4]);
  float kk = 0, qq = 0, kq = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    kk += k[e] * k[e];
    qq += q[e] * q[e];
    kq += k[e] * q[e];
  }
  kk = group_sum<C::L>(kk);
  qq = group_sum<C::L>(qq);
  kq = group_sum<C::L>(kq);
  const float nk = 1.0f / sqrtf(kk + kNormEps);
  const float nq = 1.0f / (sqrtf(qq + kNormEps) * sqrtf(float(D)));
  const f4 kh = k * nk;
  const f4 ak = a * kh, aq = a * q * nq;
  kq *= nk * nq;

  float* dst = y.state + (keep ? fin * y.s_slot : 0) + hd * D;
#pragma unroll
  for (int r = 0; r < C::PASSES; ++r) {
    const int row = row0 + r * C::RPP;
    float u = 0, o = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      u += s[r][e] * ak[e];
      o += s[r][e] * aq[e];
    }
    u = group_sum<C::L>(u);
    o = group_sum<C::L>(o);
    const float c = beta * (qkv[2][row] - u);
    if (keep) st_stream(dst + row * D + lane * 4, s[r] * a + kh * c);
    if (lane == 0)
      st_elem(y.out, b * y.s_out + hd + row, o + c * kq,
              y.flags & kOutBf16);
  }
}

template <int D>
int launch_decode_dim(const DecodeParams& p, bool act_bf16,
                      hipStream_t stream) {
  const dim3 grid(uint32_t(p.y.B) * uint32_t(p.y.H));
  const dim3 block(DecodeCfg<D>::NT);
  if (act_bf16)
    launch_kernel(kda_decode_kernel<D, true>, grid, block, 0, stream, p);
  else
    launch_kernel(kda_decode_kernel<D, false>, grid, block, 0, stream, p);
  return int(hipGetLastError());
}

}  // namespace

int launch_decode(const DecodeParams& p, int D, bool act_bf16,
                  hipStream_t stream) {
  switch (D) {
    case 16: return launch_decode_dim<16>(p, act_bf16, stream);
    case 32: return launch_decode_dim<32>(p, act_bf16, stream);
    case 64: return launch_decode_dim<64>(p, act_bf16, stream);
    case 128: return launch_decode_dim<128>(p, act_bf16, stream);
    default: return int(hipErrorInvalidValue);
  }
}

}  // namespace kda
