// Device pieces shared by the prefill and the decode of a KDA layer: the
// gate, with a softplus that keeps its relative accuracy where it is small (a
// state carries the errors of hundreds of decays near 1, which the verify's
// few steps do not), and the parameters.
#pragma once

#include "kda_device.hpp"
#include "kda_internal.hpp"

namespace kda {

// e^x by the hardware exponential of x log2(e): the product's rounding makes
// a relative error of up to (|x| + 1) 2^-23.  That is an ulp where it counts:
// a sigmoid or softplus at a large |x| is 1, x, or too small to matter, and a
// decay e^g at a large |g| leaves nothing to be wrong about.
__device__ __forceinline__ float exp_(float x) { return __expf(x); }

__device__ __forceinline__ float sigmoid_(float x) {
  return rcp_(1.0f + exp_(-x));
}

__device__ __forceinline__ float silu_(float x) { return x * sigmoid_(x); }

// ln(1 + e) for 0 <= e <= 1, relative to its value: 2 atanh(z) with
// z = e / (2 + e).  atanh(z) / z over z^2 <= 1/9 is the polynomial through its
// values at the five Chebyshev nodes, 4e-9 off, 8e-9 with its coefficients in
// fp32.
__device__ __forceinline__ float log1p_(float e) {
  const float z = e * rcp_(2.0f + e);
  const float s = z * z;
  float p = 0.14078889f;
  p = __builtin_fmaf(p, s, 0.13982579f);
  p = __builtin_fmaf(p, s, 0.20012298f);
  p = __builtin_fmaf(p, s, 0.33333161f);
  p = __builtin_fmaf(p, s, 1.0f);
  return 2.0f * z * p;
}

// Log-decay of one channel (the verify's kda_gate): bounded, or -A softplus,
// with softplus the identity above 20 and max(x, 0) + ln(1 + e^-|x|) below,
// which keeps its relative accuracy where it is small.
__device__ __forceinline__ float layer_gate(float x, float A, bool use_lb,
                                            float lb) {
  if (use_lb) return lb * sigmoid_(A * x);
  const float sp =
      x > 20.0f ? x : fmaxf(x, 0.0f) + log1p_(exp_(-fabsf(x)));
  return -A * sp;
}

// Inputs, parameters and pools of one layer.  Strides in elements.
struct LayerParams {
  const void* mixed_qkv;    // [T, 3HD]
  const void* raw_gate;     // [T, HD]
  const void* raw_beta;     // [T, H]
  const float* A_log;       // [H]
  const float* dt_bias;     // [H, D]
  float* state;             // [N, H, D, D]
  void* out;                // [T, HD]
  void* conv_state;         // conv: [N, 3HD, Lc] seen dim-first
  const void* conv_weight;  // conv: [3HD, W]
  int64_t s_x, s_g, s_beta, s_out, s_slot;
  int64_t s_cs_slot, s_cs_chan, s_cs_tok, s_w_chan, s_w_tap;
  const int32_t* slots;     // [B]
  const int32_t* accepted;  // [B] or null (1)
  int32_t B, H, N, Q, null_id;
  int32_t flags;            // kOutBf16 | kWBf16 | kLowerBound | kNoConv
  float lb;
};

__device__ __forceinline__ bool live_slot(const LayerParams& p, int slot) {
  return slot > p.null_id && slot >= 0 && slot < p.N;
}

// Offset of the oldest of the three history inputs in a slot's conv rows.
__device__ __forceinline__ int history_at(const LayerParams& p, int b) {
  return (p.accepted ? min(max(p.accepted[b], 1), p.Q) : 1) - 1;
}

}  // namespace kda
