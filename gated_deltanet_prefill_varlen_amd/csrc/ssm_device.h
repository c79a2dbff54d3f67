// Device helpers of the state space layers: the convolution with its bias and
// the steps.
#pragma once

#include "gdn_device.h"
#include "ssm_internal.h"

namespace gdn {

// 2^POW2 silu(bias + the four taps), taps and bias scaled by -log2(e)
// (conv_tap), in the order of conv4_silu; not rounded.
template <int POW2 = 0>
__device__ __forceinline__ float conv4_bias_silu(float b, float w0, float w1, float w2, float w3, float x0, float x1,
                                                 float x2, float x3) {
  constexpr float k = kNegLog2e / (1 << POW2);
  float zs = fmaf(w0, x0, b);
  zs = fmaf(w1, x1, zs);
  zs = fmaf(w2, x2, zs);
  zs = fmaf(w3, x3, zs);
  return zs * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_exp2f(zs), k, k));
}

// The step of a head at a token: clamp(softplus(raw + bias)).  softplus(v) =
// max(v, 0) + log(1 + e^-|v|), whose last term keeps its relative precision
// for far negative v (log1pf).  NaN stays NaN through both.
__device__ __forceinline__ float ssm_step(const SsmLayer& l, const void* dt, int64_t at, int h) {
  float v = l.dt_f32 ? static_cast<const float*>(dt)[at] : bf16_to_f32(static_cast<const uint16_t*>(dt)[at]);
  if (l.dt_bias) v += l.dt_bias[h];
  if (l.softplus) v = fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
  return v < l.dt_min ? l.dt_min : v > l.dt_max ? l.dt_max : v;
}

}  // namespace gdn
