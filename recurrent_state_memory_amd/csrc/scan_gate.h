// scan_gate.h -- the channelwise recurrence's gates in fp32.
//
//   w = e^-|d|,  softplus(d) = max(d, 0) + log1p(w),  u = A softplus(d),
//   a = e^-u,  m = 1 - a^2,  sigmoid(g) = 1 / (1 + e^-g)
//
// Channels that forget slowly have u of 1e-3 and less, where a rounds to 24
// bits but m = 2u - ... must keep its relative accuracy (the input is scaled by
// sqrt(m)).  So log1p corrects the rounding of 1 + w (s = fl(1 + w), c = w - (s
// - 1) exactly, log1p(w) = log s + c / s, and c / s = c to within 2^-24 of the
// result: where c matters s is near 1), and m comes from the series of
// 1 - e^-z below z = 2u = 1/4 and from 1 - a a above it (relative error 4e-7 at
// the border).  exp, log, rcp and sqrt are the hardware's, 1 ulp each.
#pragma once
#include <hip/hip_runtime.h>

namespace gdr {
namespace scan {

constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.69314718f;

__device__ inline float exp_fast(float x) { return __builtin_amdgcn_exp2f(x * kLog2e); }

// e^-|d| and softplus(d)
__device__ inline float softplus(float d, float& w) {
  w = __builtin_amdgcn_exp2f(-__builtin_fabsf(d) * kLog2e);
  const float s = 1.f + w;
  const float c = w - (s - 1.f);
  return fmaxf(d, 0.f) + fmaf(__builtin_amdgcn_logf(s), kLn2, c);
}

// 1 - e^-2u, a = e^-u
__device__ inline float one_minus_sq(float u, float a) {
  const float z = 2.f * u;
  float p = fmaf(z, -1.f / 720.f, 1.f / 120.f);
  p = fmaf(z, p, -1.f / 24.f);
  p = fmaf(z, p, 1.f / 6.f);
  p = fmaf(z, p, -0.5f);
  p = fmaf(z, p, 1.f);
  return z < 0.25f ? z * p : fmaf(-a, a, 1.f);
}

__device__ inline float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.f + exp_fast(-g)); }

}  // namespace scan
}  // namespace gdr
