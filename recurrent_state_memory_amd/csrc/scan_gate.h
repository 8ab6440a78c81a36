// scan_gate.h -- the channelwise recurrence's gates in fp32.
//
//   w = e^-|d|,  softplus(d) = max(d, 0) + log1p(w),  u = A softplus(d),
//   a = e^-u,  m = 1 - a^2,  sigmoid(g) = 1 / (1 + e^-g)
//
// Channels that forget slowly have u of 1e-3 and less, where a rounds to 24
// bits but m = 2u - ... must keep its relative accuracy (the input is scaled by
// sqrt(m)).  So log1p corrects the rounding of 1 + w (s = fl(1 + w), c = w - (s
// - 1) exactly, log1p(w) = log s + c / s, and c / s = c to within 2^-24 of the
// result: where c matters s is near 1).  And m is z q(z) below z = 2u = 1/2, with
// q a degree-4 fit of (1 - e^-z) / z at the Chebyshev nodes of [0, 1/2] (relative
// error 1.04e-7), and 1 - a a above it, where the rounding of a is at most 2 in m.
// exp, log, rcp and sqrt are the hardware's, 1 ulp each.  The scan kernels spend
// about as long on these as on memory, so the scale's products are formed once a
// channel.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {
namespace scan {

constexpr float kLog2e = 1.44269504f;
constexpr float kLn2 = 0.69314718f;

// A channel's scale A in the two forms that it is used in.
struct Scale {
  float exp2, twice;   // -A log2 e, 2 A
  __device__ explicit Scale(float A = 0.f) : exp2(-A * kLog2e), twice(2.f * A) {}
};

__device__ inline float softplus(float d, float& w, float& s) {
  w = __builtin_amdgcn_exp2f(-__builtin_fabsf(d) * kLog2e);
  s = 1.f + w;
  const float c = w - (s - 1.f);
  // max(d, 0) on the bits, one instruction (fmaxf takes two), and at most the largest
  // float, so that a = 0 of an infinite d has no 0 * Inf in its gradients; a NaN d
  // comes through w
  const int bits = __float_as_int(d), pos = bits > 0 ? bits : 0;
  return __int_as_float(pos < 0x7f7fffff ? pos : 0x7f7fffff) + fmaf(__builtin_amdgcn_logf(s), kLn2, c);
}
__device__ inline float softplus(float d) {
  float w, s;
  return softplus(d, w, s);
}
// with sigmoid(d) = 1 / (1 + w) or w / (1 + w)
__device__ inline float softplus(float d, float& sig) {
  float w, s;
  const float sp = softplus(d, w, s);
  const float r = __builtin_amdgcn_rcpf(s);
  sig = d > 0.f ? r : w * r;
  return sp;
}
__device__ inline float decay(const Scale& A, float sp) { return __builtin_amdgcn_exp2f(A.exp2 * sp); }

__device__ inline float one_minus_sq(const Scale& A, float sp, float a) {
  const float z = A.twice * sp;
  float q = fmaf(z, 0x1.bc858cp-8f, -0x1.4ffafp-5f);
  q = fmaf(z, q, 0x1.55192ep-3f);
  q = fmaf(z, q, -0x1.fffe22p-2f);
  q = fmaf(z, q, 0x1.fffffep-1f);
  return z < 0.5f ? z * q : fmaf(-a, a, 1.f);
}

__device__ inline float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -kLog2e));
}

// A gate's s = sigmoid(g) and 1 - s in one number, each with its full relative
// accuracy: the smaller of the two, min(s, 1 - s) = e / (1 + e) with e = e^-|g|, and
// g's sign, which says which one it is.  Its fraction x - floor(x) is 1 - s, that of its
// negative s.  An open gate's number stays off 0, whose negative has no fraction: at
// least 2^-126 (the larger of the bits, of which a closed gate's have the sign set), so a
// closed gate's s is exactly 0.
__device__ inline float gate_pair(float g) {
  const float e = __builtin_amdgcn_exp2f(-__builtin_fabsf(g) * kLog2e);
  const uint32_t bits = __float_as_uint(__builtin_copysignf(e * __builtin_amdgcn_rcpf(1.f + e), g));
  return __uint_as_float(bits > 0x00800000u ? bits : 0x00800000u);
}
__device__ inline float gate_open(float pair) { return __builtin_amdgcn_fractf(-pair); }
__device__ inline float gate_shut(float pair) { return __builtin_amdgcn_fractf(pair); }

}  // namespace scan
}  // namespace gdr
