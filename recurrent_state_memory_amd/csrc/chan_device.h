// chan_device.h -- device helpers shared by the channelwise operators: element
// and vector access in bf16 and fp32, the 8-bit checkpoint codes, wave sums.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {
namespace chan {

// One element as fp32 and back (bf16 stores round to nearest even).
__device__ inline float ld(const float* p) { return *p; }
__device__ inline float ld(const __bf16* p) { return (float)*p; }
__device__ inline void st(float* p, float v) { *p = v; }
__device__ inline void st(__bf16* p, float v) { *p = (__bf16)v; }

// Exponent byte of a group from its largest finite magnitude (fp32 bits): the
// least E in [1, 254] with max <= 448 * 2^(E - 127).  448 = 1.75 * 2^8, so E is
// the maximum's own exponent less 8, one more if its fraction exceeds 1.75.
__device__ inline int ckpt8_exponent(uint32_t max_bits) {
  const int e = (int)(max_bits >> 23) - 8 + ((max_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e;
}
// |x| as bits, 0 for NaN and Inf, for the group's maximum
__device__ inline uint32_t finite_mag_bits(float x) {
  const uint32_t b = __float_as_uint(x) & 0x7fffffffu;
  return b < 0x7f800000u ? b : 0u;
}
// 2^(E - 127) and its inverse, E in [1, 254]: both are normal numbers up to
// E = 253; E is at most 247 here, and a foreign exponent byte only feeds scale_of.
__device__ inline float scale_of(uint32_t e) {
  return e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}
__device__ inline float inv_scale_of(int e) { return __uint_as_float((uint32_t)(254 - e) << 23); }

// Two (four) scaled values as e4m3 codes, RNE.  The scaled magnitude is at most
// 448, so nothing saturates; NaN and Inf are made NaN codes here rather than
// left to the conversion's overflow rule.
__device__ inline float no_inf(float x) { return __builtin_fabsf(x) == __builtin_inff() ? __builtin_nanf("") : x; }
__device__ inline uint32_t pack4_e4m3(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(no_inf(a), no_inf(b), 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(no_inf(c), no_inf(d), r, true);
  return (uint32_t)r;
}
__device__ inline uint8_t pack1_e4m3(float a) {
  return (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(no_inf(a), 0.f, 0, false);
}
// Codes as numbers (byte i of c).
template <int I>
__device__ inline float code_f32(uint32_t c) {
  return __builtin_amdgcn_cvt_f32_fp8((int)c, I);
}
__device__ inline float code1_f32(uint8_t c) { return code_f32<0>(c); }

__device__ inline float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off);
  return v;
}

}  // namespace chan
}  // namespace gdr
