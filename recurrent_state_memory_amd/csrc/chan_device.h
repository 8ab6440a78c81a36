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

// 16 bytes of a row: 8 bf16 or 4 fp32 values, aligned to the element alone (rows of
// any length follow each other; the hardware takes vector accesses at any address).
// The row's last run may be shorter: `n` values from p exist.
typedef uint32_t raw4 __attribute__((ext_vector_type(4)));
typedef uint32_t raw2 __attribute__((ext_vector_type(2)));
template <typename T>
struct Run;
template <>
struct Run<float> {
  static constexpr int N = 4;
  typedef raw4 at4 __attribute__((aligned(4), may_alias));
  static __device__ inline raw4 load(const float* p, int n) {
    if (n >= N) return *(const at4*)p;
    raw4 r = {0u, 0u, 0u, 0u};
    if (n > 0) r[0] = __float_as_uint(p[0]);
    if (n > 1) r[1] = __float_as_uint(p[1]);
    if (n > 2) r[2] = __float_as_uint(p[2]);
    return r;
  }
  static __device__ inline float get(const raw4& r, int k) { return __uint_as_float(r[k]); }
  static __device__ inline void store(float* p, int n, const float (&v)[N]) {
    if (n >= N) {
      *(at4*)p = raw4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n) p[k] = v[k];
    }
  }
};
template <>
struct Run<__bf16> {
  static constexpr int N = 8;
  typedef raw4 at2 __attribute__((aligned(2), may_alias));
  static __device__ inline raw4 load(const __bf16* p, int n) {
    if (n >= N) return *(const at2*)p;
    raw4 r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < N - 1; ++k)
      if (k < n) r[k >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, p[k]) << (16 * (k & 1));
    return r;
  }
  static __device__ inline float get(const raw4& r, int k) {
    return __uint_as_float(k & 1 ? r[k >> 1] & 0xffff0000u : r[k >> 1] << 16);
  }
  static __device__ inline void store(__bf16* p, int n, const float (&v)[N]) {
    if (n >= N) {
      typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
      bf16x8 h;
#pragma unroll
      for (int k = 0; k < N; ++k) h[k] = (__bf16)v[k];
      *(at2*)p = __builtin_bit_cast(raw4, h);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n) p[k] = (__bf16)v[k];
    }
  }
};
// The same run of NC values kept as 8-bit codes (NC = 8 or 4).
template <int NC>
struct Codes;
template <>
struct Codes<8> {
  using R = raw2;
  typedef raw2 at1 __attribute__((aligned(1), may_alias));
  static __device__ inline R load(const uint8_t* p, int n) {
    if (n >= 8) return *(const at1*)p;
    R r = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 7; ++k)
      if (k < n) r[k >> 2] |= (uint32_t)p[k] << (8 * (k & 3));
    return r;
  }
  static __device__ inline void store(uint8_t* p, int n, const R& r) {
    if (n >= 8) {
      *(at1*)p = r;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < n) p[k] = (uint8_t)(r[k >> 2] >> (8 * (k & 3)));
    }
  }
  static __device__ inline void unpack(const R& r, float (&v)[8]) {
    v[0] = code_f32<0>(r[0]);
    v[1] = code_f32<1>(r[0]);
    v[2] = code_f32<2>(r[0]);
    v[3] = code_f32<3>(r[0]);
    v[4] = code_f32<0>(r[1]);
    v[5] = code_f32<1>(r[1]);
    v[6] = code_f32<2>(r[1]);
    v[7] = code_f32<3>(r[1]);
  }
  static __device__ inline R pack(const float (&v)[8], float inv) {
    return R{pack4_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
             pack4_e4m3(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
  }
};
template <>
struct Codes<4> {
  using R = uint32_t;
  typedef uint32_t at1 __attribute__((aligned(1), may_alias));
  static __device__ inline R load(const uint8_t* p, int n) {
    if (n >= 4) return *(const at1*)p;
    R r = 0u;
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) r |= (uint32_t)p[k] << (8 * k);
    return r;
  }
  static __device__ inline void store(uint8_t* p, int n, const R& r) {
    if (n >= 4) {
      *(at1*)p = r;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k < n) p[k] = (uint8_t)(r >> (8 * k));
    }
  }
  static __device__ inline void unpack(const R& r, float (&v)[4]) {
    v[0] = code_f32<0>(r);
    v[1] = code_f32<1>(r);
    v[2] = code_f32<2>(r);
    v[3] = code_f32<3>(r);
  }
  static __device__ inline R pack(const float (&v)[4], float inv) {
    return pack4_e4m3(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv);
  }
};

// Sum (maximum) over L neighbouring lanes, L a power of two up to 64.
template <int L>
__device__ inline float lane_sum(float v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off);
  return v;
}
template <int L>
__device__ inline uint32_t lane_max(uint32_t v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) {
    const uint32_t o = __shfl_xor(v, off);
    v = o > v ? o : v;
  }
  return v;
}

}  // namespace chan
}  // namespace gdr
