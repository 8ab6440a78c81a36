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

// Scaled values as e4m3 codes, RNE.  The scaled magnitude is at most 448, so nothing
// saturates; Inf is made NaN before rather than left to the conversion's rule.
__device__ inline float no_inf(float x) { return __builtin_fabsf(x) == __builtin_inff() ? __builtin_nanf("") : x; }
__device__ inline uint32_t pack4_e4m3(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
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

// Sum (maximum) over L neighbouring lanes, L a power of two from 2 to 64, in every
// one of them.  Within rows of 16 lanes by rotation (DPP, no LDS), across rows by
// the lane swaps: with both operands v, permlane16_swap leaves the even and the odd
// rows' values in its two results, permlane32_swap the lower and the upper half's.
template <int ROR>
__device__ inline uint32_t row_ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + ROR, 0xf, 0xf, false);
}
template <int L, typename OP>
__device__ inline uint32_t lane_join(uint32_t v, OP op) {
  static_assert(L == 2 || L == 4 || L == 8 || L == 16 || L == 32 || L == 64, "lanes");
  if constexpr (L <= 8) {   // up to eight lanes of a row: exchanges within them
    v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false));                           // lane ^ 1
    if constexpr (L >= 4) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false));     // lane ^ 2
    if constexpr (L == 8) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, false));    // 7 - lane
    return v;
  } else {
    v = op(v, row_ror<8>(v));
    v = op(v, row_ror<4>(v));
    v = op(v, row_ror<2>(v));
    v = op(v, row_ror<1>(v));
    if constexpr (L >= 32) {
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      v = op(r[0], r[1]);
    }
    if constexpr (L == 64) {
      const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      v = op(r[0], r[1]);
    }
    return v;
  }
}
template <int L>
__device__ inline float lane_sum(float v) {
  return __uint_as_float(lane_join<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int L>
__device__ inline uint32_t lane_max(uint32_t v) {
  return lane_join<L>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// 8-bit codes of a run that lies in a group of 128 values held by L lanes side by
// side, and the group's exponent.  A group without NaN and Inf, nearly every one,
// takes its maximum from the magnitudes' bits as they are.
template <typename T, int L>
__device__ inline typename Codes<Run<T>::N>::R pack_run(const raw4& r, int& e) {
  constexpr int N = Run<T>::N;
  float v[N];
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = Run<T>::get(r, k);
  uint32_t m = 0;
  if constexpr (N == 8) {   // bf16: two magnitudes to a register
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 h = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) h = __builtin_elementwise_max(h, __builtin_bit_cast(u16x2, r[i] & 0x7fff7fffu));
    m = (uint32_t)(h[0] > h[1] ? h[0] : h[1]) << 16;
  } else {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t b = r[k] & 0x7fffffffu;
      m = b > m ? b : m;
    }
  }
  m = lane_max<L>(m);
  if (m >= 0x7f800000u) {
    m = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const uint32_t b = finite_mag_bits(v[k]);
      m = b > m ? b : m;
      v[k] = no_inf(v[k]);
    }
    m = lane_max<L>(m);
  }
  e = ckpt8_exponent(m);
  return Codes<N>::pack(v, inv_scale_of(e));
}

}  // namespace chan
}  // namespace gdr
