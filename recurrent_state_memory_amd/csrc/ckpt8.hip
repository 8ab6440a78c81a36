// ckpt8.hip -- 8-bit activation checkpoints: pack and unpack, gfx950.
//
// One wave per group of up to 128 values, two values per lane.
#include "chan_device.h"
#include "norm_kernels.h"

namespace gdr {
namespace ckpt8 {

using chan::ld;
using chan::st;

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(gdr_ckpt8_pack_args p) {
  const int G = (p.D + 127) / 128, l = threadIdx.x & 63;
  const size_t n = (size_t)p.R * G;
  for (size_t g = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6); g < n; g += (size_t)gridDim.x * 4) {
    const size_t row = g / G;
    const int c0 = (int)(g % G) * 128;
    float v[2];
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + l + 64 * k;
      v[k] = c < p.D ? ld((const T*)p.x + row * p.D + c) : 0.f;
      const uint32_t b = chan::finite_mag_bits(v[k]);
      m = b > m ? b : m;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
      const uint32_t o = __shfl_xor(m, off);
      m = o > m ? o : m;
    }
    const int e = chan::ckpt8_exponent(m);
    const float inv = chan::inv_scale_of(e);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = c0 + l + 64 * k;
      if (c < p.D) p.code[row * p.D + c] = chan::pack1_e4m3(v[k] * inv);
    }
    if (l == 0) p.exp[g] = (uint8_t)e;
  }
}

template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(gdr_ckpt8_unpack_args p) {
  const int G = (p.D + 127) / 128, l = threadIdx.x & 63;
  const size_t n = (size_t)p.R * G;
  for (size_t g = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6); g < n; g += (size_t)gridDim.x * 4) {
    const size_t row = g / G;
    const float sc = chan::scale_of(p.exp[g]);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int c = (int)(g % G) * 128 + l + 64 * k;
      if (c < p.D) st((T*)p.x + row * p.D + c, chan::code1_f32(p.code[row * p.D + c]) * sc);
    }
  }
}

static unsigned grid_of(int64_t R, int D) {
  const size_t n = ((size_t)R * ((D + 127) / 128) + 3) / 4;
  return (unsigned)(n < 65536 ? n : 65536);
}

hipError_t launch_pack(const gdr_ckpt8_pack_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(pack_kernel<__bf16>, dim3(grid_of(a.R, a.D)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(pack_kernel<float>, dim3(grid_of(a.R, a.D)), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_unpack(const gdr_ckpt8_unpack_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(unpack_kernel<__bf16>, dim3(grid_of(a.R, a.D)), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(unpack_kernel<float>, dim3(grid_of(a.R, a.D)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ckpt8
}  // namespace gdr
