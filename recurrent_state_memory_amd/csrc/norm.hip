// norm.hip -- layer norm forward and backward, gfx950.
//
// One workgroup per row; the columns' sums by one thread per column.
#include "chan_device.h"
#include "norm_kernels.h"

namespace gdr {
namespace norm {

using chan::ld;
using chan::st;

__device__ inline float block_sum(float v) {
  __shared__ float part[4];
  v = chan::wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  return part[0] + part[1] + part[2] + part[3];
}

template <typename T>
__global__ __launch_bounds__(256) void norm_fwd_kernel(gdr_norm_args p) {
  const size_t row = blockIdx.x;
  const T* x = (const T*)p.x + row * p.D;
  float s = 0.f;
  for (int i = threadIdx.x; i < p.D; i += 256) s += ld(x + i);
  const float mean = block_sum(s) / p.D;
  s = 0.f;
  for (int i = threadIdx.x; i < p.D; i += 256) {
    const float c = ld(x + i) - mean;
    s += c * c;
  }
  const float rstd = 1.f / sqrtf(block_sum(s) / p.D + p.eps);
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
  for (int i = threadIdx.x; i < p.D; i += 256)
    st((T*)p.y + row * p.D + i,
       (ld(x + i) - mean) * rstd * (p.weight ? p.weight[i] : 1.f) + (p.bias ? p.bias[i] : 0.f));
}

template <typename T>
__device__ inline float load_x(const gdr_norm_bwd_args& p, size_t row, int i) {
  if (!p.x_exp) return ld((const T*)p.x + row * p.D + i);
  return chan::code1_f32(((const uint8_t*)p.x)[row * p.D + i]) *
         chan::scale_of(p.x_exp[row * ((p.D + 127) / 128) + i / 128]);
}

template <typename T>
__global__ __launch_bounds__(256) void norm_bwd_kernel(gdr_norm_bwd_args p) {
  const size_t row = blockIdx.x;
  const float mean = p.mean[row], rstd = p.rstd[row];
  float s0 = 0.f, s1 = 0.f;
  for (int i = threadIdx.x; i < p.D; i += 256) {
    const float g = ld((const T*)p.grad_y + row * p.D + i) * (p.weight ? p.weight[i] : 1.f);
    s0 += g;
    s1 += g * (load_x<T>(p, row, i) - mean) * rstd;
  }
  s0 = block_sum(s0) / p.D;
  s1 = block_sum(s1) / p.D;
  for (int i = threadIdx.x; i < p.D; i += 256) {
    const float g = ld((const T*)p.grad_y + row * p.D + i) * (p.weight ? p.weight[i] : 1.f);
    st((T*)p.grad_x + row * p.D + i, rstd * (g - s0 - (load_x<T>(p, row, i) - mean) * rstd * s1));
  }
}

constexpr int kParts = 64;

template <typename T>
__global__ __launch_bounds__(64) void norm_cols_kernel(gdr_norm_bwd_args p) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= p.D) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t r = blockIdx.y; r < p.R; r += kParts) {
    const float dy = ld((const T*)p.grad_y + (size_t)r * p.D + c);
    sw += dy * (load_x<T>(p, (size_t)r, c) - p.mean[r]) * p.rstd[r];
    sb += dy;
  }
  float* part = (float*)p.workspace + (size_t)blockIdx.y * 2 * p.D;
  part[c] = sw;
  part[p.D + c] = sb;
}

__global__ __launch_bounds__(64) void norm_join_kernel(gdr_norm_bwd_args p) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= p.D) return;
  float sw = 0.f, sb = 0.f;
  for (int k = 0; k < kParts; ++k) {
    const float* part = (const float*)p.workspace + (size_t)k * 2 * p.D;
    sw += part[c];
    sb += part[p.D + c];
  }
  if (p.grad_weight) p.grad_weight[c] = sw;
  if (p.grad_bias) p.grad_bias[c] = sb;
}

size_t bwd_workspace(int64_t, int D) { return (size_t)kParts * 2 * D * sizeof(float); }

template <typename T>
static void launch_bwd(const gdr_norm_bwd_args& a, hipStream_t s) {
  hipLaunchKernelGGL(norm_bwd_kernel<T>, dim3((unsigned)a.R), dim3(256), 0, s, a);
  if (a.grad_weight || a.grad_bias) {
    hipLaunchKernelGGL(norm_cols_kernel<T>, dim3((a.D + 63) / 64, kParts), dim3(64), 0, s, a);
    hipLaunchKernelGGL(norm_join_kernel, dim3((a.D + 63) / 64), dim3(64), 0, s, a);
  }
}

hipError_t launch_norm_fwd(const gdr_norm_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(norm_fwd_kernel<__bf16>, dim3((unsigned)a.R), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(norm_fwd_kernel<float>, dim3((unsigned)a.R), dim3(256), 0, s, a);
  if (a.x_code) {
    gdr_ckpt8_pack_args c{a.R, a.D, a.io_dtype, a.x, a.x_code, a.x_exp};
    return ckpt8::launch_pack(c, s);
  }
  return hipGetLastError();
}

hipError_t launch_norm_bwd(const gdr_norm_bwd_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) launch_bwd<__bf16>(a, s);
  else launch_bwd<float>(a, s);
  return hipGetLastError();
}

}  // namespace norm
}  // namespace gdr
