// scan_fwd.hip -- channelwise gated linear recurrence, forward and step, gfx950.
//
// One thread per (batch row, channel) walks the tokens in order.
#include "chan_device.h"
#include "scan_gate.h"
#include "scan_kernels.h"

namespace gdr {
namespace scan {

using chan::ld;
using chan::st;

template <typename T>
__device__ inline void coefficients(const float* alpha, const void* decay_x, const void* gate_x, float A, int normalise,
                                    size_t i, float x, float& a, float& v) {
  v = x;
  if (alpha) {
    a = alpha[i];
    return;
  }
  float w;
  const float u = A * softplus(ld((const T*)decay_x + i), w);
  a = exp_fast(-u);
  if (gate_x) v *= sigmoid(ld((const T*)gate_x + i));
  if (normalise) v *= __builtin_amdgcn_sqrtf(one_minus_sq(u, a));
}

template <typename T>
__global__ __launch_bounds__(64) void scan_fwd_kernel(gdr_scan_args p) {
  const size_t n = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (n >= (size_t)p.B * p.C) return;
  const int b = (int)(n / p.C), c = (int)(n % p.C);
  const float A = p.alpha ? 0.f : p.decay_a[c];
  const size_t nb = blocks_of(p.T);
  float h = p.h0 ? p.h0[n] : 0.f;
  for (int t = 0; t < p.T; ++t) {
    const size_t i = ((size_t)b * p.T + t) * p.C + c;
    if (p.ckpt && t % GDR_SCAN_BLOCK == 0) p.ckpt[((size_t)b * nb + t / GDR_SCAN_BLOCK) * p.C + c] = h;
    float a, v;
    coefficients<T>(p.alpha, p.decay_x, p.gate_x, A, p.normalise, i, ld((const T*)p.x + i), a, v);
    h = fmaf(a, h, v);
    st((T*)p.y + i, h);
  }
  if (p.h_out) p.h_out[n] = h;
}

template <typename T>
__global__ __launch_bounds__(256) void scan_step_kernel(gdr_scan_step_args p) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (size_t)p.N * p.C) return;
  const float A = p.alpha ? 0.f : p.decay_a[i % p.C];
  float a, v;
  coefficients<T>(p.alpha, p.decay_x, p.gate_x, A, p.normalise, i, ld((const T*)p.x + i), a, v);
  const float h = fmaf(a, p.h[i], v);
  p.h_out[i] = h;
  st((T*)p.y + i, h);
}

size_t fwd_workspace(int, int, int) { return 0; }

hipError_t launch_scan_fwd(const gdr_scan_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(((size_t)a.B * a.C + 63) / 64));
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(scan_fwd_kernel<__bf16>, grid, dim3(64), 0, s, a);
  else hipLaunchKernelGGL(scan_fwd_kernel<float>, grid, dim3(64), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_scan_step(const gdr_scan_step_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(((size_t)a.N * a.C + 255) / 256));
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(scan_step_kernel<__bf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(scan_step_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace scan
}  // namespace gdr
