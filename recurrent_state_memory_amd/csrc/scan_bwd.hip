// scan_bwd.hip -- gradients of the channelwise gated linear recurrence, gfx950.
//
// One thread per (batch row, channel).  Blocks of 32 tokens are taken from the
// last to the first: the states inside a block are computed again from its
// start state, then G_t = grad_y_t + a_{t+1} G_{t+1} runs backwards through it.
#include "chan_device.h"
#include "scan_gate.h"
#include "scan_kernels.h"

namespace gdr {
namespace scan {

using chan::ld;
using chan::st;

struct Gates {
  float a, s, m, sp, sig;   // decay, input gate, 1 - a^2, softplus, sigmoid(decay_x)
};

template <typename T>
__device__ inline Gates gates(const gdr_scan_bwd_args& p, float A, size_t i) {
  Gates g{0.f, 1.f, 1.f, 0.f, 0.f};
  if (p.alpha) {
    g.a = p.alpha[i];
    return g;
  }
  float w;
  const float d = ld((const T*)p.decay_x + i);
  g.sp = softplus(d, w);
  const float r = __builtin_amdgcn_rcpf(1.f + w);
  g.sig = d > 0.f ? r : w * r;
  g.a = exp_fast(-A * g.sp);
  if (p.gate_x) g.s = sigmoid(ld((const T*)p.gate_x + i));
  if (p.normalise) g.m = one_minus_sq(A * g.sp, g.a);
  return g;
}

template <typename T>
__device__ inline float load_x(const gdr_scan_bwd_args& p, size_t row, int c) {
  const size_t i = row * p.C + c;
  if (!p.x_exp) return ld((const T*)p.x + i);
  return chan::code1_f32(((const uint8_t*)p.x)[i]) * chan::scale_of(p.x_exp[row * ((p.C + 127) / 128) + c / 128]);
}

template <typename T>
__global__ __launch_bounds__(64) void ckpt_kernel(gdr_scan_bwd_args p, float* ckpt) {
  const size_t n = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (n >= (size_t)p.B * p.C) return;
  const int b = (int)(n / p.C), c = (int)(n % p.C);
  const float A = p.alpha ? 0.f : p.decay_a[c];
  float h = p.h0 ? p.h0[n] : 0.f;
  for (int t = 0; t < p.T; ++t) {
    const size_t row = (size_t)b * p.T + t;
    if (t % GDR_SCAN_BLOCK == 0) ckpt[((size_t)b * blocks_of(p.T) + t / GDR_SCAN_BLOCK) * p.C + c] = h;
    const Gates g = gates<T>(p, A, row * p.C + c);
    h = fmaf(g.a, h, load_x<T>(p, row, c) * g.s * __builtin_amdgcn_sqrtf(g.m));
  }
}

template <typename T>
__global__ __launch_bounds__(64) void scan_bwd_kernel(gdr_scan_bwd_args p, const float* ckpt, float* ga) {
  const size_t n = (size_t)blockIdx.x * 64 + threadIdx.x;
  if (n >= (size_t)p.B * p.C) return;
  const int b = (int)(n / p.C), c = (int)(n % p.C);
  const float A = p.alpha ? 0.f : p.decay_a[c];
  float K = p.grad_h ? p.grad_h[n] : 0.f, sum = 0.f;
  for (int j = (int)blocks_of(p.T) - 1; j >= 0; --j) {
    const int t0 = j * GDR_SCAN_BLOCK, t1 = t0 + GDR_SCAN_BLOCK < p.T ? t0 + GDR_SCAN_BLOCK : p.T;
    float prev[GDR_SCAN_BLOCK];
    float h = ckpt[((size_t)b * blocks_of(p.T) + j) * p.C + c];
    for (int t = t0; t < t1; ++t) {
      const size_t row = (size_t)b * p.T + t;
      const Gates g = gates<T>(p, A, row * p.C + c);
      prev[t - t0] = h;
      h = fmaf(g.a, h, load_x<T>(p, row, c) * g.s * __builtin_amdgcn_sqrtf(g.m));
    }
    for (int t = t1 - 1; t >= t0; --t) {
      const size_t row = (size_t)b * p.T + t, i = row * p.C + c;
      const Gates g = gates<T>(p, A, i);
      const float G = K + ld((const T*)p.grad_y + i), bb = g.s * __builtin_amdgcn_sqrtf(g.m);
      st((T*)p.grad_x + i, bb * G);
      if (p.alpha) {
        p.grad_alpha[i] = G * prev[t - t0];
      } else {
        const float v = bb * load_x<T>(p, row, c);
        if (p.gate_x) st((T*)p.grad_gate_x + i, G * v * (1.f - g.s));
        float in = -prev[t - t0];
        if (p.normalise && g.m > 0.f) in += v * g.a / g.m;
        const float du = G * g.a * in;
        st((T*)p.grad_decay_x + i, du * A * g.sig);
        sum += du * g.sp;
      }
      K = g.a * G;
    }
  }
  if (p.grad_h0) p.grad_h0[n] = K;
  if (ga) ga[n] = sum;
}

__global__ __launch_bounds__(64) void sum_rows_kernel(const float* part, float* out, int rows, int C) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= C) return;
  float s = 0.f;
  for (int r = 0; r < rows; ++r) s += part[(size_t)r * C + c];
  out[c] = s;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

size_t bwd_workspace(int B, int T, int C, bool gated, bool ckpt) {
  return (ckpt ? 0 : align256((size_t)B * blocks_of(T) * C * 4)) + (gated ? align256((size_t)B * C * 4) : 0);
}

template <typename T>
static void launch(const gdr_scan_bwd_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(((size_t)a.B * a.C + 63) / 64));
  char* ws = (char*)a.workspace;
  const float* ckpt = a.ckpt;
  if (!ckpt) {
    hipLaunchKernelGGL(ckpt_kernel<T>, grid, dim3(64), 0, s, a, (float*)ws);
    ckpt = (const float*)ws;
    ws += align256((size_t)a.B * blocks_of(a.T) * a.C * 4);
  }
  float* ga = a.alpha ? nullptr : (float*)ws;
  hipLaunchKernelGGL(scan_bwd_kernel<T>, grid, dim3(64), 0, s, a, ckpt, ga);
  if (ga) hipLaunchKernelGGL(sum_rows_kernel, dim3((a.C + 63) / 64), dim3(64), 0, s, ga, a.grad_decay_a, a.B, a.C);
}

hipError_t launch_scan_bwd(const gdr_scan_bwd_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) launch<__bf16>(a, s);
  else launch<float>(a, s);
  return hipGetLastError();
}

}  // namespace scan
}  // namespace gdr
