// conv.hip -- short causal convolution, its backward and its single-token step, gfx950.
//
// A thread holds one 16-byte run of channels (four channels in the backward) and walks a
// stretch of tokens with the last K rows in registers, so x is read once (the K - 1 rows
// ahead of a stretch come from the caches).  LX threads of a workgroup share a row, the
// other 256 / LX take further stretches.  On 8 x 4096 x 2048 bf16 with 4 taps and silu the
// forward takes 52 us, the rate of a large copy (5.2 TB/s; fp32 104 us with the launch); the
// backward 91 us (4.4 TB/s; fp32 182): its arithmetic, some 30 instructions an element, takes
// about 60 of them.  Backward with eight channels a thread (two waves a SIMD):
// 99 us; rows asked for one step ahead, or runs that are known to be whole, cost the fourth
// wave's registers: 111 and 100 us.
#include <type_traits>

#include "chan_device.h"
#include "col_join.h"
#include "conv_kernels.h"

namespace gdr {
namespace conv {

using chan::raw4;
using chan::Run;

constexpr float kLog2e = 1.44269504f;
constexpr int kThreads = 256;

// Four channels a thread, 8 bytes of bf16: half the registers of a whole run.
template <typename T>
struct Four : Run<T> {};
template <>
struct Four<__bf16> {
  static constexpr int N = 4;
  typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
  typedef chan::raw2 at2 __attribute__((aligned(2), may_alias));
  static __device__ inline raw4 load(const __bf16* p, int n) {
    if (n >= N) {
      const chan::raw2 r = *(const at2*)p;
      return raw4{r[0], r[1], 0u, 0u};
    }
    raw4 r = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < N - 1; ++k)
      if (k < n) r[k >> 1] |= (uint32_t)__builtin_bit_cast(uint16_t, p[k]) << (16 * (k & 1));
    return r;
  }
  static __device__ inline float get(const raw4& r, int k) { return Run<__bf16>::get(r, k); }
  static __device__ inline void store(__bf16* p, int n, const float (&v)[N]) {
    if (n >= N) {
      bf16x4 h;
#pragma unroll
      for (int k = 0; k < N; ++k) h[k] = (__bf16)v[k];
      *(at2*)p = __builtin_bit_cast(chan::raw2, h);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < n) p[k] = (__bf16)v[k];
    }
  }
};

__device__ inline float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e)); }

// How a [B,T,C] activation is laid over workgroups: LX = 2^lx threads along a row's runs,
// 256 / LX stretches of `len` tokens, and cols x rows workgroups a batch row.
struct Plan {
  int lx, len;
  unsigned cols, rows;
  unsigned blocks(int B) const { return (unsigned)B * cols * rows; }
};
static Plan plan_of(int B, int T, int C, int n, int longest) {
  const int runs = (C + n - 1) / n;
  Plan q;
  q.lx = 0;
  while (q.lx < 6 && (1 << q.lx) < runs) ++q.lx;
  const int LX = 1 << q.lx, LY = kThreads / LX;
  q.cols = (unsigned)((runs + LX - 1) / LX);
  // 128 Ki threads are two waves a SIMD; shorter stretches than 8 tokens read mostly rows
  // of their neighbours
  const long long threads = (long long)B * q.cols * LX;
  q.len = 8;
  while (q.len < longest && threads * ((T + q.len - 1) / q.len) > 131072) q.len *= 2;
  q.rows = (unsigned)(((T + q.len - 1) / q.len + LY - 1) / LY);
  return q;
}

struct Spot {
  int b, t0, c0, n;   // batch row, first token, first channel, channels that exist (<= 0: none)
};
template <int N>
__device__ inline Spot spot_of(const Plan& q, int T, int C) {
  const unsigned col = blockIdx.x % q.cols, rest = blockIdx.x / q.cols;
  const int tx = threadIdx.x & ((1 << q.lx) - 1), ty = threadIdx.x >> q.lx;
  Spot s;
  s.b = (int)(rest / q.rows);
  const long long t = ((long long)(rest % q.rows) * (kThreads >> q.lx) + ty) * q.len;
  s.t0 = t < T ? (int)t : T;   // T: no stretch
  s.c0 = (int)((col << q.lx) + tx) * N;
  s.n = C - s.c0;
  return s;
}

template <typename R, int N>
__device__ inline void unpack(const raw4& r, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = R::get(r, k);
}

__device__ inline int row_len(const int32_t* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : n < T ? n : T;
}

// weight[c][j] of a run's channels, N K numbers in a row, and their bias; 0 behind the
// last channel.
template <int N, int K>
__device__ inline void load_params(const float* weight, const float* bias, const Spot& s, float (&w)[K][N], float (&b)[N]) {
  const float* at = weight + (size_t)s.c0 * K;
#pragma unroll
  for (int i = 0; i < N * K; i += 4) {
    const raw4 r = Run<float>::load(at + i, s.n * K - i);
#pragma unroll
    for (int k = 0; k < 4; ++k) w[(i + k) % K][(i + k) / K] = Run<float>::get(r, k);
  }
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const raw4 r = bias ? Run<float>::load(bias + s.c0 + i, s.n - i) : raw4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int k = 0; k < 4; ++k) b[i + k] = Run<float>::get(r, k);
  }
}

// The K - 1 rows before token t0, oldest first: of the sequence (0 behind its end), or of
// the state.
template <typename R, int K, typename T>
__device__ inline void load_before(const T* x, const T* state, const Spot& s, int len, int C, raw4 (&r)[K - 1]) {
#pragma unroll
  for (int i = 0; i < K - 1; ++i) {
    const int t = s.t0 - (K - 1) + i;
    r[i] = raw4{0u, 0u, 0u, 0u};
    if (t >= 0) {
      if (t < len) r[i] = R::load(x + (ptrdiff_t)t * C, s.n);
    } else if (state) r[i] = R::load(state + (ptrdiff_t)(t + K - 1) * C, s.n);
  }
}

template <typename T, int K, int U>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(gdr_conv_args p, Plan q) {
  typedef Run<T> R;
  constexpr int N = R::N;
  const int C = p.C;
  const Spot s = spot_of<N>(q, p.T, C);
  if (s.n <= 0 || s.t0 >= p.T) return;
  const int len = row_len(p.lens, s.b, p.T), t1 = min(s.t0 + q.len, p.T);
  const T* x = (const T*)p.x + (size_t)s.b * p.T * C + s.c0;
  T* y = (T*)p.y + (size_t)s.b * p.T * C + s.c0;
  float f[K - 1 + U][N];   // the rows under the taps
  {
    const T* state = p.state ? (const T*)p.state + (size_t)s.b * (K - 1) * C + s.c0 : nullptr;
    raw4 r[K - 1];
    load_before<R, K>(x, state, s, len, C, r);
    if (s.t0 == 0 && p.state_out) {
      // the row's last K - 1 inputs; this thread alone reads its part of the state, so it
      // may be overwritten from here on
      T* so = (T*)p.state_out + (size_t)s.b * (K - 1) * C + s.c0;
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        const int i = len + j;   // among the state's rows and the tokens behind them
        raw4 v = r[K - 2];
        if (i >= K - 1) {
          v = R::load(x + (ptrdiff_t)(i - (K - 1)) * C, s.n);
        } else {
#pragma unroll
          for (int k = 0; k < K - 2; ++k) v = i == k ? r[k] : v;
        }
        float o[N];
        unpack<R>(v, o);
        R::store(so + (ptrdiff_t)j * C, s.n, o);
      }
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i) unpack<R>(r[i], f[i]);
  }
  float w[K][N], bias[N];
  load_params<N, K>(p.weight, p.bias, s, w, bias);
  for (int t = s.t0; t < t1; t += U) {
    raw4 r[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      r[i] = t + i < min(t1, len) ? R::load(x + (ptrdiff_t)(t + i) * C, s.n) : raw4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < U; ++i) {
      unpack<R>(r[i], f[K - 1 + i]);
      if (t + i >= t1) break;
      float o[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        float a = bias[k];
#pragma unroll
        for (int j = 0; j < K; ++j) a = fmaf(w[j][k], f[i + j][k], a);
        if (p.silu) a *= sigmoid(a);
        o[k] = t + i < len ? a : 0.f;
      }
      R::store(y + (ptrdiff_t)(t + i) * C, s.n, o);
    }
#pragma unroll
    for (int i = 0; i < K - 1; ++i)
#pragma unroll
      for (int k = 0; k < N; ++k) f[i][k] = f[U + i][k];
  }
}

// Backward: d_t of the stretch's tokens and of the K - 1 behind it, whose taps reach into
// it; grad_x of token t - K + 1 is complete with d_t.  Each workgroup leaves a partial row
// [K + 1][C] of the weight's and the bias' sums for the join.
template <typename T, int K, int U>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(gdr_conv_bwd_args p, Plan q) {
  typedef Four<T> R;
  constexpr int N = R::N;
  const int C = p.C;
  const Spot s = spot_of<N>(q, p.T, C);
  float dw[K + 1][N];   // the last one is the bias'
#pragma unroll
  for (int j = 0; j <= K; ++j)
#pragma unroll
    for (int k = 0; k < N; ++k) dw[j][k] = 0.f;
  if (s.n > 0 && s.t0 < p.T) {
    const int len = row_len(p.lens, s.b, p.T), t1 = min(s.t0 + q.len, p.T);
    const size_t row0 = (size_t)s.b * p.T * C + s.c0, edge0 = (size_t)s.b * (K - 1) * C + s.c0;
    const T* x = (const T*)p.x + row0;
    const T* gy = (const T*)p.grad_y + row0;
    T* gx = (T*)p.grad_x + row0;
    T* gs = p.grad_state ? (T*)p.grad_state + edge0 : nullptr;
    const T* gso = p.grad_state_out ? (const T*)p.grad_state_out + edge0 : nullptr;
    float w[K][N], bias[N];
    load_params<N, K>(p.weight, p.bias, s, w, bias);
    float f[K - 1 + U][N], d[K - 1 + U][N];
    {
      raw4 r[K - 1];
      load_before<R, K>(x, p.state ? (const T*)p.state + edge0 : nullptr, s, len, C, r);
#pragma unroll
      for (int i = 0; i < K - 1; ++i) {
        unpack<R>(r[i], f[i]);
#pragma unroll
        for (int k = 0; k < N; ++k) d[i][k] = 0.f;
      }
    }
    for (int t = s.t0; t < t1 + K - 1; t += U) {
      raw4 rx[U], rg[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const bool on = t + i < min(t1 + K - 1, len);
        rx[i] = on ? R::load(x + (ptrdiff_t)(t + i) * C, s.n) : raw4{0u, 0u, 0u, 0u};
        rg[i] = on ? R::load(gy + (ptrdiff_t)(t + i) * C, s.n) : raw4{0u, 0u, 0u, 0u};
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        unpack<R>(rx[i], f[K - 1 + i]);
        const bool on = t + i < len;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          float g = R::get(rg[i], k);
          if (p.silu) {
            float u = bias[k];
#pragma unroll
            for (int j = 0; j < K; ++j) u = fmaf(w[j][k], f[i + j][k], u);
            const float sg = sigmoid(u);
            g *= sg * fmaf(u, 1.f - sg, 1.f);
          }
          d[K - 1 + i][k] = on ? g : 0.f;   // behind the row's end the taps still see its last tokens
        }
        if (on && t + i < t1) {   // the next stretch sums its own
#pragma unroll
          for (int k = 0; k < N; ++k) {
            const float g = d[K - 1 + i][k];
            dw[K][k] += g;
#pragma unroll
            for (int j = 0; j < K; ++j) dw[j][k] = fmaf(g, f[i + j][k], dw[j][k]);
          }
        }
        const int o = t + i - (K - 1);   // the token whose last tap this was
        const bool here = o >= s.t0 ? o < t1 : s.t0 == 0 && o < 0 && gs != nullptr;
        if (here) {
          float v[N];
#pragma unroll
          for (int k = 0; k < N; ++k) {
            float a = 0.f;
#pragma unroll
            for (int j = 0; j < K; ++j) a = fmaf(w[j][k], d[i + K - 1 - j][k], a);
            v[k] = a;
          }
          const int e = o - len + K - 1;   // its place in state_out
          if (gso && e >= 0 && e < K - 1) {
            const raw4 r = R::load(gso + (ptrdiff_t)e * C, s.n);
#pragma unroll
            for (int k = 0; k < N; ++k) v[k] += R::get(r, k);
          }
          if (o >= 0) R::store(gx + (ptrdiff_t)o * C, s.n, v);
          else R::store(gs + (ptrdiff_t)(o + K - 1) * C, s.n, v);
        }
      }
#pragma unroll
      for (int i = 0; i < K - 1; ++i)
#pragma unroll
        for (int k = 0; k < N; ++k) {
          f[i][k] = f[U + i][k];
          d[i][k] = d[U + i][k];
        }
    }
  }
  // over the workgroup's stretches, one tap at a time: LX N sums of LY values, each shared
  // by kThreads / (LX N) threads where there are fewer sums than threads
  __shared__ float part[kThreads * N], few[kThreads];
  const int LX = 1 << q.lx, LY = kThreads >> q.lx, sums = LX * N;
  const int share = sums < kThreads ? kThreads / sums : 1;
  float* out = (float*)p.workspace + (size_t)(blockIdx.x / q.cols) * (K + 1) * C;
#pragma unroll
  for (int j = 0; j <= K; ++j) {
#pragma unroll
    for (int k = 0; k < N; ++k) part[k * kThreads + threadIdx.x] = dw[j][k];
    __syncthreads();
    for (int i = threadIdx.x; i < sums * share; i += kThreads) {
      const int m = i / sums, k = (i - m * sums) / LX, l = i & (LX - 1), c = (int)((blockIdx.x % q.cols) * LX + l) * N + k;
      float a = 0.f;
      for (int y = m; y < LY; y += share) a += part[k * kThreads + y * LX + l];
      if (share > 1) few[i] = a;
      else if (c < C) out[(size_t)j * C + c] = a;
    }
    __syncthreads();
    if (share > 1) {
      const int i = threadIdx.x, c = (int)((blockIdx.x % q.cols) * LX + (i & (LX - 1))) * N + i / LX;
      if (i < sums && c < C) {
        float a = 0.f;
        for (int m = 0; m < share; ++m) a += few[m * sums + i];
        out[(size_t)j * C + c] = a;
      }
    }
  }
}

// Where a column of the partial rows goes.
struct ParamGrads {
  int C, K;
  float *weight, *bias;
  __device__ void operator()(size_t i, float v) const {
    const int j = (int)(i / C), c = (int)(i - (size_t)j * C);
    if (j < K) weight[(size_t)c * K + j] = v;
    else if (bias) bias[c] = v;
  }
};

template <typename T, int K>
__global__ __launch_bounds__(kThreads) void conv_step_kernel(gdr_conv_step_args p, int runs) {
  typedef Run<T> R;
  constexpr int N = R::N;
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x, row = i / runs;
  if (row >= (size_t)p.N) return;
  Spot s;
  s.c0 = (int)(i - row * runs) * N;
  s.n = p.C - s.c0;
  const size_t C = p.C, at = row * (K - 1) * C + s.c0;
  const T* in = (const T*)p.state + at;
  float f[K][N];
#pragma unroll
  for (int j = 0; j < K - 1; ++j) unpack<R>(R::load(in + j * C, s.n), f[j]);
  unpack<R>(R::load((const T*)p.x + row * C + s.c0, s.n), f[K - 1]);
  T* out = (T*)p.state_out + at;
#pragma unroll
  for (int j = 0; j < K - 1; ++j) R::store(out + j * C, s.n, f[j + 1]);
  float w[K][N], o[N];
  load_params<N, K>(p.weight, p.bias, s, w, o);
#pragma unroll
  for (int k = 0; k < N; ++k) {
#pragma unroll
    for (int j = 0; j < K; ++j) o[k] = fmaf(w[j][k], f[j][k], o[k]);
    if (p.silu) o[k] *= sigmoid(o[k]);
  }
  R::store((T*)p.y + row * C + s.c0, s.n, o);
}

constexpr int kLongest = 64;   // tokens of a stretch

size_t bwd_workspace(int B, int T, int C, int K) {
  const Plan q = plan_of(B, T, C, 4, kLongest);
  return ((size_t)B * q.rows * (K + 1) * C * 4 + 255) / 256 * 256;
}

template <typename F>
static void with_taps(int K, F f) {
  switch (K) {
    case 2: f(std::integral_constant<int, 2>()); break;
    case 3: f(std::integral_constant<int, 3>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 5: f(std::integral_constant<int, 5>()); break;
    case 6: f(std::integral_constant<int, 6>()); break;
    case 7: f(std::integral_constant<int, 7>()); break;
    default: f(std::integral_constant<int, 8>()); break;
  }
}

hipError_t launch_conv_fwd(const gdr_conv_args& a, hipStream_t s) {
  const bool bf = a.io_dtype == GDR_BF16;
  const Plan q = plan_of(a.B, a.T, a.C, bf ? 8 : 4, kLongest);
  with_taps(a.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (bf) hipLaunchKernelGGL((conv_fwd_kernel<__bf16, K, 4>), dim3(q.blocks(a.B)), dim3(kThreads), 0, s, a, q);
    else hipLaunchKernelGGL((conv_fwd_kernel<float, K, 4>), dim3(q.blocks(a.B)), dim3(kThreads), 0, s, a, q);
  });
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const gdr_conv_bwd_args& a, hipStream_t s) {
  const bool bf = a.io_dtype == GDR_BF16;
  const Plan q = plan_of(a.B, a.T, a.C, 4, kLongest);
  with_taps(a.K, [&](auto k) {
    constexpr int K = decltype(k)::value, U = K > 4 ? 1 : 4;
    if (bf) hipLaunchKernelGGL((conv_bwd_kernel<__bf16, K, U>), dim3(q.blocks(a.B)), dim3(kThreads), 0, s, a, q);
    else hipLaunchKernelGGL((conv_bwd_kernel<float, K, U>), dim3(q.blocks(a.B)), dim3(kThreads), 0, s, a, q);
  });
  launch_col_join((const float*)a.workspace, (size_t)a.B * q.rows, (size_t)(a.K + 1) * a.C,
                  ParamGrads{a.C, a.K, a.grad_weight, a.grad_bias}, s);
  return hipGetLastError();
}

hipError_t launch_conv_step(const gdr_conv_step_args& a, hipStream_t s) {
  const bool bf = a.io_dtype == GDR_BF16;
  const int n = bf ? 8 : 4, runs = (a.C + n - 1) / n;
  const dim3 blocks((unsigned)(((size_t)a.N * runs + kThreads - 1) / kThreads));
  with_taps(a.K, [&](auto k) {
    constexpr int K = decltype(k)::value;
    if (bf) hipLaunchKernelGGL((conv_step_kernel<__bf16, K>), blocks, dim3(kThreads), 0, s, a, runs);
    else hipLaunchKernelGGL((conv_step_kernel<float, K>), blocks, dim3(kThreads), 0, s, a, runs);
  });
  return hipGetLastError();
}

}  // namespace conv
}  // namespace gdr
