// gnorm.hip -- gated group norm forward and backward, gfx950.
//
// A group of a row is held in registers by L threads of NV 16-byte runs each (thread l has
// runs l, l + L, ...; the forward asks for the next row ahead), so everything is read once:
// the mean, then the squares about it, then the outputs.  L is a part of a wave for short groups (several groups side by side in
// a wave, no barrier) or up to 1024 threads.  Bound by HBM: 32768 x 2048 bf16 in 16 groups,
// gated, forward 83 us (4.9 TB/s), backward 129 us (5.2 TB/s).  Of groups of more than 8192
// values the backward spills up to 36 registers: 4096 rows of one group of 16384, gated, 298 us
// in bf16 (2.3 TB/s; 8192 rows of 8192 149) and 383 in fp32 (3.5 TB/s), the forward 91 and 155.
#include "chan_device.h"
#include "col_join.h"
#include "gnorm_kernels.h"

namespace gdr {
namespace gnorm {

using chan::lane_sum;
using chan::raw4;
using chan::Run;

constexpr float kLog2e = 1.44269504f;
__device__ inline float sigmoid(float v) { return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -kLog2e)); }

// Groups of more than a wave have a workgroup to themselves, so every barrier of a sum is
// reached by all of it.
constexpr int fwd_threads(int L) { return L > 64 ? L : 256; }
constexpr int bwd_threads(int L) { return L > 64 ? L : 1024; }

// Sums over the group's L threads; more than a wave: through LDS, in one of two places by
// turns, so that one barrier a sum is enough.
template <int TH, int NSUM>
struct Parts {
  float v[2][NSUM][TH / 64];
};
template <int TH, int L, int NSUM>
__device__ inline void group_sum(float (&v)[NSUM], Parts<TH, NSUM>& lds, int& turn) {
#pragma unroll
  for (int i = 0; i < NSUM; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
  if constexpr (L > 64) {
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NSUM; ++i) lds.v[turn][i][threadIdx.x >> 6] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NSUM; ++i) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < L / 64; ++k) s += lds.v[turn][i][k];
      v[i] = s;
    }
    turn ^= 1;
  }
}

// N fp32 numbers of a parameter, `none` where it is absent.
template <int N>
__device__ inline void load_param(const float* p, int c0, int n, float none, float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const raw4 r = p ? Run<float>::load(p + c0 + k, n - k) : raw4{};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[k + i] = p ? Run<float>::get(r, i) : none;
  }
}

// A thread keeps one group's columns for all its rows, so its weights (and in the backward
// the columns' sums) stay in registers: a workgroup's TH / L places go to `wide` groups of
// blockIdx.y, `deep` rows of each at a time.
struct Lay {
  int wide, deep;
  unsigned rows, groups;   // workgroups along the rows and along the groups
};

template <typename T, int L, int NV>
__global__ __launch_bounds__(fwd_threads(L)) void gnorm_fwd_kernel(gdr_gnorm_args p, Lay q) {
  constexpr int N = Run<T>::N, TH = fwd_threads(L);
  __shared__ Parts<TH, 1> sums;
  int turn = 0;
  const int l = threadIdx.x % L, D = p.C / p.G;
  const int place = threadIdx.x / L, m = place / q.wide, g = (int)blockIdx.y * q.wide + place - m * q.wide;
  if (m >= q.deep || g >= p.G) return;   // never a part of a group, and no barrier is for more than one
  float w[NV][N], b[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * L + l) * N;
    load_param<N>(p.weight, g * D + c0, D - c0, 1.f, w[j]);
    load_param<N>(p.bias, g * D + c0, D - c0, 0.f, b[j]);
  }
  const float inv = 1.f / D;
  const int64_t first = (int64_t)blockIdx.x * q.deep + m, step = (int64_t)gridDim.x * q.deep;
  raw4 nx[NV], nz[NV];   // the next row
  auto load = [&](int64_t row) {
    const size_t at = (size_t)row * p.C + (size_t)g * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * L + l) * N;
      nx[j] = Run<T>::load((const T*)p.x + at + c0, D - c0);
      nz[j] = p.z ? Run<T>::load((const T*)p.z + at + c0, D - c0) : raw4{};
    }
  };
  if (first < p.R) load(first);
  for (int64_t row = first; row < p.R; row += step) {
    raw4 r[NV], rz[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] = nx[j], rz[j] = nz[j];
    if (row + step < p.R) load(row + step);
    float mean = 0.f, s[1];
    if (p.center) {
      s[0] = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int k = 0; k < N; ++k) s[0] += Run<T>::get(r[j], k);   // 0 behind the group's end
      group_sum<TH, L>(s, sums, turn);
      mean = s[0] * inv;
    }
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float c = (j * L + l) * N + k < D ? Run<T>::get(r[j], k) - mean : 0.f;
        s[0] = fmaf(c, c, s[0]);
      }
    group_sum<TH, L>(s, sums, turn);
    const float rstd = 1.f / sqrtf(fmaf(s[0], inv, p.eps));
    if (l == 0) {
      const size_t st = (size_t)row * p.G + g;
      if (p.mean) p.mean[st] = mean;
      if (p.rstd) p.rstd[st] = rstd;
    }
    T* y = (T*)p.y + (size_t)row * p.C + (size_t)g * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * L + l) * N;
      float o[N];
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float u = fmaf((Run<T>::get(r[j], k) - mean) * rstd, w[j][k], b[j][k]);
        const float v = p.z ? Run<T>::get(rz[j], k) : u;
        const float a = p.silu ? v * sigmoid(v) : v;
        o[k] = p.z ? u * a : a;
      }
      Run<T>::store(y + c0, D - c0, o);
    }
  }
}

// Backward.  A workgroup leaves one partial row [2][C] of the columns' sums for the join.
template <typename T, int L, int NV>
__global__ __launch_bounds__(bwd_threads(L)) void gnorm_bwd_kernel(gdr_gnorm_bwd_args p, Lay q) {
  constexpr int N = Run<T>::N, TH = bwd_threads(L);
  __shared__ Parts<TH, 2> sums;
  int turn = 0;
  const int l = threadIdx.x % L, D = p.C / p.G;
  const int place = threadIdx.x / L, m = place / q.wide, g = (int)blockIdx.y * q.wide + place - m * q.wide;
  const bool here = m < q.deep && g < p.G;
  const int base = here ? g * D : 0;
  float w[NV][N], b[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * L + l) * N;
    load_param<N>(p.weight, base + c0, D - c0, 1.f, w[j]);
    load_param<N>(p.bias, base + c0, D - c0, 0.f, b[j]);
#pragma unroll
    for (int k = 0; k < N; ++k) dw[j][k] = db[j][k] = 0.f;
  }
  const float inv = 1.f / D;
  if (here) {
    for (int64_t row = (int64_t)blockIdx.x * q.deep + m; row < p.R; row += (int64_t)gridDim.x * q.deep) {
      const size_t at = (size_t)row * p.C + base, st = (size_t)row * p.G + g;
      raw4 rx[NV], ry[NV], rz[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N, n = D - c0;
        rx[j] = Run<T>::load((const T*)p.x + at + c0, n);
        ry[j] = Run<T>::load((const T*)p.grad_y + at + c0, n);
        rz[j] = p.z ? Run<T>::load((const T*)p.z + at + c0, n) : raw4{};
      }
      const float mean = p.mean ? p.mean[st] : 0.f, rstd = p.rstd[st];
      float s[2] = {0.f, 0.f};
      float xh[NV][N], gw[NV][N];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N, n = D - c0;
        float dz[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float h = k < n ? (Run<T>::get(rx[j], k) - mean) * rstd : 0.f;
          const float u = fmaf(h, w[j][k], b[j][k]), dy = Run<T>::get(ry[j], k);
          const float v = p.z ? Run<T>::get(rz[j], k) : u;
          float act = v, slope = 1.f;
          if (p.silu) {
            const float sg = sigmoid(v);
            act = v * sg;
            slope = sg * fmaf(v, 1.f - sg, 1.f);
          }
          dz[k] = dy * u * slope;
          const float du = p.z ? dy * act : dy * slope;
          dw[j][k] = fmaf(du, h, dw[j][k]);
          db[j][k] += du;
          xh[j][k] = h;
          gw[j][k] = du * w[j][k];
          s[0] += gw[j][k];
          s[1] = fmaf(gw[j][k], h, s[1]);
        }
        if (p.z) Run<T>::store((T*)p.grad_z + at + c0, n, dz);
      }
      group_sum<TH, L>(s, sums, turn);
      const float s0 = p.mean ? s[0] * inv : 0.f, s1 = s[1] * inv;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N;
        float o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = rstd * (gw[j][k] - s0 - xh[j][k] * s1);
        Run<T>::store((T*)p.grad_x + at + c0, D - c0, o);
      }
    }
  }
  if (!p.grad_weight && !p.grad_bias) return;
  if constexpr (L <= 64) {   // the rows worked on side by side, halves added to halves
    __shared__ float part[TH * N];
    for (int v = 0; v < 2; ++v) {
      float(&a)[N] = v == 0 ? dw[0] : db[0];
      for (int left = q.deep; left > 1;) {
        const int half = (left + 1) / 2;
        __syncthreads();
        if (here && m >= half && m < left) {
#pragma unroll
          for (int k = 0; k < N; ++k) part[k * TH + threadIdx.x] = a[k];
        }
        __syncthreads();
        if (here && m + half < left) {
#pragma unroll
          for (int k = 0; k < N; ++k) a[k] += part[k * TH + threadIdx.x + half * q.wide * L];
        }
        left = half;
      }
    }
  }
  if (here && m == 0) {
    float* out = (float*)p.workspace + (size_t)blockIdx.x * 2 * p.C + base;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const int c = (j * L + l) * N + k;
        if (c < D) {
          out[c] = dw[j][k];
          out[p.C + c] = db[j][k];
        }
      }
  }
}

struct ParamGrads {
  size_t C;
  float *weight, *bias;
  __device__ void operator()(size_t i, float v) const {
    if (i < C) {
      if (weight) weight[i] = v;
    } else if (bias) {
      bias[i - C] = v;
    }
  }
};

// Threads and runs of a group of D values: one run a thread up to 1024 threads (what is
// under way at once hides the latency), then up to four.
struct Shape {
  int L, NV;
};
static Shape shape_of(int D, int n) {
  const int runs = (D + n - 1) / n;
  Shape s{2, 1};
  while (s.L < 1024 && s.L < runs) s.L *= 2;
  while (s.L * s.NV < runs) s.NV *= 2;
  return s;
}

// Workgroups of TH threads for R rows of G groups, `threads` in all at the most.
static Lay lay_of(int64_t R, int G, const Shape& s, int TH, int64_t threads) {
  const int places = TH / s.L;
  Lay q;
  q.wide = places < G ? places : G;
  q.deep = places / q.wide;
  q.groups = (unsigned)((G + q.wide - 1) / q.wide);
  const int64_t want = (R + q.deep - 1) / q.deep, most = (threads / TH + q.groups - 1) / q.groups;
  q.rows = (unsigned)(want < most ? want : most);
  return q;
}

// 2 x 1024 threads a CU in the backward: more rows of partial sums than that cost the join
// more than they hide.
static Lay bwd_lay(int64_t R, int G, const Shape& s) { return lay_of(R, G, s, bwd_threads(s.L), 524288); }

size_t bwd_workspace(int64_t R, int C, int G, int io_dtype) {
  const Lay q = bwd_lay(R, G, shape_of(C / G, io_dtype == GDR_BF16 ? 8 : 4));
  return ((size_t)q.rows * 2 * C * 4 + 255) / 256 * 256;
}

template <typename T, int L, int NV>
static void fwd(const gdr_gnorm_args& a, hipStream_t s) {
  constexpr int TH = fwd_threads(L);
  const Lay q = lay_of(a.R, a.G, Shape{L, NV}, TH, 1 << 20);
  hipLaunchKernelGGL((gnorm_fwd_kernel<T, L, NV>), dim3(q.rows, q.groups), dim3(TH), 0, s, a, q);
}
template <typename T, int L, int NV>
static void bwd(const gdr_gnorm_bwd_args& a, hipStream_t s) {
  const Lay q = bwd_lay(a.R, a.G, Shape{L, NV});
  hipLaunchKernelGGL((gnorm_bwd_kernel<T, L, NV>), dim3(q.rows, q.groups), dim3(bwd_threads(L)), 0, s, a, q);
  if (a.grad_weight || a.grad_bias)
    launch_col_join((const float*)a.workspace, q.rows, (size_t)2 * a.C, ParamGrads{(size_t)a.C, a.grad_weight, a.grad_bias}, s);
}

// The kernel of a group's shape; every shape that shape_of gives has one.
#define GNORM_SHAPES(CALL)                                                                  \
  do {                                                                                      \
    if (sh.NV == 1) {                                                                       \
      switch (sh.L) {                                                                       \
        case 2: CALL(2, 1); break;                                                          \
        case 4: CALL(4, 1); break;                                                          \
        case 8: CALL(8, 1); break;                                                          \
        case 16: CALL(16, 1); break;                                                        \
        case 32: CALL(32, 1); break;                                                        \
        case 64: CALL(64, 1); break;                                                        \
        case 128: CALL(128, 1); break;                                                      \
        case 256: CALL(256, 1); break;                                                      \
        case 512: CALL(512, 1); break;                                                      \
        default: CALL(1024, 1); break;                                                      \
      }                                                                                     \
    } else if (sh.NV == 2) {                                                                \
      CALL(1024, 2);                                                                        \
    } else if constexpr (Run<T>::N == 4) { /* bf16 groups need no more than two */          \
      CALL(1024, 4);                                                                        \
    }                                                                                       \
  } while (0)

template <typename T>
static void fwd_any(const gdr_gnorm_args& a, hipStream_t s) {
  const Shape sh = shape_of(a.C / a.G, Run<T>::N);
#define CALL(L, NV) fwd<T, L, NV>(a, s)
  GNORM_SHAPES(CALL);
#undef CALL
}
template <typename T>
static void bwd_any(const gdr_gnorm_bwd_args& a, hipStream_t s) {
  const Shape sh = shape_of(a.C / a.G, Run<T>::N);
#define CALL(L, NV) bwd<T, L, NV>(a, s)
  GNORM_SHAPES(CALL);
#undef CALL
}

hipError_t launch_gnorm_fwd(const gdr_gnorm_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) fwd_any<__bf16>(a, s);
  else fwd_any<float>(a, s);
  return hipGetLastError();
}

hipError_t launch_gnorm_bwd(const gdr_gnorm_bwd_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) bwd_any<__bf16>(a, s);
  else bwd_any<float>(a, s);
  return hipGetLastError();
}

}  // namespace gnorm
}  // namespace gdr
