// norm.hip -- layer norm forward and backward, gfx950.
//
// A row is held in registers by L threads of NV 16-byte runs each (thread l has
// runs l, l + L, ...), so it is read once: the mean, then the squares about it,
// then the outputs.  L is a part of a wave for short rows (64 / L rows side by side
// in a wave, no barrier), a wave up to 4 runs a lane, then 256 or 1024 threads.
// Both kernels are bound by HBM.
#include "chan_device.h"
#include "norm_kernels.h"

namespace gdr {
namespace norm {

using chan::Codes;
using chan::lane_max;
using chan::lane_sum;
using chan::raw4;
using chan::Run;

constexpr int threads_of(int L) { return L > 256 ? L : 256; }

// Sums of two values over the row's L threads; more than a wave: through LDS.
template <int L, int NSUM>
__device__ inline void row_sum(float (&v)[NSUM]) {
  constexpr int W = L / 64;
#pragma unroll
  for (int i = 0; i < NSUM; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
  if constexpr (W > 1) {
    __shared__ float part[NSUM][W];
    const int w = threadIdx.x >> 6;
    __syncthreads();   // the last sums have been read
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NSUM; ++i) part[i][w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NSUM; ++i) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) s += part[i][k];
      v[i] = s;
    }
  }
}

template <typename T, int L, int NV, bool CK>
__global__ __launch_bounds__(threads_of(L)) void norm_fwd_kernel(gdr_norm_args p) {
  constexpr int N = Run<T>::N;
  constexpr int kPer = threads_of(L) / L;           // rows of a workgroup
  constexpr int kGroupLanes = 128 / N < L ? 128 / N : L;
  const int l = threadIdx.x % L;
  const int D = p.D;
  const int64_t step = (int64_t)gridDim.x * kPer;
  for (int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / L; row < p.R; row += step) {
    const T* x = (const T*)p.x + (size_t)row * D;
    raw4 r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] = Run<T>::load(x + (j * L + l) * N, D - (j * L + l) * N);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) s[0] += Run<T>::get(r[j], k);   // 0 behind the row's end
    row_sum<L, 1>(s);
    const float mean = s[0] / D;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float c = (j * L + l) * N + k < D ? Run<T>::get(r[j], k) - mean : 0.f;
        s[0] = fmaf(c, c, s[0]);
      }
    row_sum<L, 1>(s);
    const float rstd = 1.f / sqrtf(s[0] / D + p.eps);
    if (l == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = (T*)p.y + (size_t)row * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * L + l) * N, n = D - c0;
      float o[N], w[N], b[N];
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const raw4 rw = p.weight ? Run<float>::load(p.weight + c0 + k, n - k) : raw4{};
        const raw4 rb = p.bias ? Run<float>::load(p.bias + c0 + k, n - k) : raw4{};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[k + i] = p.weight ? Run<float>::get(rw, i) : 1.f;
          b[k + i] = Run<float>::get(rb, i);
        }
      }
#pragma unroll
      for (int k = 0; k < N; ++k) o[k] = fmaf((Run<T>::get(r[j], k) - mean) * rstd, w[k], b[k]);
      Run<T>::store(y + c0, n, o);
    }
    if constexpr (CK) {
      const int G = (D + 127) / 128;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N;
        float v[N];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < N; ++k) {
          v[k] = Run<T>::get(r[j], k);
          const uint32_t b = chan::finite_mag_bits(v[k]);
          m = b > m ? b : m;
        }
        m = lane_max<kGroupLanes>(m);
        const int e = chan::ckpt8_exponent(m);
        Codes<N>::store(p.x_code + (size_t)row * D + c0, D - c0, Codes<N>::pack(v, chan::inv_scale_of(e)));
        if (c0 < D && l % kGroupLanes == 0) p.x_exp[(size_t)row * G + c0 / 128] = (uint8_t)e;
      }
    }
  }
}

// Backward.  Each group of L threads takes every `step`-th row and keeps its
// columns' sums in registers (SUMS); groups are joined over the wave and the
// workgroup, in a fixed order, and a workgroup leaves one partial row of each sum
// for join_kernel.
template <typename T, bool CODES, int NV>
struct BwdRow {
  static constexpr int N = Run<T>::N;
  raw4 y[NV];
  raw4 x[CODES ? 1 : NV];
  typename Codes<N>::R c[CODES ? NV : 1];
  uint8_t e[CODES ? NV : 1];
  float mean, rstd;
};

template <typename T, bool CODES, int L, int NV>
__device__ inline void load_row(const gdr_norm_bwd_args& p, int64_t row, int l, BwdRow<T, CODES, NV>& r) {
  constexpr int N = Run<T>::N;
  const int D = p.D;
  const size_t base = (size_t)row * D;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c0 = (j * L + l) * N;
    r.y[j] = Run<T>::load((const T*)p.grad_y + base + c0, D - c0);
    if constexpr (CODES) {
      r.c[j] = Codes<N>::load((const uint8_t*)p.x + base + c0, D - c0);
      r.e[j] = c0 < D ? p.x_exp[(size_t)row * ((D + 127) / 128) + c0 / 128] : 0;
    } else {
      r.x[j] = Run<T>::load((const T*)p.x + base + c0, D - c0);
    }
  }
  r.mean = p.mean[row];
  r.rstd = p.rstd[row];
}

template <typename T, bool CODES, int L, int NV, bool SUMS>
__global__ __launch_bounds__(threads_of(L)) void norm_bwd_kernel(gdr_norm_bwd_args p, float* part) {
  constexpr int N = Run<T>::N;
  constexpr int kThreads = threads_of(L), kPer = kThreads / L;
  const int l = threadIdx.x % L, D = p.D;
  const int64_t step = (int64_t)gridDim.x * kPer;
  float sw[SUMS ? NV : 1][N], sb[SUMS ? NV : 1][N];
  if constexpr (SUMS) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) sw[j][k] = sb[j][k] = 0.f;
  }
  int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  BwdRow<T, CODES, NV> r;
  if (row < p.R) load_row<T, CODES, L, NV>(p, row, l, r);
  for (; row < p.R; row += step) {
    // the next row is on its way while this one is worked on
    BwdRow<T, CODES, NV> next;
    if (row + step < p.R) load_row<T, CODES, L, NV>(p, row + step, l, next);
    float xh[NV][N], s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * L + l) * N, n = D - c0;
      if constexpr (CODES) {
        Codes<N>::unpack(r.c[j], xh[j]);
        const float sc = chan::scale_of(r.e[j]);
#pragma unroll
        for (int k = 0; k < N; ++k) xh[j][k] = (xh[j][k] * sc - r.mean) * r.rstd;
      } else {
#pragma unroll
        for (int k = 0; k < N; ++k) xh[j][k] = (Run<T>::get(r.x[j], k) - r.mean) * r.rstd;
      }
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const raw4 rw = p.weight ? Run<float>::load(p.weight + c0 + k, n - k) : raw4{};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float dy = Run<T>::get(r.y[j], k + i);   // 0 behind the row's end
          const float g = dy * (p.weight ? Run<float>::get(rw, i) : 1.f);
          s[0] += g;
          s[1] = fmaf(g, n > k + i ? xh[j][k + i] : 0.f, s[1]);
        }
      }
    }
    row_sum<L, 2>(s);
    s[0] /= D;
    s[1] /= D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c0 = (j * L + l) * N, n = D - c0;
      float o[N];
#pragma unroll
      for (int k = 0; k < N; k += 4) {
        const raw4 rw = p.weight ? Run<float>::load(p.weight + c0 + k, n - k) : raw4{};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float dy = Run<T>::get(r.y[j], k + i);
          const float g = dy * (p.weight ? Run<float>::get(rw, i) : 1.f);
          o[k + i] = r.rstd * (g - s[0] - xh[j][k + i] * s[1]);
          if constexpr (SUMS) {
            sw[j][k + i] = fmaf(dy, xh[j][k + i], sw[j][k + i]);
            sb[j][k + i] += dy;
          }
        }
      }
      Run<T>::store((T*)p.grad_x + (size_t)row * D + c0, n, o);
    }
    r = next;
  }
  if constexpr (SUMS) {
    float* pw = part + (size_t)blockIdx.x * 2 * D;
    if constexpr (L >= kThreads) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N;
#pragma unroll
        for (int k = 0; k < N; ++k)
          if (c0 + k < D) {
            pw[c0 + k] = sw[j][k];
            pw[D + c0 + k] = sb[j][k];
          }
      }
    } else {
      // lane groups, then waves
      __shared__ float join[kThreads / 64][2][(L < 64 ? L : 64) * N];
      const int w = threadIdx.x >> 6;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
          for (int off = L; off < 64; off <<= 1) {
            sw[j][k] += __shfl_xor(sw[j][k], off);
            sb[j][k] += __shfl_xor(sb[j][k], off);
          }
        __syncthreads();
        if ((threadIdx.x & 63) < L) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            join[w][0][l * N + k] = sw[j][k];
            join[w][1][l * N + k] = sb[j][k];
          }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * L * N; i += kThreads) {
          const int which = i / (L * N), c = i % (L * N);
          float t = 0.f;
#pragma unroll
          for (int q = 0; q < kThreads / 64; ++q) t += join[q][which][c];
          if (j * L * N + c < D) pw[(size_t)which * D + j * L * N + c] = t;
        }
      }
    }
  }
}

// Columns' sums of rows that are too long for registers to hold them beside a row:
// a second pass, one thread per column and row part.
template <typename T, bool CODES>
__global__ __launch_bounds__(256) void norm_cols_kernel(gdr_norm_bwd_args p, float* part) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= p.D) return;
  float sw = 0.f, sb = 0.f;
  for (int64_t r = blockIdx.y; r < p.R; r += gridDim.y) {
    const size_t i = (size_t)r * p.D + c;
    const float dy = chan::ld((const T*)p.grad_y + i);
    float x;
    if constexpr (CODES)
      x = chan::code1_f32(((const uint8_t*)p.x)[i]) * chan::scale_of(p.x_exp[(size_t)r * ((p.D + 127) / 128) + c / 128]);
    else
      x = chan::ld((const T*)p.x + i);
    sw = fmaf(dy, (x - p.mean[r]) * p.rstd[r], sw);
    sb += dy;
  }
  float* pw = part + (size_t)blockIdx.y * 2 * p.D;
  pw[c] = sw;
  pw[p.D + c] = sb;
}

// grad_weight and grad_bias from the partial rows: 16 threads a column take every
// 16th, then join.
__global__ __launch_bounds__(512) void join_kernel(const float* part, int rows, int D, float* gw, float* gb) {
  __shared__ float s[16][32];
  const int l = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + l;   // of 2 D: the weight's columns, then the bias'
  float t = 0.f;
  if (c < 2 * D)
    for (int r = y; r < rows; r += 16) t += part[(size_t)r * 2 * D + c];
  s[y][l] = t;
  __syncthreads();
  if (y == 0 && c < 2 * D) {
#pragma unroll
    for (int k = 1; k < 16; ++k) t += s[k][l];
    if (c < D) {
      if (gw) gw[c] = t;
    } else if (gb) {
      gb[c - D] = t;
    }
  }
}

// Threads of a row and runs of a thread, by the row's number of runs.
struct Shape {
  int L, NV;
};
constexpr Shape shape_of(int runs) {
  if (runs <= 8) return {8, 1};
  if (runs <= 16) return {16, 1};
  if (runs <= 32) return {32, 1};
  if (runs <= 256) return {64, runs <= 64 ? 1 : runs <= 128 ? 2 : runs <= 192 ? 3 : 4};
  if (runs <= 2048) return {256, runs <= 512 ? 2 : runs <= 768 ? 3 : runs <= 1024 ? 4 : runs <= 1280 ? 5 : runs <= 1536 ? 6 : 8};
  return {1024, runs <= 4096 ? 4 : runs <= 8192 ? 8 : 16};
}
inline int runs_of(int D, int io_dtype) { const int n = io_dtype == GDR_BF16 ? 8 : 4; return (D + n - 1) / n; }
inline int64_t rows_per_group(int L) { return threads_of(L) / L; }

// Workgroups of a forward launch (a grid holds 2^32 threads); they take further rows in turn.
constexpr int64_t kMaxGroups = 1 << 20;

// Partial rows of the columns' sums: enough workgroups to fill the card, no more
// than there are rows for.
constexpr int kParts = 512;
inline int parts_of(int64_t R, int L) {
  const int64_t n = (R + rows_per_group(L) - 1) / rows_per_group(L);
  return (int)(n < kParts ? n : kParts);
}

size_t bwd_workspace(int64_t R, int D) {
  (void)R;
  return (size_t)kParts * 2 * D * sizeof(float);
}

#define GDR_NORM_SHAPES(X)                                                                                      \
  X(8, 1) X(16, 1) X(32, 1) X(64, 1) X(64, 2) X(64, 3) X(64, 4) X(256, 2) X(256, 3) X(256, 4) X(256, 5) X(256, 6) \
  X(256, 8) X(1024, 4) X(1024, 8) X(1024, 16)

template <typename T>
static hipError_t fwd(const gdr_norm_args& a, hipStream_t s) {
  const Shape sh = shape_of(runs_of(a.D, a.io_dtype));
  const int64_t groups = (a.R + rows_per_group(sh.L) - 1) / rows_per_group(sh.L);
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
#define GDR_LAUNCH(LL, NN)                                                                                            \
  if (sh.L == LL && sh.NV == NN) {                                                                                    \
    if constexpr (LL * NN * Run<T>::N <= 65536) {                                                                     \
      if (a.x_code) hipLaunchKernelGGL((norm_fwd_kernel<T, LL, NN, true>), grid, dim3(threads_of(LL)), 0, s, a);      \
      else hipLaunchKernelGGL((norm_fwd_kernel<T, LL, NN, false>), grid, dim3(threads_of(LL)), 0, s, a);              \
      return hipGetLastError();                                                                                       \
    }                                                                                                                 \
  }
  GDR_NORM_SHAPES(GDR_LAUNCH)
#undef GDR_LAUNCH
  return hipErrorInvalidValue;
}

template <typename T, bool CODES>
static hipError_t bwd(const gdr_norm_bwd_args& a, hipStream_t s) {
  const Shape sh = shape_of(runs_of(a.D, a.io_dtype));
  const bool sums = a.grad_weight || a.grad_bias;
  const int parts = parts_of(a.R, sh.L);
  float* part = (float*)a.workspace;
  const bool beside = sh.L <= 256;   // the sums fit beside the row
  bool launched = false;
#define GDR_LAUNCH(LL, NN)                                                                                           \
  if (sh.L == LL && sh.NV == NN) {                                                                                   \
    if constexpr (LL * NN * Run<T>::N <= 65536) {                                                                    \
      if constexpr (LL <= 256) {                                                                                     \
        if (sums) hipLaunchKernelGGL((norm_bwd_kernel<T, CODES, LL, NN, true>), dim3(parts), dim3(256), 0, s, a, part); \
      }                                                                                                              \
      if (!sums || !beside)                                                                                          \
        hipLaunchKernelGGL((norm_bwd_kernel<T, CODES, LL, NN, false>), dim3(parts), dim3(threads_of(LL)), 0, s, a, part); \
      launched = true;                                                                                               \
    }                                                                                                                \
  }
  GDR_NORM_SHAPES(GDR_LAUNCH)
#undef GDR_LAUNCH
  if (!launched) return hipErrorInvalidValue;
  if (sums) {
    int rows = parts;
    if (!beside) {
      rows = a.R < kParts ? (int)a.R : kParts;
      hipLaunchKernelGGL((norm_cols_kernel<T, CODES>), dim3((a.D + 255) / 256, rows), dim3(256), 0, s, a, part);
    }
    hipLaunchKernelGGL(join_kernel, dim3((2 * a.D + 31) / 32), dim3(512), 0, s, part, rows, a.D, a.grad_weight, a.grad_bias);
  }
  return hipGetLastError();
}

hipError_t launch_norm_fwd(const gdr_norm_args& a, hipStream_t s) {
  return a.io_dtype == GDR_BF16 ? fwd<__bf16>(a, s) : fwd<float>(a, s);
}

hipError_t launch_norm_bwd(const gdr_norm_bwd_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) return a.x_exp ? bwd<__bf16, true>(a, s) : bwd<__bf16, false>(a, s);
  return a.x_exp ? bwd<float, true>(a, s) : bwd<float, false>(a, s);
}

}  // namespace norm
}  // namespace gdr
