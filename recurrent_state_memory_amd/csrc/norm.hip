// norm.hip -- layer norm forward and backward, gfx950.
//
// A row is held in registers by L threads of NV 16-byte runs each (thread l has
// runs l, l + L, ...), so it is read once: the mean, then the squares about it,
// then the outputs.  L is a part of a wave for short rows (64 / L rows side by side
// in a wave, no barrier), a wave, or up to 1024 threads: few runs a thread, since what
// is under way at once hides the latency (backward of 64 Mi bf16 elements in rows of
// 8192: one run of each of 1024 threads 82 us, four of 256 142 us).  Both kernels are
// bound by HBM: forward of 32768 x 2048 bf16 53 us (5.1 TB/s), with the 8-bit copy 69 us
// (4.9 TB/s), backward 79 us (5.1 TB/s); per-head rows of 128 channels 57 and 80 us.
// Registers spill in the forward of fp32 rows above 32768 (512 x 65536: 110 us, 2.4 TB/s)
// and, a few of them, in the backward from codes at the longest rows held.
#include "chan_device.h"
#include "norm_kernels.h"

namespace gdr {
namespace norm {

using chan::Codes;
using chan::lane_sum;
using chan::raw4;
using chan::Run;

constexpr int threads_of(int L) { return L > 256 ? L : 256; }   // of a forward workgroup

// Sums over the row's L threads of a workgroup of TH; more than a wave: through LDS,
// in one of two places by turns, so that one barrier a sum is enough.
template <int TH, int NSUM>
struct RowSums {
  float part[2][NSUM][TH / 64];
};
template <int TH, int L, int NSUM>
__device__ inline void row_sum(float (&v)[NSUM], RowSums<TH, NSUM>& lds, int& turn) {
  constexpr int W = L / 64;
#pragma unroll
  for (int i = 0; i < NSUM; ++i) v[i] = lane_sum<(L < 64 ? L : 64)>(v[i]);
  if constexpr (W > 1) {
    const int w = threadIdx.x >> 6, w0 = w / W * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < NSUM; ++i) lds.part[turn][i][w] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NSUM; ++i) {
      float s = 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) s += lds.part[turn][i][w0 + k];
      v[i] = s;
    }
    turn ^= 1;
  }
}

template <typename T, int L, int NV, bool CK>
__global__ __launch_bounds__(threads_of(L)) void norm_fwd_kernel(gdr_norm_args p) {
  constexpr int N = Run<T>::N;
  constexpr int kPer = threads_of(L) / L;           // rows of a workgroup
  constexpr int kGroupLanes = 128 / N < L ? 128 / N : L;
  __shared__ RowSums<threads_of(L), 1> sums;
  int turn = 0;
  const int l = threadIdx.x % L;
  const int D = p.D;
  const int64_t step = (int64_t)gridDim.x * kPer;
  // Rows of several waves that share a workgroup meet in row_sum: all of them make the
  // same number of rounds, and where one has no row left it reads the last one again.
  // (A workgroup for each row of two waves: up to 10 % slower.)
  constexpr bool kMeet = L > 64 && kPer > 1;
  const int64_t own = threadIdx.x / L;
  for (int64_t first = (int64_t)blockIdx.x * kPer + (kMeet ? 0 : own); first < p.R; first += step) {
    const bool here = !kMeet || first + own < p.R;
    const int64_t row = !kMeet ? first : here ? first + own : p.R - 1;
    const T* x = (const T*)p.x + (size_t)row * D;
    raw4 r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) r[j] = Run<T>::load(x + (j * L + l) * N, D - (j * L + l) * N);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) s[0] += Run<T>::get(r[j], k);   // 0 behind the row's end
    row_sum<threads_of(L), L>(s, sums, turn);
    const float mean = s[0] / D;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) {
        const float c = (j * L + l) * N + k < D ? Run<T>::get(r[j], k) - mean : 0.f;
        s[0] = fmaf(c, c, s[0]);
      }
    row_sum<threads_of(L), L>(s, sums, turn);
    if (!here) continue;   // no sum follows in this round
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
        int e;
        const auto c = chan::pack_run<T, kGroupLanes>(r[j], e);
        Codes<N>::store(p.x_code + (size_t)row * D + c0, D - c0, c);
        if (c0 < D && l % kGroupLanes == 0) p.x_exp[(size_t)row * G + c0 / 128] = (uint8_t)e;
      }
    }
  }
}

// Backward.  A workgroup of 1024 threads takes 1024 / L rows at a time, every
// (gridDim 1024 / L)-th; a thread keeps its columns' sums in registers (SUMS).  Groups
// are joined over the wave and the workgroup, in a fixed order, and a workgroup
// leaves one partial row of each sum for join_kernel.
template <typename T, bool CODES, int NV>
struct BwdRow {
  static constexpr int N = Run<T>::N;
  raw4 y[NV];
  raw4 x[CODES ? 1 : NV];
  typename Codes<N>::R c[CODES ? NV : 1];
  uint8_t e[CODES ? NV : 1];
  float mean, rstd;
  // x of run j as fp32
  __device__ inline void get_x(int j, float (&v)[N]) const {
    if constexpr (CODES) {
      Codes<N>::unpack(c[j], v);
      const float sc = chan::scale_of(e[j]);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] *= sc;
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] = Run<T>::get(x[j], k);
    }
  }
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

// weight of the columns from c0 on (1 without weights), 0 behind the row's end
template <int N>
__device__ inline void load_weight(const gdr_norm_bwd_args& p, int c0, float (&w)[N]) {
#pragma unroll
  for (int k = 0; k < N; k += 4) {
    const int n = p.D - c0 - k;
    const raw4 r = p.weight ? Run<float>::load(p.weight + c0 + k, n) : raw4{};
#pragma unroll
    for (int i = 0; i < 4; ++i) w[k + i] = p.weight ? Run<float>::get(r, i) : n > i ? 1.f : 0.f;
  }
}

template <typename T, bool CODES, int L, int NV, bool SUMS>
__global__ __launch_bounds__(1024) void norm_bwd_kernel(gdr_norm_bwd_args p, float* part) {
  constexpr int TH = 1024;
  constexpr int N = Run<T>::N;
  constexpr int kPer = TH / L;
  constexpr int kJoin = SUMS && L < TH ? TH / (L < 64 ? 64 : L) : 1;   // sets of sums that meet in LDS
  __shared__ RowSums<TH, 2> sums;
  __shared__ float join[kJoin][kJoin > 1 ? L * N : 1];
  int turn = 0;
  const int l = threadIdx.x % L, D = p.D;
  const int64_t step = (int64_t)gridDim.x * kPer;
  float sw[SUMS ? NV : 1][N], sb[SUMS ? NV : 1][N], w[NV][N];   // the weights stay in registers
  if constexpr (SUMS) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < N; ++k) sw[j][k] = sb[j][k] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) load_weight<N>(p, (j * L + l) * N, w[j]);
  BwdRow<T, CODES, NV> r;
  int64_t row = (int64_t)blockIdx.x * kPer + threadIdx.x / L;
  if (row < p.R) load_row<T, CODES, L, NV>(p, row, l, r);
  // the workgroup's threads make the same number of rounds: they meet in row_sum
  for (int64_t first = (int64_t)blockIdx.x * kPer; first < p.R; first += step, row += step) {
    const bool here = row < p.R;
    BwdRow<T, CODES, NV> next;
    if (row + step < p.R) load_row<T, CODES, L, NV>(p, row + step, l, next);   // on its way meanwhile
    float s[2] = {0.f, 0.f};
    if (here) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float x[N];
        r.get_x(j, x);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          // behind the row's end grad_y and the weight read as 0
          const float dy = Run<T>::get(r.y[j], k), g = dy * w[j][k];
          const float xh = (x[k] - r.mean) * r.rstd;
          s[0] += g;
          s[1] = fmaf(g, xh, s[1]);
          if constexpr (SUMS) {
            sw[j][k] = fmaf(dy, xh, sw[j][k]);
            sb[j][k] += dy;
          }
        }
      }
    }
    row_sum<TH, L>(s, sums, turn);
    s[0] /= D;
    s[1] /= D;
    if (here) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c0 = (j * L + l) * N;
        float x[N], o[N];
        r.get_x(j, x);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float xh = (x[k] - r.mean) * r.rstd;
          o[k] = r.rstd * (fmaf(Run<T>::get(r.y[j], k), w[j][k], -s[0]) - xh * s[1]);
        }
        Run<T>::store((T*)p.grad_x + (size_t)row * D + c0, D - c0, o);
      }
    }
    r = next;
  }
  if constexpr (SUMS) {
    float* pw = part + (size_t)blockIdx.x * 2 * D;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        float* out = pw + (size_t)which * D;
        float t[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
          t[k] = which == 0 ? sw[j][k] : sb[j][k];
#pragma unroll
          for (int off = L; off < 64; off <<= 1) t[k] += __shfl_xor(t[k], off);
        }
        if constexpr (kJoin == 1) {
          Run<float>::store(out + (j * L + l) * N, D - (j * L + l) * N, *(const float(*)[4]) & t[0]);
          if constexpr (N == 8)
            Run<float>::store(out + (j * L + l) * N + 4, D - (j * L + l) * N - 4, *(const float(*)[4]) & t[4]);
        } else {
          const int set = threadIdx.x / (L < 64 ? 64 : L);
          if (L >= 64 || (threadIdx.x & 63) < L) {
#pragma unroll
            for (int k = 0; k < N; ++k) join[set][l * N + k] = t[k];
          }
          __syncthreads();
          for (int c = threadIdx.x; c < L * N; c += TH) {
            float u = 0.f;
#pragma unroll
            for (int q = 0; q < kJoin; ++q) u += join[q][c];
            if (j * L * N + c < D) out[j * L * N + c] = u;
          }
          __syncthreads();
        }
      }
    }
  }
}

// Rows longer than 1024 threads hold beside their sums: a workgroup a row, read twice,
// the second time mostly from the caches (fp32 512 x 65536: 229 us; held in registers,
// which spilled, 537).
template <typename T, bool CODES>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(gdr_norm_bwd_args p) {
  constexpr int N = Run<T>::N;
  __shared__ RowSums<1024, 2> sums;
  int turn = 0;
  const int D = p.D, runs = (D + N - 1) / N;
  for (int64_t row = blockIdx.x; row < p.R; row += gridDim.x) {
    const float mean = p.mean[row], rstd = p.rstd[row];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      for (int j = threadIdx.x; j < runs; j += 1024) {
        BwdRow<T, CODES, 1> r;
        load_row<T, CODES, 0, 1>(p, row, j, r);   // run j alone
        float x[N], w[N], o[N];
        r.get_x(0, x);
        load_weight<N>(p, j * N, w);
#pragma unroll
        for (int k = 0; k < N; ++k) {
          const float g = Run<T>::get(r.y[0], k) * w[k], xh = (x[k] - mean) * rstd;
          if (pass == 0) {
            s[0] += g;
            s[1] = fmaf(g, xh, s[1]);
          } else {
            o[k] = rstd * ((g - s[0]) - xh * s[1]);
          }
        }
        if (pass == 1) Run<T>::store((T*)p.grad_x + (size_t)row * D + j * N, D - j * N, o);
      }
      if (pass == 0) {
        row_sum<1024, 1024>(s, sums, turn);
        s[0] /= D;
        s[1] /= D;
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

// grad_weight and grad_bias from the partial rows: 64 threads a column take every
// 64th, then join.
__global__ __launch_bounds__(1024) void join_kernel(const float* part, int rows, int D, float* gw, float* gb) {
  __shared__ float s[64][17];
  const int l = threadIdx.x & 15, y = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + l;   // of 2 D: the weight's columns, then the bias'
  float t = 0.f;
  if (c < 2 * D)
    for (int r = y; r < rows; r += 64) t += part[(size_t)r * 2 * D + c];
  s[y][l] = t;
  __syncthreads();
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;   // a wave joins a column
  t = chan::lane_sum<64>(s[lane][w]);
  const int cw = blockIdx.x * 16 + w;
  if (lane == 0 && cw < 2 * D) {
    if (cw < D) {
      if (gw) gw[cw] = t;
    } else if (gb) {
      gb[cw - D] = t;
    }
  }
}

// Threads of a row and runs of a thread, by the row's number of runs.
struct Shape {
  int L, NV;
};
constexpr Shape fwd_shape(int runs, bool ck) {
  if (runs <= 2) return {2, 1};
  if (runs <= 4) return {4, 1};
  if (runs <= 8) return {8, 1};
  if (runs <= 16) return {16, 1};
  if (runs <= 32) return {32, 1};
  if (runs <= 64) return {64, 1};
  if (runs <= 128) return {64, 2};
  if (ck) {   // packing wants registers: fewer runs a thread
    if (runs <= 384) return {128, runs <= 256 ? 2 : 3};
    if (runs <= 1024) return {256, runs <= 512 ? 2 : runs <= 768 ? 3 : 4};
    return {512, runs <= 1536 ? 3 : runs <= 2048 ? 4 : 0};   // 0: packed by a launch of its own
  }
  if (runs <= 256) return {64, runs <= 192 ? 3 : 4};
  if (runs <= 384) return {128, 3};
  if (runs <= 1024) return {256, runs <= 512 ? 2 : runs <= 768 ? 3 : 4};
  if (runs <= 2048) return {512, runs <= 1536 ? 3 : 4};
  return {1024, runs <= 4096 ? 4 : runs <= 8192 ? 8 : 16};
}
constexpr Shape bwd_shape(int runs, int N) {
  if (runs <= 2) return {2, 1};
  if (runs <= 4) return {4, 1};
  if (runs <= 8) return {8, 1};
  if (runs <= 16) return {16, 1};
  if (runs <= 32) return {32, 1};
  if (runs <= 64) return {64, 1};
  if (runs <= 128) return {128, 1};
  if (runs <= 256) return {256, 1};
  if (runs <= 512) return {512, 1};
  if (N == 8 && runs <= 1024) return {1024, 1};
  if (N == 4 && runs <= 1536) return {512, runs <= 1024 ? 2 : 3};
  if (runs <= 2048) return {1024, 2};
  if (N == 4 && runs <= 3 * 1024) return {1024, 3};
  return {1024, 0};   // norm_bwd_long_kernel
}
#define GDR_NORM_SHAPES(X) X(2, 1) X(4, 1) X(8, 1) X(16, 1) X(32, 1) X(64, 1) X(512, 3)
#define GDR_NORM_FWD_SHAPES(X) \
  X(64, 2) X(64, 3) X(64, 4) X(128, 2) X(128, 3) X(256, 2) X(256, 3) X(256, 4) X(512, 4) X(1024, 4) X(1024, 8) X(1024, 16)
#define GDR_NORM_BWD_SHAPES(X) X(128, 1) X(256, 1) X(512, 1) X(512, 2) X(1024, 1) X(1024, 2) X(1024, 3)

// How often the launches below name a shape: each that a row has, once.
constexpr int fwd_listed(Shape s) {
#define GDR_COUNT(LL, NN) + (s.L == LL && s.NV == NN)
  return 0 GDR_NORM_SHAPES(GDR_COUNT) GDR_NORM_FWD_SHAPES(GDR_COUNT);
}
constexpr int bwd_listed(Shape s) {
  return 0 GDR_NORM_SHAPES(GDR_COUNT) GDR_NORM_BWD_SHAPES(GDR_COUNT);
#undef GDR_COUNT
}
constexpr bool all_listed(int N) {
  for (int runs = 1; runs <= 65536 / N; runs += runs < 64 ? 1 : 64) {   // shapes change after multiples of 64
    const Shape f = fwd_shape(runs, false), k = fwd_shape(runs, true), b = bwd_shape(runs, N);
    if (fwd_listed(f) != 1 || (k.NV > 0 && fwd_listed(k) != 1) || (b.NV > 0 && bwd_listed(b) != 1)) return false;
  }
  return true;
}
static_assert(all_listed(4) && all_listed(8), "every row's shape has a kernel");
// Whether some row of runs of N values has this shape.
constexpr bool bwd_has(int N, int L, int NV) {
  for (int runs = 1; runs <= 3 * 1024; ++runs)
    if (bwd_shape(runs, N).L == L && bwd_shape(runs, N).NV == NV) return true;
  return false;
}
constexpr bool fwd_has(int N, int L, int NV, bool ck) {
  for (int runs = 1; runs <= 65536 / N; runs += runs < 64 ? 1 : 64)
    if (fwd_shape(runs, ck).L == L && fwd_shape(runs, ck).NV == NV) return true;
  return false;
}
inline int runs_of(int D, int io_dtype) { const int n = io_dtype == GDR_BF16 ? 8 : 4; return (D + n - 1) / n; }

// Workgroups of a forward launch (a grid holds 2^32 threads); they take further rows in turn.
constexpr int64_t kMaxGroups = 1 << 20;

// Workgroups of a backward launch, and partial rows of the columns' sums: one for each
// CU, as more mostly write more partial rows (fp32 5000 x 5003: 512 took 85 us, 256 76).
constexpr int kParts = 256;

size_t bwd_workspace(int64_t R, int D) {
  (void)R;
  return (size_t)kParts * 2 * D * sizeof(float);
}

template <typename T>
static hipError_t fwd(const gdr_norm_args& a, hipStream_t s) {
  constexpr int N = Run<T>::N;
  const int runs = runs_of(a.D, a.io_dtype);
  const bool ck = a.x_code && fwd_shape(runs, true).NV > 0;   // packed on the way
  const Shape sh = fwd_shape(runs, ck);
  const int per = threads_of(sh.L) / sh.L;
  const int64_t groups = (a.R + per - 1) / per;
  const dim3 grid((unsigned)(groups < kMaxGroups ? groups : kMaxGroups));
#define GDR_LAUNCH(LL, NN)                                                                               \
  if (sh.L == LL && sh.NV == NN) {                                                                       \
    if constexpr (fwd_has(N, LL, NN, true))                                                              \
      if (ck) hipLaunchKernelGGL((norm_fwd_kernel<T, LL, NN, true>), grid, dim3(threads_of(LL)), 0, s, a); \
    if constexpr (fwd_has(N, LL, NN, false))                                                             \
      if (!ck) hipLaunchKernelGGL((norm_fwd_kernel<T, LL, NN, false>), grid, dim3(threads_of(LL)), 0, s, a); \
  }
  GDR_NORM_SHAPES(GDR_LAUNCH)
  GDR_NORM_FWD_SHAPES(GDR_LAUNCH)
#undef GDR_LAUNCH
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.x_code || ck) return e;
  const gdr_ckpt8_pack_args c{a.R, a.D, a.io_dtype, a.x, a.x_code, a.x_exp};
  return ckpt8::launch_pack(c, s);
}

template <typename T, bool CODES>
static hipError_t bwd(const gdr_norm_bwd_args& a, hipStream_t s) {
  constexpr int N = Run<T>::N;
  const Shape sh = bwd_shape(runs_of(a.D, a.io_dtype), N);
  const bool sums = a.grad_weight || a.grad_bias;
  float* part = (float*)a.workspace;
  int parts = (int)(a.R < kParts ? a.R : kParts);
  if (sh.NV == 0) {
    hipLaunchKernelGGL((norm_bwd_long_kernel<T, CODES>), dim3(parts), dim3(1024), 0, s, a);
    if (sums) hipLaunchKernelGGL((norm_cols_kernel<T, CODES>), dim3((a.D + 255) / 256, parts), dim3(256), 0, s, a, part);
  } else {
    const int per = 1024 / sh.L;
    const int64_t groups = (a.R + per - 1) / per;
    if (groups < parts) parts = (int)groups;
#define GDR_LAUNCH(LL, NN)                                                                                             \
  if constexpr (bwd_has(N, LL, NN)) {                                                                                  \
    if (sh.L == LL && sh.NV == NN) {                                                                                   \
      if (sums) hipLaunchKernelGGL((norm_bwd_kernel<T, CODES, LL, NN, true>), dim3(parts), dim3(1024), 0, s, a, part); \
      else hipLaunchKernelGGL((norm_bwd_kernel<T, CODES, LL, NN, false>), dim3(parts), dim3(1024), 0, s, a, part);     \
    }                                                                                                                  \
  }
    GDR_NORM_SHAPES(GDR_LAUNCH)
    GDR_NORM_BWD_SHAPES(GDR_LAUNCH)
#undef GDR_LAUNCH
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !sums) return e;
  hipLaunchKernelGGL(join_kernel, dim3((2 * a.D + 15) / 16), dim3(1024), 0, s, part, parts, a.D, a.grad_weight, a.grad_bias);
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
