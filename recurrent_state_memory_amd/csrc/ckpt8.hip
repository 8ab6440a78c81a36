// ckpt8.hip -- 8-bit activation checkpoints: pack and unpack, gfx950.
//
// A group of 128 values is 16 lanes of 8 bf16 values or 32 lanes of 4 fp32 ones,
// 16 bytes a lane; lanes are numbered over all groups of all rows, so short rows
// waste no wave.  Both directions are bound by HBM: 32768 x 2048 bf16 packed and
// unpacked again in 75 us, 404 MB at 5.4 TB/s.
#include "chan_device.h"
#include "norm_kernels.h"

namespace gdr {
namespace ckpt8 {

using chan::Codes;
using chan::raw4;
using chan::Run;

constexpr int kMany = 4;   // groups a lane has under way at once

// A lane's run of one group.
struct Spot {
  size_t row;
  int c0, n;   // first column, values that exist (none: <= 0)
};
template <int N>
__device__ inline Spot spot_of(size_t g, size_t groups, int per_row, int D) {
  constexpr int kLanes = GDR_CKPT8_GROUP / N;
  if (g >= groups) return Spot{0, 0, 0};
  const size_t row = per_row == 1 ? g : g / per_row;
  const int c0 = (int)(g - row * per_row) * GDR_CKPT8_GROUP + (int)(threadIdx.x % kLanes) * N;
  return Spot{row, c0, D - c0};
}

template <typename T>
__global__ __launch_bounds__(256) void pack_kernel(gdr_ckpt8_pack_args p, size_t groups, int per_row) {
  constexpr int N = Run<T>::N, kLanes = GDR_CKPT8_GROUP / N, kPer = 256 / kLanes;
  const size_t step = (size_t)gridDim.x * kPer;
  for (size_t g0 = (size_t)blockIdx.x * kPer + threadIdx.x / kLanes; g0 < groups; g0 += kMany * step) {
    Spot q[kMany];
    raw4 r[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      q[i] = spot_of<N>(g0 + i * step, groups, per_row, p.D);
      r[i] = Run<T>::load((const T*)p.x + q[i].row * p.D + q[i].c0, q[i].n);
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      int e;
      const auto c = chan::pack_run<T, kLanes>(r[i], e);
      Codes<N>::store(p.code + q[i].row * p.D + q[i].c0, q[i].n, c);
      if (threadIdx.x % kLanes == 0 && q[i].n > 0) p.exp[g0 + i * step] = (uint8_t)e;
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void unpack_kernel(gdr_ckpt8_unpack_args p, size_t groups, int per_row) {
  constexpr int N = Run<T>::N, kLanes = GDR_CKPT8_GROUP / N, kPer = 256 / kLanes;
  const size_t step = (size_t)gridDim.x * kPer;
  for (size_t g0 = (size_t)blockIdx.x * kPer + threadIdx.x / kLanes; g0 < groups; g0 += kMany * step) {
    Spot q[kMany];
    typename Codes<N>::R r[kMany];
    uint8_t e[kMany];
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      q[i] = spot_of<N>(g0 + i * step, groups, per_row, p.D);
      r[i] = Codes<N>::load(p.code + q[i].row * p.D + q[i].c0, q[i].n);
      e[i] = q[i].n > 0 ? p.exp[g0 + i * step] : 0;
    }
#pragma unroll
    for (int i = 0; i < kMany; ++i) {
      float v[N];
      Codes<N>::unpack(r[i], v);
      const float sc = chan::scale_of(e[i]);
#pragma unroll
      for (int k = 0; k < N; ++k) v[k] *= sc;
      Run<T>::store((T*)p.x + q[i].row * p.D + q[i].c0, q[i].n, v);
    }
  }
}

struct Grid {
  size_t groups;
  int per_row;
  dim3 blocks;
};
static Grid grid_of(int64_t R, int D, int n) {
  Grid g;
  g.per_row = (D + GDR_CKPT8_GROUP - 1) / GDR_CKPT8_GROUP;
  g.groups = (size_t)R * g.per_row;
  const size_t per = 256 / (GDR_CKPT8_GROUP / n), want = (g.groups + per * kMany - 1) / (per * kMany);
  g.blocks = dim3((unsigned)(want < 8192 ? want : 8192));
  return g;
}

hipError_t launch_pack(const gdr_ckpt8_pack_args& a, hipStream_t s) {
  const Grid g = grid_of(a.R, a.D, a.io_dtype == GDR_BF16 ? 8 : 4);
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(pack_kernel<__bf16>, g.blocks, dim3(256), 0, s, a, g.groups, g.per_row);
  else hipLaunchKernelGGL(pack_kernel<float>, g.blocks, dim3(256), 0, s, a, g.groups, g.per_row);
  return hipGetLastError();
}

hipError_t launch_unpack(const gdr_ckpt8_unpack_args& a, hipStream_t s) {
  const Grid g = grid_of(a.R, a.D, a.io_dtype == GDR_BF16 ? 8 : 4);
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(unpack_kernel<__bf16>, g.blocks, dim3(256), 0, s, a, g.groups, g.per_row);
  else hipLaunchKernelGGL(unpack_kernel<float>, g.blocks, dim3(256), 0, s, a, g.groups, g.per_row);
  return hipGetLastError();
}

}  // namespace ckpt8
}  // namespace gdr
