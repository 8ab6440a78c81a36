// col_join.h -- sums of partial rows, shared by the operators whose workgroups each leave
// one row of a parameter's gradient: out(i, sum over r of part[r][i]) for every column i.
// A workgroup takes 32 columns, 32 threads each, which read four rows at once: the kernel
// is a few loads' latency long.  The order of the sums depends on the number of rows alone.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>

namespace gdr {

constexpr int kJoinCols = 32, kJoinWays = 32;

template <typename Out>
__global__ __launch_bounds__(kJoinCols * kJoinWays) void col_join_kernel(const float* part, size_t rows, size_t width, Out out) {
  __shared__ float sum[kJoinWays][kJoinCols];
  const int tx = threadIdx.x % kJoinCols, ty = threadIdx.x / kJoinCols;
  const size_t i = (size_t)blockIdx.x * kJoinCols + tx;
  float a = 0.f;
  if (i < width)
    for (size_t r = ty; r < rows; r += 4 * kJoinWays) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = r + k * kJoinWays < rows ? part[(r + k * kJoinWays) * width + i] : 0.f;
      a += (v[0] + v[1]) + (v[2] + v[3]);
    }
  sum[ty][tx] = a;
  __syncthreads();
  if (ty == 0 && i < width) {
    a = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWays; ++k) a += sum[k][tx];
    out(i, a);
  }
}

template <typename Out>
inline void launch_col_join(const float* part, size_t rows, size_t width, Out out, hipStream_t s) {
  hipLaunchKernelGGL(col_join_kernel<Out>, dim3((unsigned)((width + kJoinCols - 1) / kJoinCols)),
                     dim3(kJoinCols * kJoinWays), 0, s, part, rows, width, out);
}

}  // namespace gdr
