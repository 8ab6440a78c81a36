// conv_kernels.h -- launch interface of the short causal convolution.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_conv.h"

namespace gdr {
namespace conv {

constexpr int kMinK = 2, kMaxK = 8;

// Workgroups of a launch stay below 2^22: with stretches of 64 tokens there are no more than
// this counts, and shorter ones are taken only while all stretches together need at most
// 128 Ki threads.
constexpr bool too_many_tiles(int B, int T, int C) {
  return (long long)B * ((C + 255) / 256) * ((T + 255) / 256) >= (1LL << 22);
}

size_t bwd_workspace(int B, int T, int C, int K);

// Arguments already checked; a.workspace large enough.
hipError_t launch_conv_fwd(const gdr_conv_args& a, hipStream_t s);
hipError_t launch_conv_bwd(const gdr_conv_bwd_args& a, hipStream_t s);
hipError_t launch_conv_step(const gdr_conv_step_args& a, hipStream_t s);

}  // namespace conv
}  // namespace gdr
