// gnorm_kernels.h -- launch interface of the gated group norm.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_gnorm.h"

namespace gdr {
namespace gnorm {

constexpr int kMaxGroup = 16384;

size_t bwd_workspace(int64_t R, int C, int G, int io_dtype);

// Arguments already checked; a.workspace large enough.
hipError_t launch_gnorm_fwd(const gdr_gnorm_args& a, hipStream_t s);
hipError_t launch_gnorm_bwd(const gdr_gnorm_bwd_args& a, hipStream_t s);

}  // namespace gnorm
}  // namespace gdr
