// norm_kernels.h -- launch interface of the layer norm and the 8-bit checkpoints.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_ckpt8.h"
#include "../../include/gdr_norm.h"

namespace gdr {
namespace norm {

size_t bwd_workspace(int64_t R, int D);

// Arguments already checked; a.workspace large enough.
hipError_t launch_norm_fwd(const gdr_norm_args& a, hipStream_t s);
hipError_t launch_norm_bwd(const gdr_norm_bwd_args& a, hipStream_t s);

}  // namespace norm
namespace ckpt8 {

hipError_t launch_pack(const gdr_ckpt8_pack_args& a, hipStream_t s);
hipError_t launch_unpack(const gdr_ckpt8_unpack_args& a, hipStream_t s);

}  // namespace ckpt8
}  // namespace gdr
