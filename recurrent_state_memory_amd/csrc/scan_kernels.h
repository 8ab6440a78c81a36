// scan_kernels.h -- launch interface of the channelwise recurrence.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_scan.h"

namespace gdr {
namespace scan {

constexpr size_t blocks_of(int T) { return ((size_t)T + GDR_SCAN_BLOCK - 1) / GDR_SCAN_BLOCK; }

// Workspace of the forward and of the backward (bytes; 0: none needed).
size_t fwd_workspace(int B, int T, int C);
size_t bwd_workspace(int B, int T, int C, bool gated, bool ckpt);

// Arguments already checked; a.workspace large enough.
hipError_t launch_scan_fwd(const gdr_scan_args& a, hipStream_t s);
hipError_t launch_scan_bwd(const gdr_scan_bwd_args& a, hipStream_t s);
hipError_t launch_scan_step(const gdr_scan_step_args& a, hipStream_t s);

}  // namespace scan
}  // namespace gdr
