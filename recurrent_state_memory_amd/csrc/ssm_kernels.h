// ssm_kernels.h -- launch interface of the selective state space scan.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/gdr_ssm.h"

namespace gdr {
namespace ssm {

constexpr int kLanes = 64;      // channels of a workgroup, one a lane
constexpr int kMaxN = 64;

constexpr size_t blocks_of(int T) { return ((size_t)T + GDR_SSM_BLOCK - 1) / GDR_SSM_BLOCK; }
constexpr int lanes_of_group(int C, int G) { return (C / G + kLanes - 1) / kLanes; }   // workgroups of a group's channels
constexpr long long chains_of(int B, int C, int G) { return (long long)B * G * lanes_of_group(C, G); }
constexpr bool too_many_chains(int B, int C, int G) { return chains_of(B, C, G) >= (1LL << 22); }

size_t fwd_workspace(int B, int T, int C, int N, int G);
size_t bwd_workspace(int B, int T, int C, int N, int G, bool ckpt);

// Arguments already checked; a.workspace large enough.
hipError_t launch_ssm_fwd(const gdr_ssm_args& a, hipStream_t s);
hipError_t launch_ssm_bwd(const gdr_ssm_bwd_args& a, hipStream_t s);
hipError_t launch_ssm_step(const gdr_ssm_step_args& a, hipStream_t s);

}  // namespace ssm
}  // namespace gdr
