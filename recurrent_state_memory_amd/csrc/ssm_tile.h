// ssm_tile.h -- what the selective scan's kernels share: how its work is laid over
// workgroups, the vectors B_t and C_t as the kernels read them, the time step, sums over
// a wave's channels.
//
// A workgroup has 64 channels of one group, one a lane, and a batch row's tokens or a
// segment of them; its NW waves share the states: wave w has states w NS ... w NS + NS - 1.
// So a token's B_t and C_t are the same for a whole wave, which takes them from scalar
// registers, and the sum over a channel's states stays within a lane and a few waves.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "chan_device.h"
#include "scan_gate.h"
#include "ssm_kernels.h"

namespace gdr {
namespace ssm {

constexpr int kBlock = GDR_SSM_BLOCK;

struct Geo {
  int B, T, C, N, G;
  int each, nb;     // channels of a group, workgroups of them
  int pairs;        // pairs of states that the vectors are laid out for
  int Tp;           // T up to a whole block
  int segs, seg;    // segments of the tokens and their length, a multiple of kBlock
  __host__ __device__ unsigned blocks() const { return (unsigned)B * G * nb * segs; }
};

// Waves and states a wave (NS); waves beyond 8 or more than 8 states a wave serve no N.
constexpr int waves_of(int N) { return N <= 8 ? 4 : 8; }
constexpr int states_of(int N) { return N <= 16 ? 2 : N <= 32 ? 4 : 8; }

inline Geo geo_of(int B, int T, int C, int N, int G) {
  Geo q;
  q.B = B, q.T = T, q.C = C, q.N = N, q.G = G;
  q.each = C / G;
  q.nb = lanes_of_group(C, G);
  q.pairs = waves_of(N) * states_of(N) / 2;
  q.Tp = (int)blocks_of(T) * kBlock;
  q.segs = 1;
  q.seg = q.Tp;
  return q;
}

// Where a workgroup and its lanes are.
struct Place {
  int b, g, cb, seg, c;   // batch row, group, block of channels (of all groups), segment, channel
  bool on;                // whether the lane has a channel (else c is the group's last)
};
__device__ inline Place place_of(const Geo& q) {
  Place s;
  const unsigned across = (unsigned)q.G * q.nb, rest = blockIdx.x / across;
  s.cb = (int)(blockIdx.x - rest * across);
  s.seg = (int)(rest / q.B);
  s.b = (int)(rest - (unsigned)s.seg * q.B);
  s.g = s.cb / q.nb;
  const int l = (s.cb - s.g * q.nb) * kLanes + (threadIdx.x & 63);
  s.on = l < q.each;
  s.c = s.g * q.each + (s.on ? l : q.each - 1);
  return s;
}

__device__ inline int row_len(const int32_t* lens, int b, int T) {
  if (!lens) return T;
  const int n = lens[b];
  return n < 0 ? 0 : n < T ? n : T;
}

// B_t and C_t in fp32, laid out [B][G][pairs][Tp] as {B 2p, B 2p+1, C 2p, C 2p+1}, 0 where
// there is no state or no token of the row: 16 aligned bytes that a wave loads into scalar registers.
typedef float f4 __attribute__((ext_vector_type(4)));
typedef const __attribute__((address_space(4))) f4* Vectors;
__device__ inline Vectors vectors_at(const float* v, const Geo& q, int b, int g, int pair) {
  return (Vectors)(uintptr_t)(v + (((size_t)b * q.G + g) * q.pairs + pair) * q.Tp * 4);
}

// d = softplus(pre) or pre.
__device__ inline float time_step(float pre, bool softplus) { return softplus ? scan::softplus(pre) : pre; }

// Bytes of the parts of a workspace, each a multiple of 256.
inline size_t pad256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t vector_bytes(const Geo& q) { return pad256((size_t)q.B * q.G * q.pairs * q.Tp * 16); }
inline size_t ends_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.N * q.C * 4) : 0; }
inline size_t sums_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.C * 4) : 0; }

// Launches shared by the forward and the backward (ssm_fwd.hip).
hipError_t launch_vectors(int io_dtype, const void* Bv, const void* Cv, const int32_t* lens, const Geo& q, float* out,
                          hipStream_t s);
// The recurrence from h0 with a.y (NULL: only its states), the vectors already laid out.
hipError_t launch_states(const gdr_ssm_args& a, const Geo& q, const float* vec, float* ends, float* sums, hipStream_t s);

}  // namespace ssm
}  // namespace gdr
