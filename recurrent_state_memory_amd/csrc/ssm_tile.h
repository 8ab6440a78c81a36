// ssm_tile.h -- what the selective scan's kernels share: how its work is laid over
// workgroups, the vectors B_t and C_t as the kernels read them, the time step, sums over
// a wave's channels.
//
// A workgroup has 64 channels of one group, one a lane, and a batch row's tokens or a
// segment of them; its NW waves share the states: wave w has states w NS ... w NS + NS - 1.
// So a token's B_t and C_t are the same for a whole wave, and the sum over a channel's
// states stays within a lane and a few waves.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "chan_device.h"
#include "scan_gate.h"
#include "ssm_kernels.h"

namespace gdr {
namespace ssm {

constexpr int kBlock = GDR_SSM_BLOCK;

struct Geo {
  int B, T, C, N, G;
  int each, nb;     // channels of a group, workgroups of them
  int pairs;        // pairs of states that the waves have room for
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
  // Segments: where the chains of channels are fewer than half the CUs, up to two
  // workgroups a CU, of 64 tokens at least.
  const long long chains = chains_of(B, C, G);
  long long want = chains <= 128 && T >= 256 ? 512 / chains : 1;
  if (want > T / 64) want = T / 64;
  if (want < 1) want = 1;
  q.seg = (int)((blocks_of(T) + want - 1) / want) * kBlock;
  q.segs = (q.Tp + q.seg - 1) / q.seg;
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

// A loop whose index is a constant to its body.
template <int... I, typename F>
__device__ inline void each_of(std::integer_sequence<int, I...>, F f) {
  (f(std::integral_constant<int, I>()), ...);
}
template <int N, typename F>
__device__ inline void each(F f) {
  each_of(std::make_integer_sequence<int, N>(), f);
}

// B_t and C_t of a wave's states.  Each row of 16 lanes holds those of four tokens for one
// pair of states, lane 4 (t % 4) + k the k-th of {B 2p, B 2p+1, C 2p, C 2p+1}, and the
// arithmetic takes them from there by DPP (row_newbcast), at no instruction of its own.
// (From scalar registers: every scalar load misses its cache, as 64 bytes are four tokens, and
// returns out of order, so each wait is for the last one: 403 us in place of @@ on 8 x 4096
// x 2048 with 16 states.)
template <int K>
__device__ inline float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + K, 0xf, 0xf, true));
}
template <typename T, int NS, int TILE>
struct Vectors {
  static constexpr int P = NS / 2, Q = TILE / 4;
  struct Raw {
    T v[P][Q];
  };
  const T* at[P];     // the lane's element of tokens 0 to 3
  size_t step;        // elements between tokens
  int tk;             // the lane's token of four
  bool ok[P];         // whether the state exists
  bool all;           // whether all of the wave's do
  // of pairs first, first + 1, ... (state 2 first + 2 i)
  __device__ inline Vectors(const T* Bv, const T* Cv, const Geo& q, const Place& s, int first) {
    const int j = threadIdx.x & 15;
    tk = j >> 2;
    step = (size_t)q.G * q.N;
    all = 2 * (first + P) <= q.N;
    const T* base = ((j & 2) ? Cv : Bv) + ((size_t)s.b * q.T * q.G + s.g) * q.N + (size_t)tk * step;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int n = 2 * (first + i) + (j & 1);
      ok[i] = n < q.N;
      at[i] = base + (ok[i] ? n : 0);
    }
  }
  // Tokens t ... t + TILE - 1; behind the last one (end - 1) that one once more.
  __device__ inline void load(int t, int end, Raw& r) const {
    if (t + TILE <= end) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < Q; ++k) r.v[i][k] = at[i][(size_t)(t + 4 * k) * step];
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < Q; ++k) r.v[i][k] = at[i][(ptrdiff_t)(min(t + 4 * k + tk, end - 1) - tk) * (ptrdiff_t)step];
    }
  }
  // In fp32, 0 where there is no state or token.
  __device__ inline void take(int t, int end, const Raw& r, float (&v)[P][Q]) const {
    if (all && t + TILE <= end) {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < Q; ++k) v[i][k] = (float)r.v[i][k];
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int k = 0; k < Q; ++k) v[i][k] = ok[i] && t + 4 * k + tk < end ? (float)r.v[i][k] : 0.f;
    }
  }
};

// A lane's byte offset into a row that begins at a scalar address.  The compiler would
// add it to every row's base and keep the sums in vector registers, with 64-bit vector
// additions for each access; so it is told nothing about its value.
__device__ inline unsigned lane_offset(unsigned bytes) {
  asm volatile("" : "+v"(bytes));
  return bytes;
}
template <typename T>
__device__ inline const T& at_offset(const T* row, unsigned bytes) {
  return *(const T*)((const char*)row + bytes);
}
template <typename T>
__device__ inline T& at_offset(T* row, unsigned bytes) {
  return *(T*)((char*)row + bytes);
}

// d = softplus(pre) or pre.
__device__ inline float time_step(float pre, bool softplus) { return softplus ? scan::softplus(pre) : pre; }

// Bytes of the parts of a workspace, each a multiple of 256.
inline size_t pad256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t ends_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.N * q.C * 4) : 0; }
inline size_t sums_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.C * 4) : 0; }

// The recurrence from h0 with a.y (NULL: only its states) (ssm_fwd.hip).
hipError_t launch_states(const gdr_ssm_args& a, const Geo& q, float* ends, float* sums, hipStream_t s);

}  // namespace ssm
}  // namespace gdr
