// scan_tile.h -- the tile that the channelwise recurrence's kernels work on.
//
// A workgroup takes 64 channels of up to 8 waves x 32 tokens.  A thread holds 4
// neighbouring channels of 8 tokens: 16 lanes side by side cover the 64 channels,
// four lane groups the wave's 32 tokens.  So a wave is one 32-token block of the
// saved states, and one token row of the tile is a whole 128-byte line in bf16.
//
// The recurrence composes: a run of tokens takes h to P h + H with P the product
// of its decays.  Threads form (P, H) of their tokens from registers, lane groups
// and then waves are joined, and one wave carries the state from tile to tile:
// it waits for the tile before (`slot` of the chain, 64 words of a value and the
// number of tiles that it has passed), passes the state on and hands each wave
// its start state.  So every input is read once, and tiles of one chain overlap
// in all but that hand-over.  Tile numbers are drawn from a ticket, in which all
// chains' first tiles come before their second ones: a tile waits only for one
// whose workgroup has already started, so every wait ends; were it not to (a
// workspace in use elsewhere), it gives up after kSpinLimit polls with NaN.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "chan_device.h"
#include "scan_kernels.h"

namespace gdr {
namespace scan {

constexpr int kSpinLimit = 1 << 22;   // a poll takes about a microsecond

typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;
using rsrc_t = __amdgpu_buffer_rsrc_t;

struct Code8 {};   // element type of 8-bit checkpoint codes

template <typename T>
constexpr int size_of = sizeof(T);
template <>
inline constexpr int size_of<Code8> = 1;

// Buffer over `bytes` from `base`: loads past its end return zero and stores past
// it are dropped, which is how ragged ends of T and C are cut.
__device__ inline rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}
// Byte offset of lanes that have no channel: behind every buffer's end (a tile's
// rows are at most 2^28 bytes), also after a row offset is added.
constexpr int kNoLane = 0x40000000;

// Four neighbouring channels of a row: raw registers, and as fp32.  VEC: one
// access of all four (a row's channels are a multiple of 4: all are there, or none).
// Else one access each, of the `nv` that are there.
__device__ inline int at(int off, int k, int nv, int size) { return k < nv ? off + k * size : kNoLane; }

template <typename T>
struct Four;
template <>
struct Four<float> {
  using R = u32x4;
  template <bool VEC>
  static __device__ inline R load(rsrc_t b, int off, int nv) {
    if constexpr (VEC) return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0);
    R r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __builtin_amdgcn_raw_buffer_load_b32(b, at(off, k, nv, 4), 0, 0);
    return r;
  }
  static __device__ inline float get(const R& r, int k) { return __uint_as_float(r[k]); }
  template <bool VEC>
  static __device__ inline void store(rsrc_t b, int off, int nv, const float (&v)[4]) {
    R r;
#pragma unroll
    for (int k = 0; k < 4; ++k) r[k] = __float_as_uint(v[k]);
    if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b128(r, b, off, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) __builtin_amdgcn_raw_buffer_store_b32(r[k], b, at(off, k, nv, 4), 0, 0);
    }
  }
};
template <>
struct Four<__bf16> {
  using R = u32x2;
  template <bool VEC>
  static __device__ inline R load(rsrc_t b, int off, int nv) {
    if constexpr (VEC) return __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0);
    uint32_t h[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __builtin_amdgcn_raw_buffer_load_b16(b, at(off, k, nv, 2), 0, 0);
    return R{h[0] | h[1] << 16, h[2] | h[3] << 16};
  }
  static __device__ inline float get(const R& r, int k) {
    return __uint_as_float(k & 1 ? r[k >> 1] & 0xffff0000u : r[k >> 1] << 16);
  }
  template <bool VEC>
  static __device__ inline void store(rsrc_t b, int off, int nv, const float (&v)[4]) {
    if constexpr (VEC) {
      typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
      const bf16x4 h = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
      __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(R, h), b, off, 0, 0);
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v[k]), b, at(off, k, nv, 2), 0, 0);
    }
  }
};
template <>
struct Four<Code8> {
  using R = uint32_t;
  template <bool VEC>
  static __device__ inline R load(rsrc_t b, int off, int nv) {
    if constexpr (VEC) return __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0);
    R r = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      r |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(b, at(off, k, nv, 1), 0, 0) << (8 * k);
    return r;
  }
  static __device__ inline float get(const R& r, int k) {
    return k == 0 ? chan::code_f32<0>(r) : k == 1 ? chan::code_f32<1>(r) : k == 2 ? chan::code_f32<2>(r) : chan::code_f32<3>(r);
  }
};

// Hides where a register's value came from, so that what was computed from it is
// computed again and not kept.
template <typename R>
__device__ inline void forget(R& r) {
  asm volatile("" : "+v"(r));
}

constexpr int V = 4;                      // channels of a thread
constexpr int S = GDR_SCAN_BLOCK / V;     // its tokens
constexpr int kSide = kTileC / V;         // lanes side by side
constexpr int kGroups = 64 / kSide;       // lane groups of a wave
static_assert(kGroups * S == GDR_SCAN_BLOCK, "a wave covers one block of tokens");

// A thread's place in the launch and in its tile.
struct Place {
  int chain, tt;     // chain (batch row and channel tile), tile number along it
  int b, c0;         // batch row, first channel of the tile
  int lane, wave, nw;
  int grp, cl, c;    // lane group, the thread's first channel in the tile and in the row
  int nv;            // its channels that exist (4, or fewer; none: <= 0)
};

// The next tile in ticket order (or the workgroup's own, when no tile waits for
// another).  Contains barriers: every thread of the workgroup calls it.
__device__ inline Place take_place(int C, int nchain, int nct, uint32_t* ticket) {
  __shared__ uint32_t drawn;
  uint32_t tile = blockIdx.x;
  if (ticket) {
    if (threadIdx.x == 0) drawn = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    tile = drawn;
  }
  tile = __builtin_amdgcn_readfirstlane(tile);
  Place q;
  q.chain = tile % (uint32_t)nchain;
  q.tt = tile / (uint32_t)nchain;
  q.b = q.chain / nct;
  q.c0 = (q.chain % nct) * kTileC;
  q.lane = threadIdx.x & 63;
  q.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  q.nw = blockDim.x >> 6;
  q.grp = q.lane / kSide;
  q.cl = (q.lane % kSide) * V;
  q.c = q.c0 + q.cl;
  q.nv = C - q.c;
  return q;
}

// Join (P, H) over the wave's lane groups, earlier tokens in lower groups (UP)
// or in higher ones: on return P, H cover the thread's run and all before it,
// Pe, He all before it.
template <bool UP>
__device__ inline float from_group(float x, int dist) {
  return UP ? __shfl_up(x, dist * kSide) : __shfl_down(x, dist * kSide);
}
template <bool UP>
__device__ inline void join_groups(float (&P)[V], float (&H)[V], float (&Pe)[V], float (&He)[V], int grp) {
  const int pos = UP ? grp : kGroups - 1 - grp;   // place in the order of joining
#pragma unroll
  for (int dist = 1; dist < kGroups; dist *= 2) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float p = from_group<UP>(P[k], dist), h = from_group<UP>(H[k], dist);
      if (pos >= dist) {
        H[k] = fmaf(P[k], h, H[k]);
        P[k] *= p;
      }
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const float p = from_group<UP>(P[k], 1), h = from_group<UP>(H[k], 1);
    Pe[k] = pos > 0 ? p : 1.f;
    He[k] = pos > 0 ? h : 0.f;
  }
}

// The state that the tile before hands over, for channel `lane` of the chain.
__device__ inline float wait_for(const uint64_t* slot, int tt) {
  uint64_t w = 0;
  for (int n = 0; n < kSpinLimit; ++n) {
    w = __hip_atomic_load(slot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__all((int)(w >> 32) == tt)) return __uint_as_float((uint32_t)w);
    __builtin_amdgcn_s_sleep(1);
  }
  return __builtin_nanf("");
}
// Value and count in one 64-bit store: nothing else has to be ordered with it.
// The slot is free: only the tile that writes it now has waited for its last value.
__device__ inline void hand_over(uint64_t* slot, float h, int count) {
  __hip_atomic_store(slot, ((uint64_t)(uint32_t)count << 32) | __float_as_uint(h), __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace scan
}  // namespace gdr
