// scan_tile.h -- the tile that the channelwise recurrence's kernels work on.
//
// A workgroup takes 64 channels of up to 8 waves x 32 tokens.  A thread holds 4
// neighbouring channels of 8 tokens: 16 lanes side by side cover the 64 channels,
// four lane groups the wave's 32 tokens.  So a wave is one 32-token block of the
// saved states, and one token row of the tile is a whole 128-byte line in bf16.
//
// The recurrence composes: a run of tokens takes h to P h + H with P the product
// of its decays.  Threads form (P, H) of their tokens from registers, lane groups
// and then waves are joined.  Along the sequence, 8 tiles make a super: each tile
// publishes its own (P, H) as soon as it has it, which depends on nothing before
// it, and the last tile of a super publishes the state behind the super.  A tile's
// start state is the state before its super, taken through the maps of the tiles
// between.  So every input is read once, and one hand-over, a store that the next
// reader sees about a microsecond later, serves 8 tiles (with one per tile, a
// single sequence of 32785 tokens took 140 us, 128 hand-overs of about 1.05 us).
//
// Tile numbers are drawn from a ticket.  Chains are taken in teams, and a team's
// first tiles come before its second ones: a tile waits only for tiles whose
// workgroups have already started, and each publishes its map before it waits, so
// every wait ends.  Where the workspace is in use elsewhere, against the rules, the
// results are lost but nothing else is: a wait gives up after kSpinLimit polls with NaN,
// and a number that no tile has ends its workgroup.
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
typedef __attribute__((ext_vector_type(4))) float f32x4;
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

__device__ inline uint32_t bf16_pair(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}

// Four neighbouring channels of a row: raw registers, and as fp32.  `load` and
// `store` go through a buffer; `from` and `to` take the elements wherever they are
// (aligned to one of them), `some` of them where a row ends.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using R = u32x4;
  typedef u32x4 at4 __attribute__((aligned(4), may_alias));
  static __device__ inline R load(rsrc_t b, int off) { return __builtin_amdgcn_raw_buffer_load_b128(b, off, 0, 0); }
  static __device__ inline float get(const R& r, int k) { return __uint_as_float(r[k]); }
  static __device__ inline R pack(const float (&v)[4]) {
    return R{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  }
  static __device__ inline void store(rsrc_t b, int off, const R& r) { __builtin_amdgcn_raw_buffer_store_b128(r, b, off, 0, 0); }
  static __device__ inline R from(const char* p) { return *(const at4*)p; }
  static __device__ inline R some(const char* p, int n) {
    const uint32_t* e = (const uint32_t*)p;
    return R{n > 0 ? e[0] : 0u, n > 1 ? e[1] : 0u, n > 2 ? e[2] : 0u, 0u};
  }
  static __device__ inline void to(char* p, const R& r) { *(at4*)p = r; }
  static __device__ inline void to(char* p, const R& r, int k) { ((uint32_t*)p)[k] = r[k]; }
};
template <>
struct Four<__bf16> {
  using R = u32x2;
  typedef u32x2 at2 __attribute__((aligned(2), may_alias));
  static __device__ inline R load(rsrc_t b, int off) { return __builtin_amdgcn_raw_buffer_load_b64(b, off, 0, 0); }
  static __device__ inline float get(const R& r, int k) {
    return __uint_as_float(k & 1 ? r[k >> 1] & 0xffff0000u : r[k >> 1] << 16);
  }
  static __device__ inline R pack(const float (&v)[4]) { return R{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}; }
  static __device__ inline void store(rsrc_t b, int off, const R& r) { __builtin_amdgcn_raw_buffer_store_b64(r, b, off, 0, 0); }
  static __device__ inline R from(const char* p) { return *(const at2*)p; }
  static __device__ inline R some(const char* p, int n) {
    const uint16_t* e = (const uint16_t*)p;
    const uint32_t e0 = n > 0 ? e[0] : 0u, e1 = n > 1 ? e[1] : 0u, e2 = n > 2 ? e[2] : 0u;
    return R{e0 | e1 << 16, e2};
  }
  static __device__ inline void to(char* p, const R& r) { *(at2*)p = r; }
  static __device__ inline void to(char* p, const R& r, int k) { ((uint16_t*)p)[k] = (uint16_t)(r[k >> 1] >> (16 * (k & 1))); }
};
template <>
struct Four<Code8> {
  using R = uint32_t;
  typedef uint32_t at1 __attribute__((aligned(1), may_alias));
  static __device__ inline R load(rsrc_t b, int off) { return __builtin_amdgcn_raw_buffer_load_b32(b, off, 0, 0); }
  static __device__ inline float get(const R& r, int k) {
    return k == 0 ? chan::code_f32<0>(r) : k == 1 ? chan::code_f32<1>(r) : k == 2 ? chan::code_f32<2>(r) : chan::code_f32<3>(r);
  }
  static __device__ inline R from(const char* p) { return *(const at1*)p; }
  static __device__ inline R some(const char* p, int n) {
    const uint8_t* e = (const uint8_t*)p;
    return (n > 0 ? e[0] : 0u) | (n > 1 ? (uint32_t)e[1] << 8 : 0u) | (n > 2 ? (uint32_t)e[2] << 16 : 0u);
  }
};

// A thread's rows of one of the call's arrays, from the tile's first element on.
// VEC (rows of a multiple of 4 channels, in buffers aligned to 4 elements): through a
// buffer that ends with the tile's rows.  Else with a test of what exists: four
// channels at once wherever they lie, one by one at a row's end (4 x 2048 x 2047 bf16,
// gated: forward 62 us, backward 98; one access for each channel took 71 and 145).
template <typename T, bool VEC>
struct View {
  rsrc_t b;
  int off;
  char* p;
  int nv, mine, step;
  __device__ inline View(const void* array, size_t base, int rows, int C, int r0, int c, int nv_) {
    step = C * size_of<T>;
    const int first = r0 * step + c * size_of<T>;
    char* tile = (char*)const_cast<void*>(array) + base * size_of<T>;
    if constexpr (VEC) {
      b = buffer(tile, rows * step);
      off = nv_ > 0 ? first : kNoLane;
    } else {
      p = tile + first;
      nv = nv_;
      mine = rows - r0;
    }
  }
  __device__ inline typename Four<T>::R load(int i) const {
    if constexpr (VEC) {
      return Four<T>::load(b, off + i * step);
    } else {
      typename Four<T>::R r = {};
      if (i < mine) {
        if (nv >= 4) r = Four<T>::from(p + i * step);
        else if (nv > 0) r = Four<T>::some(p + i * step, nv);
      }
      return r;
    }
  }
  __device__ inline void store(int i, const float (&v)[4]) const {
    const typename Four<T>::R r = Four<T>::pack(v);
    if constexpr (VEC) {
      Four<T>::store(b, off + i * step, r);
    } else if (i < mine) {
      if (nv >= 4) {
        Four<T>::to(p + i * step, r);
      } else {
#pragma unroll
        for (int k = 0; k < 3; ++k)
          if (k < nv) Four<T>::to(p + i * step, r, k);
      }
    }
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
// another); chain -1: none.  Contains barriers: every thread of the workgroup calls it.
__device__ inline Place take_place(int C, int nchain, int nct, int nt, int team_size, uint32_t* ticket) {
  __shared__ uint32_t drawn;
  uint32_t tile = blockIdx.x;
  if (ticket) {
    if (threadIdx.x == 0) drawn = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    tile = drawn;
  }
  tile = __builtin_amdgcn_readfirstlane(tile);
  const Turn turn = turn_of(tile, nchain, nt, team_size);
  Place q;
  q.tt = turn.tt;
  q.chain = turn.chain;
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

// (P, H) of one run after another.
__device__ inline float2 after(float2 later, float2 earlier) {
  return float2{later.x * earlier.x, fmaf(later.x, earlier.y, later.y)};
}
// Join (P, H) over the wave's four lane groups, which are its rows of 16 lanes,
// earlier tokens in lower rows (UP) or in higher ones: on return P, H cover the
// whole wave, Pe, He all before the thread's run.  The lane swaps (VALU, no LDS)
// give every row the values of its pair's even and odd row, and every half those of
// both halves.
template <bool UP>
__device__ inline void join_groups(float (&P)[V], float (&H)[V], float (&Pe)[V], float (&He)[V], int grp) {
  const bool second = (grp & 1) == (UP ? 1 : 0), behind = (grp >> 1) == (UP ? 1 : 0);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(P[k]), __float_as_uint(P[k]), false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(H[k]), __float_as_uint(H[k]), false, false);
    const float2 even = {__uint_as_float(p[0]), __uint_as_float(h[0])}, odd = {__uint_as_float(p[1]), __uint_as_float(h[1])};
    const float2 a = UP ? even : odd, pair = after(UP ? odd : even, a);
    const auto pp = __builtin_amdgcn_permlane32_swap(__float_as_uint(pair.x), __float_as_uint(pair.x), false, false);
    const auto hh = __builtin_amdgcn_permlane32_swap(__float_as_uint(pair.y), __float_as_uint(pair.y), false, false);
    const float2 low = {__uint_as_float(pp[0]), __uint_as_float(hh[0])}, high = {__uint_as_float(pp[1]), __uint_as_float(hh[1])};
    const float2 b = UP ? low : high, all = after(UP ? high : low, b);
    float2 ex = second ? a : float2{1.f, 0.f};
    if (behind) ex = after(ex, b);
    P[k] = all.x;
    H[k] = all.y;
    Pe[k] = ex.x;
    He[k] = ex.y;
  }
}

// A tile's map for one channel as one word, so that nothing else has to be ordered
// with its store; P is kept inverted, and 0 (an all-ones NaN, which is not stored)
// means that the word has not been written.
__device__ inline void put_map(uint64_t* word, float2 r) {
  const uint32_t p = r.x != r.x ? 0x7fc00000u : __float_as_uint(r.x);
  __hip_atomic_store(word, ((uint64_t)__float_as_uint(r.y) << 32) | (uint32_t)~p, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
// A state as one word: the value, and 1 where it has been written.
__device__ inline void put_state(uint64_t* word, float h) {
  __hip_atomic_store(word, ((uint64_t)__float_as_uint(h) << 32) | 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline uint64_t look(const uint64_t* word) {
  return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// The wave's 64 words once all are written (0 after kSpinLimit polls); w is what
// the lane saw at its first look.
__device__ inline uint64_t wait_words(const uint64_t* word, uint64_t w) {
  for (int n = 0; n < kSpinLimit; ++n) {
    if (__all((uint32_t)w != 0u)) return w;
    __builtin_amdgcn_s_sleep(1);
    w = look(word);
  }
  return 0;
}
__device__ inline float2 get_map(const uint64_t* word, uint64_t seen) {
  const uint64_t w = wait_words(word, seen);
  if ((uint32_t)w == 0u) return float2{__builtin_nanf(""), __builtin_nanf("")};
  return float2{__uint_as_float(~(uint32_t)w), __uint_as_float((uint32_t)(w >> 32))};
}
__device__ inline float get_state(const uint64_t* word, uint64_t seen) {
  const uint64_t w = wait_words(word, seen);
  return (uint32_t)w == 0u ? __builtin_nanf("") : __uint_as_float((uint32_t)(w >> 32));
}

// LDS of the joins between waves and tiles.
template <int NW>
struct Joins {
  float2 run[NW][kTileC];        // (P, H) of each wave, in the order of joining
  float2 pre[kSuper - 1][kTileC];   // of the tiles before this one in its super
  float start[kTileC];           // the state before the chain, then the tile
  float from[NW][kTileC];        // and before each wave
};

// A tile's words, and a first look at those it will need, taken when its inputs are
// asked for: where tiles outnumber the workgroups that run at once, the tiles
// before are long done and nothing is waited for later.
template <int NW>
struct Words {
  static constexpr int kMaps = (kSuper - 1 + NW - 1) / NW;   // maps that a wave fetches
  uint64_t *tile, *super;
  uint64_t map[kMaps], state;
};
template <int NW>
__device__ inline Words<NW> look_ahead(const Chains& ch, const Place& q, int nt, int pos) {
  Words<NW> w;
  if (!ch.ticket) return w;
  const int r = q.tt % kSuper, su = q.tt / kSuper, ns = (nt + kSuper - 1) / kSuper;
  w.tile = ch.tiles + ((size_t)q.chain * nt + q.tt) * kTileC + q.lane;
  w.super = ch.supers + ((size_t)q.chain * ns + su) * kTileC + q.lane;
#pragma unroll
  for (int i = 0; i < Words<NW>::kMaps; ++i) {
    const int k = q.wave + i * NW;
    w.map[i] = k < r ? look(w.tile - (size_t)(r - k) * kTileC) : 0u;
  }
  w.state = pos == NW - 1 && su > 0 ? look(w.super) : 0u;
  return w;
}

// From the waves' maps (j.run, written before the call) to the state before each
// wave, for channel `lane` (returned) and in j.from for the wave's own threads.
// `pos` is the wave's place in the order of joining, `first` the state before the
// chain (in the last wave in order), `last` receives the state behind the
// tile in that wave.  Every thread of the workgroup calls it.
//
// The chain's last tile may write its final state over the start state (h_out = h0), once
// it has the maps of the tiles before it.  So `first` goes to LDS ahead of the barrier
// that the map's publication follows: a load of it is complete by then, in whichever
// wave it is.
template <int NW>
__device__ inline float join_tiles(Joins<NW>& j, const Chains& ch, const Place& q, const Words<NW>& words, int nt,
                                   int pos, float first, float& last) {
  const int lane = q.lane, r = q.tt % kSuper, su = q.tt / kSuper;
  if (pos == q.nw - 1) j.start[lane] = first;
  __syncthreads();
  if (ch.ticket) {
    if (q.wave == 0 && r < kSuper - 1 && q.tt + 1 < nt) {
      float2 m = {1.f, 0.f};
#pragma unroll
      for (int w = 0; w < NW; ++w) m = after(j.run[w][lane], m);
      put_map(words.tile, m);
    }
#pragma unroll
    for (int i = 0; i < Words<NW>::kMaps; ++i) {
      const int k = q.wave + i * NW;
      if (k < r) j.pre[k][lane] = get_map(words.tile - (size_t)(r - k) * kTileC, words.map[i]);
    }
    if (r > 0) __syncthreads();
  }
  if (pos == q.nw - 1) {
    float2 before = {1.f, 0.f}, own = {1.f, 0.f};
#pragma unroll
    for (int k = 0; k < kSuper - 1; ++k)
      if (k < r) before = after(j.pre[k][lane], before);
#pragma unroll
    for (int w = 0; w < NW; ++w)
      if (w < q.nw) own = after(j.run[w][lane], own);
    const float in = su > 0 ? get_state(words.super, words.state) : j.start[lane];
    const float h = fmaf(before.x, in, before.y);
    last = fmaf(own.x, h, own.y);
    if (r == kSuper - 1 && q.tt + 1 < nt) put_state(words.super + kTileC, last);
    j.start[lane] = h;
  }
  __syncthreads();
  float h = j.start[lane];
#pragma unroll
  for (int w = 0; w < NW; ++w)
    if (w < pos) {
      const float2 a = j.run[w][lane];
      h = fmaf(a.x, h, a.y);
    }
  j.from[pos][lane] = h;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // read by the same wave's lanes
  __builtin_amdgcn_wave_barrier();
  return h;
}

}  // namespace scan
}  // namespace gdr
