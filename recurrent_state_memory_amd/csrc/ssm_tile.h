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
constexpr float kRate = 0x1p64f;   // decay rates are held to +-kRate

struct Geo {
  int B, T, C, N, G;
  int each, nb;     // channels of a group, workgroups of them
  int room;         // states that the backward's waves write partial sums of
  int Tp;           // T up to a whole block
  int segs, seg;    // segments of the tokens and their length, a multiple of kBlock
  __host__ __device__ unsigned blocks() const { return (unsigned)B * G * nb * segs; }
};

constexpr int kWaves = 8;   // of a workgroup

// The forward's and the backward's.
inline Geo geo_of(int B, int T, int C, int N, int G, bool backward) {
  Geo q;
  q.B = B, q.T = T, q.C = C, q.N = N, q.G = G;
  q.each = C / G;
  q.nb = lanes_of_group(C, G);
  // waves of one state or two; those without one write nothing, but for 9 to 16 states
  q.room = N <= 8 ? N : N <= 16 ? 16 : N + N % 2;
  q.Tp = (int)blocks_of(T) * kBlock;
  // Segments.  Forward: where the chains of channels are no more than half the CUs, two
  // workgroups a CU of 64 tokens at least (a second one a CU fills the first one's waits):
  // 128 chains of 2048 tokens in 4 segments 127 us, 256 in one 171; 32 of 256 tokens in 4
  // segments 18 us, of 255 in one 24.
  // Backward: one fits a CU, so the number of segments that leaves the fewest rounds of
  // whole rows, with a fifth of the time of a round for the adjoint's first pass over all
  // rows but the last segments'.
  const long long chains = chains_of(B, C, G);
  long long want = 1;
  if (!backward) {
    if (chains <= 128 && T >= 256) want = 512 / chains < T / 64 ? 512 / chains : T / 64;
    if (want > 128) want = 128;
  } else {
    double best = 0;
    for (int n = 1; n <= 128 && n * kBlock <= T; n = n < 16 ? n + 1 : n * 2) {
      const double cost = ((chains * n + 255) / 256 + 0.2 * ((double)chains / 256) * (n - 1)) / n;
      if (n == 1 || cost < 0.97 * best) best = cost, want = n;
    }
  }
  // and a segment's rows, and some behind it, stay within a buffer descriptor's 2^31 bytes
  const long long wide = (long long)(C > G * N ? C : G * N) * 4, most = ((1LL << 31) / wide - 128) / kBlock;
  const long long least = ((long long)blocks_of(T) + most - 1) / most;
  if (want < least) want = least;
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

// A segment's rows of an activation through a buffer descriptor: its base is a scalar, a
// lane's place in it a 32-bit offset (so no 64-bit arithmetic), reads behind its end give 0
// and writes there are dropped (so no masks at a row's end or for lanes without a channel,
// whose offset is kNowhere).  Offsets behind the end stay below 2^31 as well (geo_of).
typedef __amdgpu_buffer_rsrc_t Buffer;
constexpr unsigned kNowhere = 0x80000000u;
__device__ inline Buffer buffer_at(const void* p, size_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00027000);
}
template <typename T>
struct Io;
template <>
struct Io<float> {
  typedef uint32_t Raw;
  static __device__ inline Raw load(Buffer b, unsigned at) { return __builtin_amdgcn_raw_buffer_load_b32(b, at, 0, 0); }
  static __device__ inline float get(Raw r) { return __uint_as_float(r); }
  static __device__ inline void store(Buffer b, unsigned at, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), b, at, 0, 0);
  }
};
template <>
struct Io<__bf16> {
  typedef uint16_t Raw;
  static __device__ inline Raw load(Buffer b, unsigned at) { return __builtin_amdgcn_raw_buffer_load_b16(b, at, 0, 0); }
  static __device__ inline float get(Raw r) { return __uint_as_float((uint32_t)r << 16); }
  static __device__ inline void store(Buffer b, unsigned at, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), b, at, 0, 0);
  }
};
// Rows t to end - 1 (none: an empty buffer) of batch row b of a [B][T][C] array.
template <typename T>
__device__ inline Buffer rows_at(const void* base, const Geo& q, int b, int t, int end) {
  return buffer_at((const T*)base + ((size_t)b * q.T + t) * q.C, t < end ? (size_t)(end - t) * q.C * sizeof(T) : 0);
}

// B_t and C_t of a wave's states, two registers for eight tokens and a pair of states (or
// sixteen tokens and the wave's only state): each row of 16 lanes holds B's (C's) of both
// states for the eight, lane 2 (t % 8) + i, and the arithmetic takes them from there by DPP
// (row_newbcast), mostly at no instruction of its own.  (From scalar registers: every scalar
// load misses its cache, as 64 bytes are four tokens, and returns out of order, so that each
// wait is for the last one.)
template <int K>
__device__ inline float row_lane(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x150 + K, 0xf, 0xf, true));
}
// Sums of products with row lanes.  The compiler takes a DPP operand into a multiplication
// but not into a multiply-add (it moves it first), so these are written out; a register read
// by DPP must not be one that either of the two instructions before wrote, hence the s_nop.
// acc_u = c_0 h0_u + c_1 h1_u (MORE: added to acc_u) for four tokens, whose c_0, c_1 are the
// row lanes L + 2 u and L + 2 u + 1 of cv.
#define GDR_DPP(OP, DST, SRC, K, B) OP " " DST ", " SRC ", " B " row_newbcast:" K " row_mask:0xf bank_mask:0xf\n\t"
template <int L, bool MORE>
__device__ inline void row_dots(float cv, float h00, float h01, float h02, float h03, float h10, float h11, float h12, float h13,
                                float (&acc)[4]) {
  if constexpr (MORE)
    asm("s_nop 1\n\t" GDR_DPP("v_fmac_f32_dpp", "%0", "%4", "%13", "%5") GDR_DPP("v_fmac_f32_dpp", "%1", "%4", "%15", "%6")
            GDR_DPP("v_fmac_f32_dpp", "%2", "%4", "%17", "%7") GDR_DPP("v_fmac_f32_dpp", "%3", "%4", "%19", "%8")
                GDR_DPP("v_fmac_f32_dpp", "%0", "%4", "%14", "%9") GDR_DPP("v_fmac_f32_dpp", "%1", "%4", "%16", "%10")
                    GDR_DPP("v_fmac_f32_dpp", "%2", "%4", "%18", "%11") GDR_DPP("v_fmac_f32_dpp", "%3", "%4", "%20", "%12")
        : "+&v"(acc[0]), "+&v"(acc[1]), "+&v"(acc[2]), "+&v"(acc[3])
        : "v"(cv), "v"(h00), "v"(h01), "v"(h02), "v"(h03), "v"(h10), "v"(h11), "v"(h12), "v"(h13), "n"(L), "n"(L + 1),
          "n"(L + 2), "n"(L + 3), "n"(L + 4), "n"(L + 5), "n"(L + 6), "n"(L + 7));
  else
    asm("s_nop 1\n\t" GDR_DPP("v_mul_f32_dpp", "%0", "%4", "%13", "%5") GDR_DPP("v_mul_f32_dpp", "%1", "%4", "%15", "%6")
            GDR_DPP("v_mul_f32_dpp", "%2", "%4", "%17", "%7") GDR_DPP("v_mul_f32_dpp", "%3", "%4", "%19", "%8")
                GDR_DPP("v_fmac_f32_dpp", "%0", "%4", "%14", "%9") GDR_DPP("v_fmac_f32_dpp", "%1", "%4", "%16", "%10")
                    GDR_DPP("v_fmac_f32_dpp", "%2", "%4", "%18", "%11") GDR_DPP("v_fmac_f32_dpp", "%3", "%4", "%20", "%12")
        : "=&v"(acc[0]), "=&v"(acc[1]), "=&v"(acc[2]), "=&v"(acc[3])
        : "v"(cv), "v"(h00), "v"(h01), "v"(h02), "v"(h03), "v"(h10), "v"(h11), "v"(h12), "v"(h13), "n"(L), "n"(L + 1),
          "n"(L + 2), "n"(L + 3), "n"(L + 4), "n"(L + 5), "n"(L + 6), "n"(L + 7));
}
// K0, K1 += c_0 g, c_1 g; returns b_0 K0 + b_1 K1 (row lanes L, L + 1 of cv and bv).
template <int L>
__device__ inline float row_adjoint(float cv, float bv, float g, float& K0, float& K1) {
  float p;
  asm("s_nop 1\n\t" GDR_DPP("v_fmac_f32_dpp", "%0", "%3", "%6", "%5") GDR_DPP("v_fmac_f32_dpp", "%1", "%3", "%7", "%5")
          GDR_DPP("v_mul_f32_dpp", "%2", "%4", "%6", "%0") GDR_DPP("v_fmac_f32_dpp", "%2", "%4", "%7", "%1")
      : "+&v"(K0), "+&v"(K1), "=&v"(p)
      : "v"(cv), "v"(bv), "v"(g), "n"(L), "n"(L + 1));
  return p;
}
#undef GDR_DPP

template <typename T, int NS, int TILE>
struct Vectors {
  static constexpr int W = NS > 1 ? 2 : 1, P = NS / W, M = 16 / W, Q = TILE / M;   // M tokens a register
  struct Raw {
    typename Io<T>::Raw b[P][Q], c[P][Q];
  };
  struct Set {
    float b[P][Q], c[P][Q];
  };
  Buffer Bv, Cv;      // of tokens t0 to end - 1; the last one's row ends with its group's vector
  unsigned step;      // bytes between tokens
  unsigned at[P];     // the lane's offset behind a multiple of M tokens
  // of states first ... first + NS - 1
  __device__ inline Vectors(const void* b, const void* c, const Geo& q, const Place& s, int t0, int end, int first) {
    const size_t row = (size_t)q.G * q.N, base = (((size_t)s.b * q.T + t0) * q.G + s.g) * q.N;
    const size_t bytes = t0 < end ? ((size_t)(end - 1 - t0) * row + q.N) * sizeof(T) : 0;
    step = (unsigned)(row * sizeof(T));
    Bv = buffer_at((const T*)b + base, bytes);
    Cv = buffer_at((const T*)c + base, bytes);
    states(q, first);
  }
  __device__ inline void states(const Geo& q, int first) {
    const int j = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int n = first + W * i + j % W;
      at[i] = n < q.N ? j / W * step + n * (unsigned)sizeof(T) : kNowhere;
    }
  }
  // Tokens t ... t + TILE - 1 (counted from t0), zeros behind the last one and where there
  // is no state.
  __device__ inline void load(int t, Raw& r) const {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const unsigned o = at[i] + (unsigned)(t + M * k) * step;
        r.b[i][k] = Io<T>::load(Bv, o);
        r.c[i][k] = Io<T>::load(Cv, o);
      }
  }
  // Between two passes over the same vectors: else the compiler keeps the first one's lane
  // reads in registers of their own for the second.
  static __device__ inline void forget(Set& v) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int k = 0; k < Q; ++k) asm volatile("" : "+v"(v.b[i][k]), "+v"(v.c[i][k]));
  }
  static __device__ inline void take(const Raw& r, Set& v) {
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int k = 0; k < Q; ++k) v.b[i][k] = Io<T>::get(r.b[i][k]), v.c[i][k] = Io<T>::get(r.c[i][k]);
  }
};

// d = softplus(pre) or pre.
__device__ inline float time_step(float pre, bool softplus) { return softplus ? scan::softplus(pre) : pre; }

// A rate as the kernels use it (a NaN stays one).  Behind a row's end the time step is 0 and
// the slope of softplus too, and neither 0 A log2 e nor 0 A h H may be 0 times an Inf.
__device__ inline float held(float A) { return __builtin_fabsf(A) > kRate ? __builtin_copysignf(kRate, A) : A; }

// A state (an adjoint) taken through the segments from, from + dir, ... (to excluded): of
// each one its end and the sum of its time steps.  Several are asked for at once, else
// each would cost a load's latency.
template <int NS>
__device__ inline void pass_segments(const Geo& q, const Place& s, int first, int from, int to, int dir,
                                     const float (&A2)[NS], const float* ends, const float* sums, float (&h)[NS]) {
  constexpr int KB = NS <= 2 ? 8 : 2;
  for (int k0 = from; k0 != to;) {
    float e[KB][NS], d[KB];
    const int left = (to - k0) * dir, n = left < KB ? left : KB;
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      const size_t at = (size_t)s.b * q.segs + (k0 + (j < n ? j : 0) * dir);
      d[j] = sums[at * q.C + s.c];
#pragma unroll
      for (int i = 0; i < NS; ++i) e[j][i] = first + i < q.N ? ends[(at * q.N + first + i) * q.C + s.c] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < KB; ++j) {
      if (j < n) {
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          // The factor's root, twice, and finite: a growing segment's may pass fp32 where what
          // it multiplies is 0 or small.  Without decay, or where the steps sum to 0 (behind
          // a row's end), it is 1 whatever the other one is; a NaN stays one.
          const float half = A2[i] == 0.f || d[j] == 0.f ? 0.f : 0.5f * A2[i] * d[j];
          const float root = __builtin_amdgcn_exp2f(half > 127.f ? 127.f : half);
          h[i] = fmaf(root, root * h[i], e[j][i]);
        }
      }
    }
    k0 += n * dir;
  }
}

// Bytes of the parts of a workspace, each a multiple of 256.
inline size_t pad256(size_t n) { return (n + 255) / 256 * 256; }
inline size_t ends_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.N * q.C * 4) : 0; }
inline size_t sums_bytes(const Geo& q) { return q.segs > 1 ? pad256((size_t)q.B * q.segs * q.C * 4) : 0; }

// The recurrence from h0 with a.y (NULL: only its states) (ssm_fwd.hip).
hipError_t launch_states(const gdr_ssm_args& a, const Geo& q, float* ends, float* sums, hipStream_t s);

}  // namespace ssm
}  // namespace gdr
