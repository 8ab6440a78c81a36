// ssm_bwd.hip -- selective state space scan: backward, gfx950.
//
// Workgroups as in the forward, through the blocks of 32 tokens from the last to the first.
// A block's decays and states are computed again from its saved start state, then the
// adjoint H runs back through it.  Sums over a channel's states: each wave's parts meet in
// LDS.  Sums over the channels (grad_Bv, grad_Cv): over the 64 lanes by lane swaps and DPP, 64
// values at a time, then over the workgroups through partial results that
// ssm_vector_join_kernel adds up.
//
// Bound by the issue of instructions, two waves a SIMD as in the forward: 16 slots a state and
// token cannot be done without (6 again, 10 for the adjoint and the two sums), 518 us of the
// 923 on 8 x 4096 x 2048 with 16 states, gated; 25 are issued, 6 of them for the sums over
// lanes.  LDS and registers allow one workgroup a CU.  Half of a block's decays computed
// twice instead of kept: 1060; LDS read where it is used: 1006; row lanes moved to
// registers of their own before a multiply-add: 980 us.  (The same for all of a block makes
// the compiler spill: 2880.)
// More than 16 states go through each block in turns of 16 (8 x 2048 x 2048 bf16, gated, with
// 32: 1087 us, 64: 2072), a state at 7 to 13 % more than where there are 16 (482); two states
// at a time with half a block's tokens in registers took 1570 and 2790.  Waves without a state skip the recurrence
// (4 states: 330 -> 284 us).
#include "col_join.h"
#include "ssm_tile.h"

namespace gdr {
namespace ssm {

// ---------------------------------------------------------------- sums over lanes
// 64 values of every lane in, lane_value(v)'s sum over the 64 lanes out, by halves: each
// step adds two registers' halves into one that holds both sums.
__device__ inline float swap32_add(float x, float y) {   // lanes 0-31: x, 32-63: y
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ inline float swap16_add(float x, float y) {   // even rows of 16 lanes: x, odd ones: y
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL, int BANKS>
__device__ inline float dpp_into(float old, float src) {
  return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(src), CTRL, 0xf, BANKS, false));
}
__device__ inline float half8_add(float x, float y) {    // lanes 0-7 of a row: x, 8-15: y
  return dpp_into<0x128, 0x3>(y, x) + dpp_into<0x128, 0xc>(x, y);
}
__device__ inline float half4_add(float x, float y) {    // lanes 0-3 of 8: x, 4-7: y
  return dpp_into<0x141, 0x5>(y, x) + dpp_into<0x141, 0xa>(x, y);
}
template <int CTRL>
__device__ inline float pick_add(bool second, float x, float y) {
  return (second ? y : x) + dpp_into<CTRL, 0xf>(0.f, second ? x : y);
}
// Of four registers that hold 16 lanes' quads: quad lane i has register perm(i)'s sum.
__device__ inline float quads_add(const float (&r)[4]) {   // lane & 2: r[1], r[3]; lane & 1: r[2], r[3]
  const bool b1 = threadIdx.x & 2, b0 = threadIdx.x & 1;
  const float lo = pick_add<0x4E>(b1, r[0], r[1]), hi = pick_add<0x4E>(b1, r[2], r[3]);
  return pick_add<0xB1>(b0, lo, hi);
}

// ---------------------------------------------------------------- reverse segments
// What a segment does to the adjoint: a_t (C_t g_t + ...) from its end (zero; grad_h at the
// last segment's) to its start, and the sum of its time steps.
template <typename T, int NS>
__global__ __launch_bounds__(kWaves * 64) void ssm_adjoint_kernel(gdr_ssm_bwd_args p, Geo q, float* ends, float* sums) {
  constexpr int NW = kWaves, kTile = 16, J = kTile / NW;
  __shared__ float2 in[2][kTile][kLanes];   // d, g
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Place s = place_of(q);
  ++s.seg;   // the first one's start has no use
  const int len = row_len(p.lens, s.b, q.T), t0 = s.seg * q.seg, end = min(min(t0 + q.seg, q.T), len);
  const size_t nc = (size_t)q.N * q.C;
  float A2[NS], K[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = w * NS + i;
    A2[i] = n < q.N ? held(p.A[(size_t)s.c * q.N + n]) * scan::kLog2e : 0.f;
    K[i] = n < q.N && p.grad_h && s.seg == q.segs - 1 ? p.grad_h[((size_t)s.b * q.C + s.c) * q.N + n] : 0.f;
  }
  const float bias = p.dt_bias ? p.dt_bias[s.c] : 0.f;
  const bool softplus = p.softplus != 0, gate = p.z != nullptr;
  const Buffer dt = rows_at<T>(p.dt, q, s.b, t0, end), gy = rows_at<T>(p.grad_y, q, s.b, t0, end),
               z = rows_at<T>(p.z, q, s.b, t0, gate ? end : t0);
  const unsigned row_bytes = (unsigned)(q.C * sizeof(T)), col = s.on ? (unsigned)(s.c * sizeof(T)) : kNowhere;
  // One step of vectors (only C_t is used) and inputs ahead; tiles from the last to the first.
  typedef Vectors<T, NS, kTile> V;
  const V vectors(p.Bv, p.Cv, q, s, t0, end, w * NS);
  typename V::Raw vr;
  typedef typename Io<T>::Raw Raw;
  Raw nd[J], ng[J], nz[J];
  auto load = [&](int i) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const unsigned at = col + (unsigned)(i * kTile + j * NW + w) * row_bytes;
      nd[j] = Io<T>::load(dt, at);
      ng[j] = Io<T>::load(gy, at);
    }
    if (gate) {
#pragma unroll
      for (int j = 0; j < J; ++j) nz[j] = Io<T>::load(z, col + (unsigned)(i * kTile + j * NW + w) * row_bytes);
    }
  };
  const int n = end > t0 ? (end - t0 + kTile - 1) / kTile : 0;
  float total = 0.f;
  if (n > 0) load(n - 1), vectors.load((n - 1) * kTile, vr);
  for (int i = n - 1; i >= 0; --i) {
    const int tt = t0 + i * kTile;
    float tile = 0.f;
    typename V::Set v;
    vectors.take(vr, v);
    if (i > 0) vectors.load((i - 1) * kTile, vr);
    float2(*to)[kLanes] = in[i & 1];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = j * NW + w;
      const float d = tt + t < end ? time_step(Io<T>::get(nd[j]) + bias, softplus) : 0.f;
      float g = Io<T>::get(ng[j]);   // 0 from `end` on, and z with it
      if (gate) {
        const float zf = Io<T>::get(nz[j]);
        g *= zf * scan::sigmoid(zf);
      }
      to[t][lane] = float2{d, g};
      tile += d;
    }
    total += tile;
    if (i > 0) load(i - 1);
    __syncthreads();   // the tile before last is read no more
    if (NS == 1 && w >= q.N) continue;   // a wave without a state
    each<kTile>([&](auto back) {
      constexpr int t = kTile - 1 - decltype(back)::value, L = t % V::M * V::W;
      const float2 d = to[t][lane];
#pragma unroll
      for (int k = 0; k < V::P; ++k) {
        const float cv = v.c[k][t / V::M];
        float* Kk = K + V::W * k;
        const float* Ak = A2 + V::W * k;
        Kk[0] = __builtin_amdgcn_exp2f(d.x * Ak[0]) * fmaf(row_lane<L>(cv), d.y, Kk[0]);
        if constexpr (V::W == 2) Kk[1] = __builtin_amdgcn_exp2f(d.x * Ak[1]) * fmaf(row_lane<L + 1>(cv), d.y, Kk[1]);
      }
    });
  }
  __syncthreads();
  in[0][w][lane].x = total;
  __syncthreads();
  if (w == 0 && s.on) {
    total = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) total += in[0][k][lane].x;
    sums[((size_t)s.b * q.segs + s.seg) * q.C + s.c] = total;
  }
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (w * NS + i < q.N && s.on) ends[((size_t)s.b * q.segs + s.seg) * nc + (size_t)(w * NS + i) * q.C + s.c] = K[i];
}

// ---------------------------------------------------------------- backward
// What the kernel below starts with: the adjoints of states first ... behind a segment.
template <int NS>
__device__ inline void adjoint_behind(const gdr_ssm_bwd_args& p, const Geo& q, const Place& s, int first,
                                      const float (&A2)[NS], const float* ends, const float* sums, float (&K)[NS]) {
  const bool last = s.seg == q.segs - 1;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = first + i;
    K[i] = 0.f;
    if (n >= q.N) continue;
    if (!last) K[i] = ends[(((size_t)s.b * q.segs + q.segs - 1) * q.N + n) * q.C + s.c];
    else if (p.grad_h) K[i] = p.grad_h[((size_t)s.b * q.C + s.c) * q.N + n];
  }
  if (!last) pass_segments<NS>(q, s, first, q.segs - 2, s.seg, -1, A2, ends, sums, K);
#pragma unroll
  for (int i = 0; i < NS; ++i)
    if (!s.on) K[i] = 0.f;   // lanes without a channel add nothing to the sums
}
// The lane's place among the 64 sums of a wave: of 16 tokens and two states' B and C, or
// of 32 tokens and one state's; from the first state's B of the first token on, in a plane
// [Tp] each: [states][B, C][Tp].
template <int NS>
__device__ inline size_t sum_place(int Tp) {
  const int l = threadIdx.x & 63, b5 = l >> 5, b4 = l >> 4 & 1, b3 = l >> 3 & 1, b2 = l >> 2 & 1, b1 = l >> 1 & 1, b0 = l & 1;
  if (NS == 2) return (size_t)(b5 * 2 + b4) * Tp + (b3 | b2 << 1 | b1 << 2 | b0 << 3);
  return (size_t)b5 * Tp + (b4 | b3 << 1 | b2 << 2 | b1 << 3 | b0 << 4);
}
// A turn's values among all turns', which are registers.
template <int NCH, int NS>
__device__ inline void pick(int ch, const float (&all)[NCH][NS], float (&v)[NS]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < NS; ++k) v[k] = c == 0 || c == ch ? all[c][k] : v[k];
}
template <int NCH, int NS>
__device__ inline void put(int ch, const float (&v)[NS], float (&all)[NCH][NS]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int k = 0; k < NS; ++k) all[c][k] = NCH == 1 || c == ch ? v[k] : all[c][k];
}
// What a channel's token is prepared to.
struct Token {
  float x, z, gy, slope;   // slope of softplus
};

// Eight waves of one or two states each; more than 16 are taken 16 at a time, NCH turns at
// the most, through each block.  A turn's 32 states and decays of a block stay in registers.
// The adjoint passes through it in four quarters; while one is worked on, the one before
// is finished (the waves' parts added, gradients written), and the next block's inputs are
// on their way (with several turns, from the third quarter on: they take registers).
template <typename T, int NS, bool GATE, int NCH>
__global__ __launch_bounds__(kWaves * 64) void ssm_bwd_kernel(gdr_ssm_bwd_args p, Geo q, const float* ckpt, const float* ends,
                                                          const float* sums, float* vpart, float* rows) {
  constexpr int NW = kWaves, J = kBlock / NW, QT = 8;
  static_assert(NW == QT && (NS == 1 || NS == 2), "a token of a quarter for every wave");
  static_assert(NCH == 1 || NS == 2, "a turn has 16 states");
  __shared__ float2 in[kBlock][kLanes];                        // d, d x
  __shared__ float gs[kBlock][kLanes];                         // g
  __shared__ float part[2][2][NW][QT][kLanes];                 // each wave's share of p and sum A q, two quarters
  __shared__ float upart[GATE ? NW : 1][GATE ? kBlock : 1][kLanes];   // of sum C h
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place s = place_of(q);
  const int len = row_len(p.lens, s.b, q.T), t0 = s.seg * q.seg, t1 = min(t0 + q.seg, q.T), end = min(t1, len);
  const size_t nc = (size_t)q.N * q.C;
  const int turns = NCH == 1 ? 1 : (q.N + NW * NS - 1) / (NW * NS);
  auto state = [&](int ch, int k) { return (ch * NW + w) * NS + k; };
  auto load_A = [&](int ch, float(&A)[NS]) {
#pragma unroll
    for (int k = 0; k < NS; ++k) A[k] = state(ch, k) < q.N ? p.A[(size_t)s.c * q.N + state(ch, k)] : 0.f;
  };
  float A[NS], A2[NS], Ks[NCH][NS], gA[NCH][NS];
#pragma unroll
  for (int ch = NCH - 1; ch >= 0; --ch) {
    load_A(ch, A);
#pragma unroll
    for (int k = 0; k < NS; ++k) A[k] = held(A[k]), A2[k] = A[k] * scan::kLog2e, gA[ch][k] = 0.f;
    adjoint_behind<NS>(p, q, s, state(ch, 0), A2, ends, sums, Ks[ch]);
  }
  const float* const ck = ckpt + ((size_t)s.b * (q.Tp / kBlock) + t0 / kBlock) * nc + s.c;   // the states' checkpoints
  const float* ck1[NS];   // the only turn's
  bool has[NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    has[k] = state(0, k) < q.N && s.on;
    ck1[k] = ck + (size_t)(has[k] ? state(0, k) : 0) * q.C;
  }
  const float bias = p.dt_bias ? p.dt_bias[s.c] : 0.f, D = p.D ? p.D[s.c] : 0.f;
  const bool softplus = p.softplus != 0;
  const Buffer x = rows_at<T>(p.x, q, s.b, t0, end), dt = rows_at<T>(p.dt, q, s.b, t0, end),
               gy = rows_at<T>(p.grad_y, q, s.b, t0, end), z = rows_at<T>(p.z, q, s.b, t0, GATE ? end : t0),
               gx = rows_at<T>(p.grad_x, q, s.b, t0, end), gdt = rows_at<T>(p.grad_dt, q, s.b, t0, end),
               gz = rows_at<T>(p.grad_z, q, s.b, t0, GATE ? end : t0);
  const unsigned row_bytes = (unsigned)(q.C * sizeof(T)), col = s.on ? (unsigned)(s.c * sizeof(T)) : kNowhere;
  typedef Vectors<T, NS, kBlock> V;
  V vectors(p.Bv, p.Cv, q, s, t0, end, w * NS);
  float* const vout0 = vpart + (((size_t)s.cb * q.B + s.b) * q.room + w * NS) * 2 * q.Tp + t0 + sum_place<NS>(q.Tp);

  auto clear = [&]() {   // an idle wave's parts
#pragma unroll
    for (int t = 0; t < 2 * QT; ++t) part[t & 1][0][w][t >> 1][lane] = part[t & 1][1][w][t >> 1][lane] = 0.f;
    if (GATE) {
#pragma unroll
      for (int t = 0; t < kBlock; ++t) upart[GATE ? w : 0][GATE ? t : 0][lane] = 0.f;
    }
  };
  if (NS == 1 && state(0, 0) >= q.N) clear();

  // the next block's inputs as they come
  typedef typename Io<T>::Raw Raw;
  Raw nx[J], nd[J], ng[J], nz[J];
  typename V::Raw vr;
  float nh[NS], nA[NS];
  auto load_states = [&](int i, int ch) {   // and what a turn starts with
    if constexpr (NCH > 1) {
      vectors.states(q, state(ch, 0));
      load_A(ch, nA);
    }
    vectors.load(i * kBlock, vr);
#pragma unroll
    for (int k = 0; k < NS; ++k)
      if constexpr (NCH == 1) nh[k] = has[k] ? ck1[k][i * nc] : 0.f;
      else nh[k] = state(ch, k) < q.N && s.on ? ck[i * nc + (size_t)state(ch, k) * q.C] : 0.f;
  };
  auto load_inputs = [&](int i, unsigned col) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const unsigned at = col + (unsigned)(i * kBlock + j * NW + w) * row_bytes;
      nx[j] = Io<T>::load(x, at);
      nd[j] = Io<T>::load(dt, at);
      ng[j] = Io<T>::load(gy, at);
      if (GATE) nz[j] = Io<T>::load(z, at);
    }
  };
  float gD = 0.f, gbias = 0.f;
  const int n = end > t0 ? (end - t0 + kBlock - 1) / kBlock : 0;   // blocks
  if (n > 0) load_inputs(n - 1, col), load_states(n - 1, 0);
#pragma unroll 1
  for (int i = n - 1; i >= 0; --i) {
    const int tt = t0 + i * kBlock;
    Token own[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = j * NW + w;
      own[j].slope = 1.f;
      float d = Io<T>::get(nd[j]) + bias, g = Io<T>::get(ng[j]);   // zeros from `end` on
      if (softplus) d = scan::softplus(d, own[j].slope);
      if (tt + t >= end) d = own[j].slope = 0.f;
      own[j].x = Io<T>::get(nx[j]);
      if (GATE) {
        own[j].gy = g;
        own[j].z = Io<T>::get(nz[j]);
        g *= own[j].z * scan::sigmoid(own[j].z);
      }
      if (!s.on) d = 0.f;   // lanes without a channel add nothing to the sums
      in[t][lane] = float2{d, d * own[j].x};
      gs[t][lane] = g;
    }
    float sp[NCH > 1 ? J : 1], sd[NCH > 1 ? J : 1], su[NCH > 1 ? J : 1];   // the turns' sums
    if constexpr (NCH > 1) {
#pragma unroll
      for (int j = 0; j < J; ++j) sp[j] = sd[j] = su[j] = 0.f;
    }
    auto turn = [&](int ch) {
      const bool last = ch == turns - 1;
      float K[NS];
      pick(ch, Ks, K);
      typename V::Set v;
      vectors.take(vr, v);
      float h[kBlock + 1][NS], a[kBlock][NS];
#pragma unroll
      for (int k = 0; k < NS; ++k) {
        h[0][k] = nh[k];
        if constexpr (NCH > 1) A[k] = held(nA[k]), A2[k] = A[k] * scan::kLog2e;
      }
      float* const vout = vout0 + (size_t)ch * (NW * NS) * 2 * q.Tp;
      // a wave without a state leaves the others its SIMD
      const bool idle = (NS == 1 || NCH > 1) && state(ch, 0) >= q.N;
      __syncthreads();
      if (NCH > 1 && idle) clear();
      if constexpr (NCH == 1) {
        if (i > 0) load_inputs(i - 1, col), load_states(i - 1, 0);
      }
      float r2[2], r4[2], r8[2], r16[4], gAb[NS];
#pragma unroll
      for (int k = 0; k < NS; ++k) gAb[k] = 0.f;
      float2 rd[2];
      float rg[2];
      if (!idle) {
        // LDS is read a group of tokens ahead; the groups stay apart, else loads of many of
        // them take the registers
        float2 dn[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) dn[u] = in[u][lane];
        each<kBlock / 4>([&](auto gi) {
          constexpr int t4 = decltype(gi)::value * 4;
          const float2 d4[4] = {dn[0], dn[1], dn[2], dn[3]};
          if constexpr (t4 + 4 < kBlock) {
#pragma unroll
            for (int u = 0; u < 4; ++u) dn[u] = in[t4 + 4 + u][lane];
          }
          each<4>([&](auto ui) {
            constexpr int u = decltype(ui)::value, t = t4 + u, L = t % V::M * V::W;
            const float2 d = d4[u];
            const float bv = v.b[0][t / V::M];
#pragma unroll
            for (int k = 0; k < NS; ++k) a[t][k] = __builtin_amdgcn_exp2f(d.x * A2[k]);
            h[t + 1][0] = fmaf(a[t][0], h[t][0], d.y * row_lane<L>(bv));
            if constexpr (NS == 2) h[t + 1][1] = fmaf(a[t][1], h[t][1], d.y * row_lane<L + 1>(bv));
            if constexpr (GATE && NS == 1) upart[w][t][lane] = row_lane<L>(v.c[0][t / V::M]) * h[t + 1][0];
          });
          if constexpr (GATE && NS == 2) {
            float u[4];
            row_dots<t4 % V::M * 2, false>(v.c[0][t4 / V::M], h[t4 + 1][0], h[t4 + 2][0], h[t4 + 3][0], h[t4 + 4][0], h[t4 + 1][1],
                                           h[t4 + 2][1], h[t4 + 3][1], h[t4 + 4][1], u);
#pragma unroll
            for (int k = 0; k < 4; ++k) upart[w][t4 + k][lane] = u[k];
          }
          __builtin_amdgcn_sched_barrier(0);
        });
        vectors.forget(v);
#pragma unroll
        for (int u = 0; u < 2; ++u) rd[u] = in[kBlock - 2 + u][lane], rg[u] = gs[kBlock - 2 + u][lane];
      }
      auto quarter = [&](auto qi) {
        constexpr int Q = decltype(qi)::value;
        if (!idle) each<QT / 2>([&](auto back) {
          constexpr int ts2 = QT - 2 - 2 * decltype(back)::value, t2 = Q * QT + ts2;
          const float2 d2[2] = {rd[0], rd[1]};
          const float g2[2] = {rg[0], rg[1]};
          if constexpr (t2 > 0) {
#pragma unroll
            for (int u = 0; u < 2; ++u) rd[u] = in[t2 - 2 + u][lane], rg[u] = gs[t2 - 2 + u][lane];
          }
          each<2>([&](auto ui) {
            constexpr int u = 1 - decltype(ui)::value, ts = ts2 + u, t = t2 + u, L = t % V::M * V::W;
            const float2 d = d2[u];
            const float g = g2[u], bv = v.b[0][t / V::M], cv = v.c[0][t / V::M];
            float H[NS], pp, dd;
            if constexpr (NS == 2) {
              H[0] = K[0], H[1] = K[1];
              pp = row_adjoint<L>(cv, bv, g, H[0], H[1]);
              r2[u] = swap16_add(swap32_add(H[0] * d.y, H[1] * d.y), swap32_add(g * h[t + 1][0], g * h[t + 1][1]));
            } else {
              H[0] = fmaf(row_lane<L>(cv), g, K[0]);
              pp = row_lane<L>(bv) * H[0];
              r2[u] = swap32_add(H[0] * d.y, g * h[t + 1][0]);
            }
#pragma unroll
            for (int k = 0; k < NS; ++k) {
              K[k] = H[k] * a[t][k];
              const float qk = K[k] * h[t][k];
              gAb[k] = fmaf(d.x, qk, gAb[k]);
              dd = k == 0 ? A[0] * qk : fmaf(A[k], qk, dd);
            }
            part[Q & 1][0][w][ts][lane] = pp;
            part[Q & 1][1][w][ts][lane] = dd;
          });
          // the lanes' sums: tokens 2m and 2m + 1 share a register, then pairs of them, ...
          if constexpr (NS == 2) {
            r8[t2 >> 1 & 1] = half8_add(r2[0], r2[1]);
            if constexpr ((t2 & 3) == 0) r16[t2 >> 2 & 3] = half4_add(r8[0], r8[1]);
            if constexpr ((t2 & 15) == 0) vout[i * kBlock + t2] = quads_add(r16);
          } else {
            r4[t2 >> 1 & 1] = swap16_add(r2[0], r2[1]);
            if constexpr ((t2 & 3) == 0) r8[t2 >> 2 & 1] = half8_add(r4[0], r4[1]);
            if constexpr ((t2 & 7) == 0) r16[t2 >> 3 & 3] = half4_add(r8[0], r8[1]);
            if constexpr ((t2 & 31) == 0) vout[i * kBlock + t2] = quads_add(r16);
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      };
      auto finish = [&](auto qi) {
        constexpr int Q = decltype(qi)::value;
        const int t = Q * QT + w;
        float pp = 0.f, dd = 0.f;
#pragma unroll
        for (int m = 0; m < NW; ++m) pp += part[Q & 1][0][m][w][lane], dd += part[Q & 1][1][m][w][lane];
        auto sum_u = [&](float u) {
#pragma unroll
          for (int m = 0; m < NW; ++m) u += upart[GATE ? m : 0][GATE ? t : 0][lane];
          return u;
        };
        if constexpr (NCH > 1) {
          pp = sp[Q] += pp, dd = sd[Q] += dd;
          if (GATE) su[Q] = sum_u(su[Q]);
          if (!last) return;
        }
        const float d = in[t][lane].x, g = gs[t][lane], gd = fmaf(pp, own[Q].x, dd) * own[Q].slope;
        const unsigned at = col + (unsigned)(i * kBlock + t) * row_bytes;
        gbias += gd;
        gD = fmaf(g, own[Q].x, gD);
        Io<T>::store(gx, at, fmaf(pp, d, D * g));
        Io<T>::store(gdt, at, gd);
        if (GATE) {
          const float u = NCH > 1 ? fmaf(D, own[Q].x, su[NCH > 1 ? Q : 0]) : sum_u(D * own[Q].x);
          const float sg = scan::sigmoid(own[Q].z);
          Io<T>::store(gz, at, own[Q].gy * u * sg * fmaf(own[Q].z, 1.f - sg, 1.f));
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      quarter(std::integral_constant<int, 3>());
      __syncthreads();
      finish(std::integral_constant<int, 3>());
      quarter(std::integral_constant<int, 2>());
      __syncthreads();
      finish(std::integral_constant<int, 2>());
      if constexpr (NCH > 1) {
        // Into the registers of the quarters that are done; in every turn, else those that do
        // not load keep the registers.
        load_inputs(i - 1, last && i > 0 ? col : kNowhere);
        load_states(last && i > 0 ? i - 1 : i, last ? 0 : ch + 1);
      }
      quarter(std::integral_constant<int, 1>());
      __syncthreads();
      finish(std::integral_constant<int, 1>());
      quarter(std::integral_constant<int, 0>());
      __syncthreads();
      // in, gs and own are this wave's own tokens' here, so the next block's may follow
      finish(std::integral_constant<int, 0>());
      put(ch, K, Ks);
#pragma unroll
      for (int c = 0; c < NCH; ++c)   // block by block: fewer additions behind a sum
#pragma unroll
        for (int k = 0; k < NS; ++k) gA[c][k] += NCH == 1 || c == ch ? gAb[k] : 0.f;
    };
    if constexpr (NCH == 1) {
      turn(0);
    } else {
#pragma unroll 1
      for (int ch = 0; ch < turns; ++ch) turn(ch);
    }
  }
  // behind the row's end the gradients are 0
  if (s.on) {
    for (int t = max(end, t0) + w; t < t1; t += NW) {
      const size_t at = ((size_t)s.b * q.T + t) * q.C + s.c;
      chan::st((T*)p.grad_x + at, 0.f);
      chan::st((T*)p.grad_dt + at, 0.f);
      if (GATE) chan::st((T*)p.grad_z + at, 0.f);
    }
  }
  // parameters' gradients: a row [N + 2][C] of this batch row and segment
  float* out = rows + ((size_t)s.b * q.segs + s.seg) * (q.N + 2) * q.C + s.c;
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch)
#pragma unroll
    for (int k = 0; k < NS; ++k) {
      const int n = state(ch, k);
      if (n < q.N && s.on) {
        out[(size_t)n * q.C] = gA[ch][k];
        if (p.grad_h0 && s.seg == 0) p.grad_h0[((size_t)s.b * q.C + s.c) * q.N + n] = Ks[ch][k];
      }
    }
  __syncthreads();
  in[w][lane] = float2{gD, gbias};
  __syncthreads();
  if (w == 0 && s.on) {
    gD = gbias = 0.f;
#pragma unroll
    for (int k = 0; k < NW; ++k) gD += in[k][lane].x, gbias += in[k][lane].y;
    out[(size_t)q.N * q.C] = gD;
    out[(size_t)(q.N + 1) * q.C] = gbias;
  }
}

// The vectors' gradients: over the workgroups of a group's channels.
template <typename T>
__global__ __launch_bounds__(256) void ssm_vector_join_kernel(const float* part, Geo q, const int32_t* lens, T* gB, T* gC) {
  const size_t total = (size_t)q.B * q.G * q.N * q.Tp, step = (size_t)q.B * q.room * 2 * q.Tp;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
    const size_t row = i / q.Tp, gb = row / q.N, g = gb / q.B, b = gb - g * q.B;
    const int t = (int)(i - row * q.Tp), n = (int)(row - gb * q.N);
    if (t >= q.T) continue;
    float sb = 0.f, sc = 0.f;
    if (t < row_len(lens, (int)b, q.T)) {
      const float* at = part + ((g * q.nb * q.B + b) * q.room + n) * 2 * q.Tp + t;
#pragma unroll 4
      for (int k = 0; k < q.nb; ++k) sb += at[k * step], sc += at[k * step + q.Tp];
    }
    const size_t o = ((b * q.T + t) * q.G + g) * q.N + n;
    chan::st(gB + o, sb);
    chan::st(gC + o, sc);
  }
}

struct ParamGrads {
  int C, N;
  float *A, *D, *bias;
  __device__ void operator()(size_t i, float v) const {
    const int n = (int)(i / C), c = (int)(i - (size_t)n * C);
    if (n < N) A[(size_t)c * N + n] = v;
    else if (n == N ? D != nullptr : bias != nullptr) (n == N ? D : bias)[c] = v;
  }
};

// The parts of a workspace: the segments' ends and sums, partial gradients of the
// vectors and of the parameters, block-start states where none were saved.
struct Parts {
  size_t ends, sums, vpart, rows, ckpt, bytes;
};
static Parts parts_of(const Geo& q, const Geo& f, bool ckpt) {   // f: of the forward that computes the states again
  Parts w;
  w.ends = 0;
  w.sums = ckpt || ends_bytes(q) > ends_bytes(f) ? ends_bytes(q) : ends_bytes(f);
  w.vpart = w.sums + (ckpt || sums_bytes(q) > sums_bytes(f) ? sums_bytes(q) : sums_bytes(f));
  w.rows = w.vpart + pad256((size_t)q.G * q.nb * q.B * q.room * 2 * q.Tp * 4);
  w.ckpt = w.rows + pad256((size_t)q.B * q.segs * (q.N + 2) * q.C * 4);
  w.bytes = w.ckpt + (ckpt ? 0 : pad256((size_t)q.B * (q.Tp / kBlock) * q.N * q.C * 4));
  return w;
}

size_t bwd_workspace(int B, int T, int C, int N, int G, bool ckpt) {
  return parts_of(geo_of(B, T, C, N, G, true), geo_of(B, T, C, N, G, false), ckpt).bytes;
}

template <typename T>
static hipError_t bwd(const gdr_ssm_bwd_args& a, hipStream_t s) {
  const Geo q = geo_of(a.B, a.T, a.C, a.N, a.G, true), fq = geo_of(a.B, a.T, a.C, a.N, a.G, false);
  const Parts w = parts_of(q, fq, a.ckpt != nullptr);
  char* ws = (char*)a.workspace;
  float *ends = (float*)(ws + w.ends), *sums = (float*)(ws + w.sums), *vpart = (float*)(ws + w.vpart),
        *rows = (float*)(ws + w.rows);
  const float* ckpt = a.ckpt;
  if (!ckpt) {
    gdr_ssm_args f{};
    f.io_dtype = a.io_dtype, f.softplus = a.softplus;
    f.x = a.x, f.dt = a.dt, f.A = a.A, f.dt_bias = a.dt_bias, f.h0 = a.h0, f.lens = a.lens;
    f.ckpt = (float*)(ws + w.ckpt);
    ckpt = f.ckpt;
    f.Bv = a.Bv, f.Cv = a.Cv;
    const hipError_t e = launch_states(f, fq, ends, sums, s);
    if (e != hipSuccess) return e;
  }
  if (q.segs > 1) {
    const dim3 some(q.blocks() / q.segs * (q.segs - 1)), block(kWaves * 64);
    if (q.N <= 8) hipLaunchKernelGGL((ssm_adjoint_kernel<T, 1>), some, block, 0, s, a, q, ends, sums);
    else if (q.N <= 16) hipLaunchKernelGGL((ssm_adjoint_kernel<T, 2>), some, block, 0, s, a, q, ends, sums);
    else if (q.N <= 32) hipLaunchKernelGGL((ssm_adjoint_kernel<T, 4>), some, block, 0, s, a, q, ends, sums);
    else hipLaunchKernelGGL((ssm_adjoint_kernel<T, 8>), some, block, 0, s, a, q, ends, sums);
  }
  const dim3 grid(q.blocks());
#define SSM_BWD(...) \
  hipLaunchKernelGGL((__VA_ARGS__), grid, dim3(kWaves * 64), 0, s, a, q, ckpt, ends, sums, vpart, rows)
  if (q.N <= 8 && a.z) SSM_BWD(ssm_bwd_kernel<T, 1, true, 1>);
  else if (q.N <= 8) SSM_BWD(ssm_bwd_kernel<T, 1, false, 1>);
  else if (q.N <= 16 && a.z) SSM_BWD(ssm_bwd_kernel<T, 2, true, 1>);
  else if (q.N <= 16) SSM_BWD(ssm_bwd_kernel<T, 2, false, 1>);
  else if (a.z) SSM_BWD(ssm_bwd_kernel<T, 2, true, 4>);
  else SSM_BWD(ssm_bwd_kernel<T, 2, false, 4>);
#undef SSM_BWD
  const size_t blocks = ((size_t)q.B * q.G * q.N * q.Tp + 255) / 256;
  hipLaunchKernelGGL(ssm_vector_join_kernel<T>, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256), 0, s,
                     vpart, q, a.lens, (T*)a.grad_Bv, (T*)a.grad_Cv);
  launch_col_join(rows, (size_t)q.B * q.segs, (size_t)(q.N + 2) * q.C, ParamGrads{q.C, q.N, a.grad_A, a.grad_D, a.grad_dt_bias}, s);
  return hipGetLastError();
}

hipError_t launch_ssm_bwd(const gdr_ssm_bwd_args& a, hipStream_t s) {
  return a.io_dtype == GDR_BF16 ? bwd<__bf16>(a, s) : bwd<float>(a, s);
}

}  // namespace ssm
}  // namespace gdr
