// ssm_fwd.hip -- selective state space scan: forward and single-token step, gfx950.
//
// Tiles of 16 tokens x 64 channels, in three steps: all waves turn the tile's inputs into
// (d, d x) in LDS; each wave runs its states through the tile (per state and token: d A,
// exp2, d x B, two fma) and leaves its part of y in LDS; all waves add the parts, D x and
// the gate.  Between two barriers the last step of one tile,
// the first of the next but one and the middle one of the tile between are done.
//
// Bound by the issue of instructions: 6.2 slots a state and token (exp2 takes 2.2), 198 us of
// the 331 that 8 x 4096 x 2048 with 16 states takes; there each SIMD has two waves, and one
// issues no more than an instruction every 8 cycles.  With four waves a SIMD the same number
// of states takes 266 us (1 x 32785 x 2048: 16 segments, after a pass of 189 us for their
// ends).  Sixteen waves of one state for few rows: 364 us, the LDS being busy.
// Two barriers a tile: 403 us; descriptors made anew each tile: 397 us.  Waves without a state
// skip the recurrence (8 x 2048 x 2048 with 4 states: 123 -> 99 us).
#include "ssm_tile.h"

namespace gdr {
namespace ssm {

using chan::ld;
using chan::raw4;
using chan::Run;

constexpr int kTile = 16;

// ---------------------------------------------------------------- forward
// MODE 0: y and everything else; 1: states alone (ckpt, h_out); 2: what a segment does to
// the state: its end from zero (the first one's from h0) and the sum of its time steps.
template <typename T, int NS, int MODE>
__global__ __launch_bounds__(kWaves * 64) void ssm_fwd_kernel(gdr_ssm_args p, Geo q, float* ends, float* sums) {
  constexpr int NW = kWaves, J = kTile / NW;   // tokens of a tile that a wave prepares and finishes
  __shared__ float2 in[2][kTile][kLanes];
  __shared__ float part[MODE == 0 ? 2 : 1][MODE == 0 ? NW : 1][kTile][kLanes];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place s = place_of(q);
  const int len = row_len(p.lens, s.b, q.T), t0 = s.seg * q.seg, t1 = min(t0 + q.seg, q.T), end = min(t1, len);
  const size_t nc = (size_t)q.N * q.C;
  // A wave without a state leaves the others its SIMD (with more states a wave at most
  // three of the eight are without: it gains 2 % at 20 states and costs 1 % where none are).
  const bool idle = NS == 1 && w * NS >= q.N;
  float A2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = w * NS + i;
    A2[i] = n < q.N ? held(p.A[(size_t)s.c * q.N + n]) * scan::kLog2e : 0.f;
    h[i] = 0.f;
    if (n < q.N) {
      // h_out may be h0, so where segments run side by side only the first pass reads h0
      const size_t slot = (size_t)s.b * q.segs * nc + (size_t)n * q.C + s.c;
      if (MODE == 2 ? s.seg == 0 : q.segs == 1) {
        if (p.h0) h[i] = p.h0[((size_t)s.b * q.C + s.c) * q.N + n];
        if (MODE == 2 && s.on) ends[slot + (size_t)(q.segs - 1) * nc] = h[i];   // the last one's end is not needed
      } else if (MODE != 2) {
        h[i] = ends[s.seg == 0 ? slot + (size_t)(q.segs - 1) * nc : slot];
      }
    }
  }
  if (MODE != 2 && s.seg > 1) pass_segments<NS>(q, s, w * NS, 1, s.seg, 1, A2, ends, sums, h);
  const float bias = p.dt_bias ? p.dt_bias[s.c] : 0.f, D = p.D ? p.D[s.c] : 0.f;
  const bool softplus = p.softplus != 0, gate = p.z != nullptr;
  const Buffer x = rows_at<T>(p.x, q, s.b, t0, end), dt = rows_at<T>(p.dt, q, s.b, t0, end),
               z = rows_at<T>(p.z, q, s.b, t0, gate ? end : t0), y = rows_at<T>(p.y, q, s.b, t0, MODE == 0 ? end : t0);
  const unsigned row_bytes = (unsigned)(q.C * sizeof(T)), col = s.on ? (unsigned)(s.c * sizeof(T)) : kNowhere;
  const int n = end > t0 ? (end - t0 + kTile - 1) / kTile : 0;   // tiles

  // Inputs as they come, of the tiles i + 1 and i + 2 while tile i is worked on, and x and
  // z of the tiles under way.
  typedef typename Io<T>::Raw Raw;
  Raw nx[2][J], nd[2][J], nz[2][J];
  float cx[2][J], cz[2][J];
  auto load = [&](int i, Raw(&ax)[J], Raw(&ad)[J], Raw(&az)[J]) {
    unsigned at[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      at[j] = col + (unsigned)(i * kTile + j * NW + w) * row_bytes;
      ax[j] = Io<T>::load(x, at[j]);
      ad[j] = Io<T>::load(dt, at[j]);
    }
    if (MODE == 0 && gate) {
#pragma unroll
      for (int j = 0; j < J; ++j) az[j] = Io<T>::load(z, at[j]);
    }
  };
  float total = 0.f;
  auto prepare = [&](int i, const Raw(&ax)[J], const Raw(&ad)[J], const Raw(&az)[J], float(&bx)[J], float(&bz)[J],
                     float2(*to)[kLanes]) {
    float tile = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = j * NW + w;
      const float d = t0 + i * kTile + t < end ? time_step(Io<T>::get(ad[j]) + bias, softplus) : 0.f;
      bx[j] = Io<T>::get(ax[j]);
      if (MODE == 0 && gate) bz[j] = Io<T>::get(az[j]);
      to[t][lane] = float2{d, d * bx[j]};
      tile += d;
    }
    if (MODE == 2) total += tile;
  };
  auto finish = [&](int i, const float(&bx)[J], const float(&bz)[J], const float(*from)[kTile][kLanes]) {
    float u[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      u[j] = D * bx[j];
#pragma unroll
      for (int k = 0; k < NW; ++k) u[j] += from[k][j * NW + w][lane];
    }
    if (gate) {
#pragma unroll
      for (int j = 0; j < J; ++j) u[j] *= bz[j] * scan::sigmoid(bz[j]);
    }
#pragma unroll
    for (int j = 0; j < J; ++j) Io<T>::store(y, col + (unsigned)(i * kTile + j * NW + w) * row_bytes, u[j]);
  };
  typedef Vectors<T, NS, kTile> V;
  const V vectors(p.Bv, p.Cv, q, s, t0, end, w * NS);
  typename V::Raw vr[2];
  auto run = [&](const typename V::Set& v, const float2(*from)[kLanes], float(*to)[kTile][kLanes]) {
    // four tokens at a time: what does not wait for the state before, then what does
    float2 d[4], dn[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) d[u] = from[u][lane];
    each<kTile / 4>([&](auto gg) {
      constexpr int t = decltype(gg)::value * 4;
      if constexpr (t + 4 < kTile) {
#pragma unroll
        for (int u = 0; u < 4; ++u) dn[u] = from[t + 4 + u][lane];
      }
      float a[4][NS], b[4][NS];
      each<4>([&](auto uu) {
        constexpr int u = decltype(uu)::value, L = (t + u) % V::M * V::W;
#pragma unroll
        for (int i = 0; i < NS; ++i) a[u][i] = __builtin_amdgcn_exp2f(d[u].x * A2[i]);
#pragma unroll
        for (int i = 0; i < V::P; ++i) {
          const float bv = v.b[i][(t + u) / V::M];
          b[u][V::W * i] = d[u].y * row_lane<L>(bv);
          if constexpr (V::W == 2) b[u][2 * i + 1] = d[u].y * row_lane<L + 1>(bv);
        }
      });
      __builtin_amdgcn_sched_barrier(0);
      float hh[4][NS], acc[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int i = 0; i < NS; ++i) hh[u][i] = h[i] = fmaf(a[u][i], h[i], b[u][i]);
        d[u] = dn[u];
      }
      if constexpr (MODE == 0) {
        constexpr int L = t % V::M * V::W;
        if constexpr (NS == 1) {
          each<4>([&](auto uu) {
            constexpr int u = decltype(uu)::value;
            acc[u] = row_lane<L + u>(v.c[0][t / V::M]) * hh[u][0];
          });
        } else {
          each<V::P>([&](auto ii) {
            constexpr int i = decltype(ii)::value;
            row_dots<L, (i > 0)>(v.c[i][t / V::M], hh[0][2 * i], hh[1][2 * i], hh[2][2 * i], hh[3][2 * i], hh[0][2 * i + 1],
                                 hh[1][2 * i + 1], hh[2][2 * i + 1], hh[3][2 * i + 1], acc);
          });
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) to[w][t + u][lane] = acc[u];
      }
    });
  };
  auto save = [&](int tt) {
    float* ck = p.ckpt + ((size_t)s.b * (q.Tp / kBlock) + tt / kBlock) * nc + s.c;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (w * NS + i < q.N && s.on) ck[(size_t)(w * NS + i) * q.C] = h[i];
  };
  // Tile i of parity P.
  auto turn = [&](auto parity, int i) {
    constexpr int P = decltype(parity)::value;
    const int tt = t0 + i * kTile;
    typename V::Set v;
    vectors.take(vr[P], v);
    vectors.load((i + 2) * kTile, vr[P]);
    if (MODE == 0 && i > 0) finish(i - 1, cx[P ^ 1], cz[P ^ 1], part[MODE == 0 ? P ^ 1 : 0]);
    prepare(i + 1, nx[P ^ 1], nd[P ^ 1], nz[P ^ 1], cx[P ^ 1], cz[P ^ 1], in[P ^ 1]);
    load(i + 3, nx[P ^ 1], nd[P ^ 1], nz[P ^ 1]);
    if (MODE != 2 && p.ckpt && tt % kBlock == 0) save(tt);
    if (!idle) run(v, in[P], part[MODE == 0 ? P : 0]);
    __syncthreads();
  };
  if (n > 0) {
    if (MODE == 0 && idle) {
#pragma unroll
      for (int t = 0; t < kTile; ++t) part[0][MODE == 0 ? w : 0][t][lane] = part[MODE == 0][MODE == 0 ? w : 0][t][lane] = 0.f;
    }
    load(0, nx[0], nd[0], nz[0]);
    load(1, nx[1], nd[1], nz[1]);
    vectors.load(0, vr[0]);
    vectors.load(kTile, vr[1]);
    prepare(0, nx[0], nd[0], nz[0], cx[0], cz[0], in[0]);
    load(2, nx[0], nd[0], nz[0]);
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < n; i += 2) {
      turn(std::integral_constant<int, 0>(), i);
      if (i + 1 < n) turn(std::integral_constant<int, 1>(), i + 1);
    }
    if (MODE == 0) {
      if (n & 1) finish(n - 1, cx[0], cz[0], part[0]);
      else finish(n - 1, cx[1], cz[1], part[MODE == 0]);
    }
  }
  // behind the row's end: y is 0 and the state what it is
  if (MODE == 0 && s.on)
    for (int t = max(end, t0) + w; t < t1; t += NW) chan::st((T*)p.y + ((size_t)s.b * q.T + t) * q.C + s.c, 0.f);
  if (MODE != 2 && p.ckpt)
    for (int tt = t0 + (n * kTile + kBlock - 1) / kBlock * kBlock; tt < t1; tt += kBlock) save(tt);
  if (MODE == 2) {
    in[0][w][lane].x = total;   // behind a barrier, and no tile is left
    __syncthreads();
    if (w == 0 && s.on) {
      total = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) total += in[0][k][lane].x;
      sums[((size_t)s.b * q.segs + s.seg) * q.C + s.c] = total;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (w * NS + i < q.N && s.on) ends[((size_t)s.b * q.segs + s.seg) * nc + (size_t)(w * NS + i) * q.C + s.c] = h[i];
  } else if (p.h_out && s.seg == q.segs - 1 && s.on) {
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (w * NS + i < q.N) p.h_out[((size_t)s.b * q.C + s.c) * q.N + w * NS + i] = h[i];
  }
}

template <typename T, int MODE>
static void launch_fwd(const gdr_ssm_args& a, const Geo& q, float* ends, float* sums, hipStream_t s) {
  const dim3 grid(MODE == 2 ? q.blocks() / q.segs * (q.segs - 1) : q.blocks());   // segments come last
  const dim3 block(kWaves * 64);
  if (q.N <= 8) hipLaunchKernelGGL((ssm_fwd_kernel<T, 1, MODE>), grid, block, 0, s, a, q, ends, sums);
  else if (q.N <= 16) hipLaunchKernelGGL((ssm_fwd_kernel<T, 2, MODE>), grid, block, 0, s, a, q, ends, sums);
  else if (q.N <= 32) hipLaunchKernelGGL((ssm_fwd_kernel<T, 4, MODE>), grid, block, 0, s, a, q, ends, sums);
  else hipLaunchKernelGGL((ssm_fwd_kernel<T, 8, MODE>), grid, block, 0, s, a, q, ends, sums);
}

hipError_t launch_states(const gdr_ssm_args& a, const Geo& q, float* ends, float* sums, hipStream_t s) {
  const bool bf = a.io_dtype == GDR_BF16;
  if (q.segs > 1) {
    if (bf) launch_fwd<__bf16, 2>(a, q, ends, sums, s);
    else launch_fwd<float, 2>(a, q, ends, sums, s);
  }
  if (a.y) {
    if (bf) launch_fwd<__bf16, 0>(a, q, ends, sums, s);
    else launch_fwd<float, 0>(a, q, ends, sums, s);
  } else {
    if (bf) launch_fwd<__bf16, 1>(a, q, ends, sums, s);
    else launch_fwd<float, 1>(a, q, ends, sums, s);
  }
  return hipGetLastError();
}

size_t fwd_workspace(int B, int T, int C, int N, int G) {
  const Geo q = geo_of(B, T, C, N, G, false);
  return ends_bytes(q) + sums_bytes(q);
}

hipError_t launch_ssm_fwd(const gdr_ssm_args& a, hipStream_t s) {
  const Geo q = geo_of(a.B, a.T, a.C, a.N, a.G, false);
  float* ends = (float*)a.workspace;
  return launch_states(a, q, ends, (float*)((char*)a.workspace + ends_bytes(q)), s);
}

// ---------------------------------------------------------------- step
// 4 states a thread, L threads a channel.
__device__ inline void load4(const float* p, int n, float (&v)[4]) {
  const raw4 r = Run<float>::load(p, n);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = Run<float>::get(r, k);
}
__device__ inline void load4(const __bf16* p, int n, float (&v)[4]) {
  typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
  typedef bf4 at2 __attribute__((aligned(2), may_alias));
  if (n >= 4) {
    const bf4 r = *(const at2*)p;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = (float)r[k];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = k < n ? (float)p[k] : 0.f;
  }
}

template <typename T, int L>
__global__ __launch_bounds__(256) void ssm_step_kernel(gdr_ssm_step_args p, int each) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, rc = i / L;
  if (rc >= (size_t)p.R * p.C) return;
  const int l = (int)(i % L), r = (int)(rc / p.C), c = (int)(rc - (size_t)r * p.C), n0 = l * 4, n = p.N - n0;
  float h[4], A[4], Bv[4], Cv[4];
  load4(p.h + rc * p.N + n0, n, h);
  const float x = ld((const T*)p.x + rc), pre = ld((const T*)p.dt + rc) + (p.dt_bias ? p.dt_bias[c] : 0.f);
  const float z = p.z ? ld((const T*)p.z + rc) : 0.f;
  load4(p.A + (size_t)c * p.N + n0, n, A);
  const size_t at = ((size_t)r * p.G + c / each) * p.N + n0;
  load4((const T*)p.Bv + at, n, Bv);
  load4((const T*)p.Cv + at, n, Cv);
  const float d = time_step(pre, p.softplus != 0), dx = d * x;
  float u = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    h[k] = fmaf(__builtin_amdgcn_exp2f(d * (held(A[k]) * scan::kLog2e)), h[k], dx * Bv[k]);
    u = k < n ? fmaf(Cv[k], h[k], u) : u;
  }
  Run<float>::store(p.h_out + rc * p.N + n0, n, h);
  if constexpr (L > 1) u = chan::lane_sum<L>(u);
  if (l == 0) {
    if (p.D) u = fmaf(p.D[c], x, u);
    if (p.z) u *= z * scan::sigmoid(z);
    chan::st((T*)p.y + rc, u);
  }
}

template <typename T>
static void step(const gdr_ssm_step_args& a, hipStream_t s) {
  const int L = a.N <= 4 ? 1 : a.N <= 8 ? 2 : a.N <= 16 ? 4 : a.N <= 32 ? 8 : 16, each = a.C / a.G;
  const dim3 grid((unsigned)(((size_t)a.R * a.C * L + 255) / 256)), block(256);
  if (L == 1) hipLaunchKernelGGL((ssm_step_kernel<T, 1>), grid, block, 0, s, a, each);
  else if (L == 2) hipLaunchKernelGGL((ssm_step_kernel<T, 2>), grid, block, 0, s, a, each);
  else if (L == 4) hipLaunchKernelGGL((ssm_step_kernel<T, 4>), grid, block, 0, s, a, each);
  else if (L == 8) hipLaunchKernelGGL((ssm_step_kernel<T, 8>), grid, block, 0, s, a, each);
  else hipLaunchKernelGGL((ssm_step_kernel<T, 16>), grid, block, 0, s, a, each);
}

hipError_t launch_ssm_step(const gdr_ssm_step_args& a, hipStream_t s) {
  if (a.io_dtype == GDR_BF16) step<__bf16>(a, s);
  else step<float>(a, s);
  return hipGetLastError();
}

}  // namespace ssm
}  // namespace gdr
