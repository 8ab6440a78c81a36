// scan_fwd.hip -- channelwise gated linear recurrence, forward and step, gfx950.
//
// The tile, its joins and the hand-over between tiles: scan_tile.h.  A thread
// keeps a and v = b x of its 32 elements in registers between forming (P, H) of
// its run and writing the outputs, so every input is read and every gate evaluated
// once.  Bound by HBM: with given decays 537 MB of least traffic (1 x 32785 x 2048)
// take 103 us, the rate of a device copy; with the gates in the kernel (8 x 4096 x
// 2048, 545 MB) 122 us, the vector units busy in two thirds of the cycles.  Each
// thread per channel walking the tokens took 3.6 ms there, and tiles that hand the
// state over one by one 140 us on the long sequence.
#include "scan_gate.h"
#include "scan_tile.h"

namespace gdr {
namespace scan {

using chan::ld;
using chan::st;

struct FwdP {
  int B, T, C, normalise;
  int nchain, nct, nt, team;   // chains, channel tiles of a row, tiles of a chain
  const void* x;
  const uint8_t* x_exp;
  const float* alpha;
  const void* decay_x;
  const float* decay_a;
  const void* gate_x;
  const float* h0;
  void* y;
  float* h_out;
  float* ckpt;
  Chains ch;
};

// KIND: 0 alpha given, 1 decay from its pre-activation, 2 with an input gate too.
// NORM: b has sqrt(1 - a^2).  X: the type x is read in (T, or Code8).
template <typename T, typename X, int KIND, bool NORM, bool VEC>
__global__ __launch_bounds__(64 * kFwdWaves) void scan_fwd_kernel(FwdP p) {
  constexpr bool kCodes = !__is_same(X, T);
  __shared__ Joins<kFwdWaves> j;
  const Place q = take_place(p.C, p.nchain, p.nct, p.nt, p.team, p.ch.ticket);
  if (q.chain < 0) return;
  const int C = p.C, t0 = q.tt * kFwdWaves * GDR_SCAN_BLOCK;
  const int rows = min(q.nw * GDR_SCAN_BLOCK, p.T - t0);   // of the tile that exist
  const int r0 = q.wave * GDR_SCAN_BLOCK + q.grp * S;      // the thread's first row
  const size_t base = ((size_t)q.b * p.T + t0) * C;

  // a wait for a load waits for those before it too: what is needed first comes
  // first, and row by row
  Scale A[V];
  if constexpr (KIND != 0) {
    const Four<float>::R r = View<float, VEC>(p.decay_a, 0, 1, C, 0, q.c, q.nv).load(0);
#pragma unroll
    for (int k = 0; k < V; ++k) A[k] = Scale(Four<float>::get(r, k));
  }
  typename Four<X>::R rx[S];
  Four<float>::R ra[KIND == 0 ? S : 1];
  typename Four<T>::R rd[KIND == 0 ? 1 : S], rg[KIND == 2 ? S : 1];
  float xs[kCodes ? S : 1];
  {
    const auto view = [&](auto t, const void* array) {
      return View<decltype(t), VEC>(array, base, rows, C, r0, q.c, q.nv);
    };
    const auto vx = view(X{}, p.x);
    const auto va = view(float{}, p.alpha);
    const auto vd = view(T{}, p.decay_x), vg = view(T{}, p.gate_x);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if constexpr (KIND == 0) ra[i] = va.load(i);
      else rd[i] = vd.load(i);
      rx[i] = vx.load(i);
      if constexpr (KIND == 2) rg[i] = vg.load(i);
    }
    if constexpr (kCodes) {   // four neighbouring channels share a group of 128
      const int ng = (C + 127) / 128;
      const rsrc_t be = buffer(p.x_exp + ((size_t)q.b * p.T + t0) * ng, rows * ng);
      const int oe = q.nv > 0 ? r0 * ng + q.c / 128 : kNoLane;
#pragma unroll
      for (int i = 0; i < S; ++i)
        xs[i] = chan::scale_of(__builtin_amdgcn_raw_buffer_load_b8(be, oe + i * ng, 0, 0));
    }
  }
  const Words<kFwdWaves> words = look_ahead<kFwdWaves>(p.ch, q, p.nt, q.wave);
  // the start state, asked for early by the wave that joins the first super's tiles to it
  const int cc = q.c0 + q.lane;
  float h_in = 0.f;
  if (q.wave == q.nw - 1 && q.tt < kSuper && p.h0 && cc < C) h_in = p.h0[(size_t)q.b * C + cc];

  float a[S][V], v[S][V], P[V], H[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    P[k] = 1.f;
    H[k] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      float x = Four<X>::get(rx[i], k);
      if constexpr (kCodes) x *= xs[i];
      if constexpr (KIND == 0) {
        a[i][k] = Four<float>::get(ra[i], k);
      } else {
        const float sp = softplus(Four<T>::get(rd[i], k));
        a[i][k] = decay(A[k], sp);
        if constexpr (KIND == 2) x *= sigmoid(Four<T>::get(rg[i], k));
        if constexpr (NORM) x *= __builtin_amdgcn_sqrtf(one_minus_sq(A[k], sp, a[i][k]));
      }
      v[i][k] = x;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      P[k] *= a[i][k];
      H[k] = fmaf(a[i][k], H[k], v[i][k]);
    }
  }
  if (rows < q.nw * GDR_SCAN_BLOCK) {   // behind the last token the state stays
#pragma unroll
    for (int k = 0; k < V; ++k) {
      P[k] = 1.f;
      H[k] = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (r0 + i >= rows) {
          a[i][k] = 1.f;
          v[i][k] = 0.f;
        }
        P[k] *= a[i][k];
        H[k] = fmaf(a[i][k], H[k], v[i][k]);
      }
    }
  }
  float Pe[V], He[V];
  join_groups<true>(P, H, Pe, He, q.grp);
  if (q.grp == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) j.run[q.wave][q.cl + k] = float2{P[k], H[k]};
  }
  float h_end;
  const float h_wave = join_tiles(j, p.ch, q, words, p.nt, q.wave, h_in, h_end);
  if (p.h_out && q.tt + 1 == p.nt && q.wave == q.nw - 1 && cc < C) p.h_out[(size_t)q.b * C + cc] = h_end;
  if (p.ckpt && cc < C && q.wave * GDR_SCAN_BLOCK < rows)
    p.ckpt[((size_t)q.b * blocks_of(p.T) + (size_t)q.tt * kFwdWaves + q.wave) * C + cc] = h_wave;
  if (!p.y) return;   // the states were all that was wanted
  const View<T, VEC> vy(p.y, base, rows, C, r0, q.c, q.nv);
  float h[V];
#pragma unroll
  for (int k = 0; k < V; ++k) h[k] = fmaf(Pe[k], j.from[q.wave][q.cl + k], He[k]);
#pragma unroll
  for (int i = 0; i < S; ++i) {
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = fmaf(a[i][k], h[k], v[i][k]);
    vy.store(i, h);
  }
}

template <typename T>
__device__ inline void coefficients(const float* alpha, const void* decay_x, const void* gate_x, float A, int normalise,
                                    size_t i, float x, float& a, float& v) {
  v = x;
  if (alpha) {
    a = alpha[i];
    return;
  }
  const Scale sc(A);
  const float sp = softplus(ld((const T*)decay_x + i));
  a = decay(sc, sp);
  if (gate_x) v *= sigmoid(ld((const T*)gate_x + i));
  if (normalise) v *= __builtin_amdgcn_sqrtf(one_minus_sq(sc, sp, a));
}

template <typename T>
__global__ __launch_bounds__(256) void scan_step_kernel(gdr_scan_step_args p) {
  const uint32_t i = blockIdx.x * 256 + threadIdx.x;   // N C < 2^31
  if (i >= (uint32_t)(p.N * p.C)) return;
  const float A = p.alpha ? 0.f : p.decay_a[i % (uint32_t)p.C];
  float a, v;
  coefficients<T>(p.alpha, p.decay_x, p.gate_x, A, p.normalise, i, ld((const T*)p.x + i), a, v);
  const float h = fmaf(a, p.h[i], v);
  p.h_out[i] = h;
  st((T*)p.y + i, h);
}

__global__ __launch_bounds__(256) void clear_kernel(ulonglong2* p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = ulonglong2{0u, 0u};
}

// The ticket (in 256 bytes), the tiles' words, the supers'.
size_t chain_bytes(int B, int T, int C, int waves) {
  const size_t nt = tiles_t(T, waves);
  return nt > 1 ? 256 + chains_of(B, C) * (nt + (nt + kSuper - 1) / kSuper) * kTileC * 8 : 0;
}

size_t fwd_workspace(int B, int T, int C) { return chain_bytes(B, T, C, kFwdWaves); }

Chains chains_at(void* workspace, int B, int T, int C, int waves) {
  if (tiles_t(T, waves) <= 1) return Chains{nullptr, nullptr, nullptr};
  uint64_t* tiles = (uint64_t*)((char*)workspace + 256);
  return Chains{(uint32_t*)workspace, tiles, tiles + chains_of(B, C) * tiles_t(T, waves) * kTileC};
}

hipError_t clear_chains(void* workspace, size_t bytes, hipStream_t s) {
  if (bytes == 0) return hipSuccess;
  const size_t n = bytes / 16, blocks = (n + 255) / 256;   // whole rows of 64 words
  hipLaunchKernelGGL(clear_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, s,
                     (ulonglong2*)workspace, n);
  return hipGetLastError();
}

template <typename T, typename X, int KIND, bool NORM>
static hipError_t launch_v(const FwdP& p, bool vec, hipStream_t s) {
  const int nw = p.nt > 1 ? kFwdWaves : (int)blocks_of(p.T);
  const dim3 grid((unsigned)((size_t)p.nchain * p.nt)), block(64 * nw);
  if (vec) hipLaunchKernelGGL((scan_fwd_kernel<T, X, KIND, NORM, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((scan_fwd_kernel<T, X, KIND, NORM, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, typename X>
static hipError_t launch_kind(const FwdP& p, bool vec, hipStream_t s) {
  if (p.alpha) return launch_v<T, X, 0, false>(p, vec, s);
  if (p.gate_x) return p.normalise ? launch_v<T, X, 2, true>(p, vec, s) : launch_v<T, X, 2, false>(p, vec, s);
  return p.normalise ? launch_v<T, X, 1, true>(p, vec, s) : launch_v<T, X, 1, false>(p, vec, s);
}

static hipError_t launch(FwdP& p, int io_dtype, void* workspace, hipStream_t s) {
  p.nct = (p.C + kTileC - 1) / kTileC;
  p.nchain = (int)chains_of(p.B, p.C);
  p.nt = (int)tiles_t(p.T, kFwdWaves);
  p.team = team_of(p.alpha != nullptr, io_dtype);
  p.ch = chains_at(workspace, p.B, p.T, p.C, kFwdWaves);
  const size_t io = io_dtype == GDR_BF16 ? 2 : 4;
  const bool vec = p.C % 4 == 0 && vec4_ok(p.x, p.x_exp ? 1 : io) && vec4_ok(p.alpha, 4) && vec4_ok(p.decay_x, io) &&
                   vec4_ok(p.gate_x, io) && vec4_ok(p.y, io);
  if (io_dtype == GDR_BF16)
    return p.x_exp ? launch_kind<__bf16, Code8>(p, vec, s) : launch_kind<__bf16, __bf16>(p, vec, s);
  return p.x_exp ? launch_kind<float, Code8>(p, vec, s) : launch_kind<float, float>(p, vec, s);
}

hipError_t launch_scan_fwd(const gdr_scan_args& a, hipStream_t s) {
  FwdP p{a.B, a.T, a.C, a.normalise, 0, 0, 0, 0, a.x, nullptr, a.alpha, a.decay_x, a.decay_a, a.gate_x, a.h0, a.y, a.h_out,
         a.ckpt, {}};
  const hipError_t e = clear_chains(a.workspace, fwd_workspace(a.B, a.T, a.C), s);
  return e == hipSuccess ? launch(p, a.io_dtype, a.workspace, s) : e;
}

hipError_t launch_ckpt(const gdr_scan_bwd_args& a, float* ckpt, void* workspace, hipStream_t s) {
  FwdP p{a.B, a.T, a.C, a.normalise, 0, 0, 0, 0, a.x, a.x_exp, a.alpha, a.decay_x, a.decay_a, a.gate_x, a.h0, nullptr,
         nullptr, ckpt, {}};
  return launch(p, a.io_dtype, workspace, s);
}

hipError_t launch_scan_step(const gdr_scan_step_args& a, hipStream_t s) {
  const dim3 grid((unsigned)(((size_t)a.N * a.C + 255) / 256));
  if (a.io_dtype == GDR_BF16) hipLaunchKernelGGL(scan_step_kernel<__bf16>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(scan_step_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace scan
}  // namespace gdr
