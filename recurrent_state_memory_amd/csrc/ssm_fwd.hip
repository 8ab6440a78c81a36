// ssm_fwd.hip -- selective state space scan: forward and single-token step, gfx950.
//
// Tiles of 16 tokens x 64 channels.  All waves turn the tile's inputs into (d, d x) in
// LDS, each wave runs its states through the tile (per state and token: d A, exp2, d x B, two
// fma; B and C from scalar registers) and leaves its part of y in LDS, and all waves add the
// parts, D x and the gate.  Bound by the vector units: 6 issue slots a state and token.
#include "ssm_tile.h"

namespace gdr {
namespace ssm {

using chan::ld;
using chan::raw4;
using chan::Run;

constexpr int kTile = 16;

// ---------------------------------------------------------------- vectors
template <typename T>
__global__ __launch_bounds__(256) void ssm_vector_kernel(const T* Bv, const T* Cv, const int32_t* lens, Geo q, f4* out) {
  const size_t total = (size_t)q.B * q.G * q.pairs * q.Tp;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
    const size_t row = i / q.Tp, bg = row / q.pairs, b = bg / q.G, g = bg - b * q.G;
    const int t = (int)(i - row * q.Tp), n = (int)(row - bg * q.pairs) * 2;
    f4 v = {0.f, 0.f, 0.f, 0.f};
    if (t < row_len(lens, (int)b, q.T)) {
      const size_t at = ((b * q.T + t) * q.G + g) * q.N + n;
      if (n < q.N) v.x = ld(Bv + at), v.z = ld(Cv + at);
      if (n + 1 < q.N) v.y = ld(Bv + at + 1), v.w = ld(Cv + at + 1);
    }
    out[i] = v;
  }
}

hipError_t launch_vectors(int io_dtype, const void* Bv, const void* Cv, const int32_t* lens, const Geo& q, float* out,
                          hipStream_t s) {
  const size_t blocks = ((size_t)q.B * q.G * q.pairs * q.Tp + 255) / 256;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536));
  if (io_dtype == GDR_BF16)
    hipLaunchKernelGGL(ssm_vector_kernel<__bf16>, grid, dim3(256), 0, s, (const __bf16*)Bv, (const __bf16*)Cv,
                       lens, q, (f4*)out);
  else
    hipLaunchKernelGGL(ssm_vector_kernel<float>, grid, dim3(256), 0, s, (const float*)Bv, (const float*)Cv, lens, q,
                       (f4*)out);
  return hipGetLastError();
}

// ---------------------------------------------------------------- forward
// MODE 0: y and everything else; 1: states alone (ckpt, h_out); 2: what a segment does to
// the state: its end from zero (the first one's from h0) and the sum of its time steps.
template <typename T, int NW, int NS, int MODE>
__global__ __launch_bounds__(NW * 64) void ssm_fwd_kernel(gdr_ssm_args p, Geo q, const float* vec, float* ends, float* sums) {
  constexpr int J = kTile / NW;   // tokens of a tile that a wave prepares and finishes
  constexpr int U = 16 / NS;
  __shared__ float2 in[kTile][kLanes];
  __shared__ float part[MODE == 0 ? NW : 1][kTile][kLanes];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place s = place_of(q);
  const int len = row_len(p.lens, s.b, q.T), t0 = s.seg * q.seg, t1 = min(t0 + q.seg, q.T);
  const size_t nc = (size_t)q.N * q.C;
  float A2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = w * NS + i;
    A2[i] = n < q.N ? p.A[(size_t)s.c * q.N + n] * scan::kLog2e : 0.f;
    h[i] = 0.f;
    if (n < q.N) {
      // h_out may be h0, so where segments run side by side only the first pass reads h0
      const size_t slot = (size_t)s.b * q.segs * nc + (size_t)n * q.C + s.c;
      if (MODE == 2 ? s.seg == 0 : q.segs == 1) {
        if (p.h0) h[i] = p.h0[((size_t)s.b * q.C + s.c) * q.N + n];
        if (MODE == 2 && s.on) ends[slot + (size_t)(q.segs - 1) * nc] = h[i];   // the last one's end is not needed
      } else if (MODE != 2) {
        if (s.seg == 0) h[i] = ends[slot + (size_t)(q.segs - 1) * nc];
        else h[i] = ends[slot];
        for (int k = 1; k < s.seg; ++k)
          h[i] = fmaf(__builtin_amdgcn_exp2f(A2[i] * sums[((size_t)s.b * q.segs + k) * q.C + s.c]), h[i], ends[slot + k * nc]);
      }
    }
  }
  Vectors v[NS / 2];
#pragma unroll
  for (int i = 0; i < NS / 2; ++i) v[i] = vectors_at(vec, q, s.b, s.g, w * (NS / 2) + i);
  const float bias = p.dt_bias ? p.dt_bias[s.c] : 0.f, D = p.D ? p.D[s.c] : 0.f;
  const bool softplus = p.softplus != 0, gate = p.z != nullptr;
  const size_t row0 = (size_t)s.b * q.T * q.C + s.c;
  const T *x = (const T*)p.x + row0, *dt = (const T*)p.dt + row0, *z = (const T*)p.z + row0;
  T* y = (T*)p.y + row0;

  float nx[J], nd[J], nz[J];   // the next tile's inputs
  auto load = [&](int tt) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = tt + j * NW + w;
      nx[j] = nd[j] = nz[j] = 0.f;
      if (t < min(t1, len)) {
        nx[j] = ld(x + (size_t)t * q.C);
        nd[j] = ld(dt + (size_t)t * q.C);
        if (MODE == 0 && gate) nz[j] = ld(z + (size_t)t * q.C);
      }
    }
  };
  load(t0);
  float total = 0.f;
  for (int tt = t0; tt < t1; tt += kTile) {
    if (MODE != 2 && p.ckpt && tt % kBlock == 0 && s.on) {
      float* ck = p.ckpt + ((size_t)s.b * (q.Tp / kBlock) + tt / kBlock) * nc + s.c;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (w * NS + i < q.N) ck[(size_t)(w * NS + i) * q.C] = h[i];
    }
    if (tt >= len) {   // behind the row's end
      if (MODE == 0) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int t = tt + j * NW + w;
          if (t < t1 && s.on) chan::st(y + (size_t)t * q.C, 0.f);
        }
      }
      continue;
    }
    float cx[J], cz[J];
    float tile = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int t = j * NW + w;
      const float d = tt + t < min(t1, len) ? time_step(nd[j] + bias, softplus) : 0.f;
      in[t][lane] = float2{d, d * nx[j]};
      tile += d;
      cx[j] = nx[j];
      cz[j] = nz[j];
    }
    total += tile;
    __syncthreads();
    load(tt + kTile);
#pragma unroll
    for (int t = 0; t < kTile; t += U) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float2 d = in[t + u][lane];
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < NS; i += 2) {
          const f4 bc = v[i / 2][tt + t + u];
          h[i] = fmaf(__builtin_amdgcn_exp2f(d.x * A2[i]), h[i], d.y * bc.x);
          h[i + 1] = fmaf(__builtin_amdgcn_exp2f(d.x * A2[i + 1]), h[i + 1], d.y * bc.y);
          if (MODE == 0) acc = fmaf(bc.w, h[i + 1], fmaf(bc.z, h[i], acc));
        }
        if (MODE == 0) part[w][t + u][lane] = acc;
      }
    }
    __syncthreads();
    if (MODE == 0) {
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int t = j * NW + w;
        float u = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) u += part[k][t][lane];
        u = fmaf(D, cx[j], u);
        if (gate) u *= cz[j] * scan::sigmoid(cz[j]);
        if (tt + t < t1 && s.on) chan::st(y + (size_t)(tt + t) * q.C, tt + t < len ? u : 0.f);
      }
    }
  }
  if (MODE == 2) {
    in[w][lane].x = total;
    __syncthreads();
    if (w == 0 && s.on) {
      total = 0.f;
#pragma unroll
      for (int k = 0; k < NW; ++k) total += in[k][lane].x;
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
static void launch_fwd(const gdr_ssm_args& a, const Geo& q, const float* vec, float* ends, float* sums, hipStream_t s) {
  const dim3 grid(MODE == 2 ? q.blocks() / q.segs * (q.segs - 1) : q.blocks());   // segments come last
  if (q.N <= 8) hipLaunchKernelGGL((ssm_fwd_kernel<T, 4, 2, MODE>), grid, dim3(256), 0, s, a, q, vec, ends, sums);
  else if (q.N <= 16) hipLaunchKernelGGL((ssm_fwd_kernel<T, 8, 2, MODE>), grid, dim3(512), 0, s, a, q, vec, ends, sums);
  else if (q.N <= 32) hipLaunchKernelGGL((ssm_fwd_kernel<T, 8, 4, MODE>), grid, dim3(512), 0, s, a, q, vec, ends, sums);
  else hipLaunchKernelGGL((ssm_fwd_kernel<T, 8, 8, MODE>), grid, dim3(512), 0, s, a, q, vec, ends, sums);
}

hipError_t launch_states(const gdr_ssm_args& a, const Geo& q, const float* vec, float* ends, float* sums, hipStream_t s) {
  const bool bf = a.io_dtype == GDR_BF16;
  if (q.segs > 1) {
    if (bf) launch_fwd<__bf16, 2>(a, q, vec, ends, sums, s);
    else launch_fwd<float, 2>(a, q, vec, ends, sums, s);
  }
  if (a.y) {
    if (bf) launch_fwd<__bf16, 0>(a, q, vec, ends, sums, s);
    else launch_fwd<float, 0>(a, q, vec, ends, sums, s);
  } else {
    if (bf) launch_fwd<__bf16, 1>(a, q, vec, ends, sums, s);
    else launch_fwd<float, 1>(a, q, vec, ends, sums, s);
  }
  return hipGetLastError();
}

size_t fwd_workspace(int B, int T, int C, int N, int G) {
  const Geo q = geo_of(B, T, C, N, G);
  return vector_bytes(q) + ends_bytes(q) + sums_bytes(q);
}

hipError_t launch_ssm_fwd(const gdr_ssm_args& a, hipStream_t s) {
  const Geo q = geo_of(a.B, a.T, a.C, a.N, a.G);
  char* ws = (char*)a.workspace;
  float *vec = (float*)ws, *ends = (float*)(ws + vector_bytes(q)), *sums = (float*)(ws + vector_bytes(q) + ends_bytes(q));
  const hipError_t e = launch_vectors(a.io_dtype, a.Bv, a.Cv, a.lens, q, vec, s);
  return e != hipSuccess ? e : launch_states(a, q, vec, ends, sums, s);
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
    h[k] = fmaf(__builtin_amdgcn_exp2f(d * (A[k] * scan::kLog2e)), h[k], dx * Bv[k]);
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
