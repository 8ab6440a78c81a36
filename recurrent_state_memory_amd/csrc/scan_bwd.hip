// scan_bwd.hip -- gradients of the channelwise gated linear recurrence, gfx950.
//
// The tile and its joins: scan_tile.h.  States run forwards inside each wave's
// block of 32 tokens from the block's saved state; K_t = a_t G_t, what a token
// hands to the one before it, runs backwards over the whole sequence, handed from
// tile to tile with the last tiles first.  G_t = grad_y_t + K_{t+1}, so a run of
// tokens takes K to P K + Q with P the same product of decays.
//
// A thread keeps a, b x, the softplus and the input gate of its 32 elements in
// registers, and sigmoid(decay_x) and n = sqrt(1 - a^2) in LDS (its own 16 bytes a
// token, no barrier), so that no exponential is evaluated twice.  The input gate is
// kept as the pair of s and 1 - s (scan_gate.h): grad_gate_x has the factor 1 - s, which
// from s alone, or from b = s n, has no correct digit left behind gate_x = 17.  That and
// 1 / n taken again from n cost 4 % (223 to 232 us below); the exponential taken again from
// gate_x instead cost a little more, and spilled in fp32.
//
// With given decays it is bound by HBM (8 x 4096 x 2048: 944 MB of least traffic in
// 181 us).  Gated in bf16 (882 MB, x in 8 bits) it takes 232 us: about 75 vector
// instructions an element keep the vector units busy in two thirds of the cycles at
// two waves per SIMD (the registers' limit).  Before the gate was kept as a pair, four
// tokens a thread at four waves per SIMD took 249 us and workgroups that stay for further
// tiles 242, against 235 then.
//
// grad_decay_a sums over all tokens: registers, lane groups, waves (one LDS pass
// in a fixed order), then one partial row per tile that sum_kernel adds up, again
// in a fixed order.
#include "scan_gate.h"
#include "scan_tile.h"

namespace gdr {
namespace scan {

// The most that 1 / n counts as, n = sqrt(1 - a^2): that of n^2 = 2^-126, fp32's least
// normal number, so that the term that n^2 divides vanishes where n, and with it b x, is 0.
constexpr float kMostInv = 0x1p63f;

struct BwdP {
  int B, T, C, normalise;
  int nchain, nct, nt, team;
  const void* x;
  const uint8_t* x_exp;
  const float* alpha;
  const void* decay_x;
  const float* decay_a;
  const void* gate_x;
  const float* ckpt;
  const void* grad_y;
  const float* grad_h;
  void* grad_x;
  float* grad_alpha;
  void* grad_decay_x;
  void* grad_gate_x;
  float* grad_h0;
  float* part;       // [tiles of a chain * B][C] partial sums of grad_decay_a
  Chains ch;
};

template <typename T, typename X, int KIND, bool NORM, bool VEC>
__global__ __launch_bounds__(64 * kBwdWaves, 2) void scan_bwd_kernel(BwdP p) {
  constexpr bool kCodes = !__is_same(X, T);
  __shared__ Joins<kBwdWaves> j;   // of the maps of K: later tokens first
  constexpr int kKept = (KIND != 0 ? 1 : 0) + (NORM ? 1 : 0);   // sigmoid(decay_x), sqrt(1 - a^2)
  __shared__ f32x4 kept[kKept == 0 ? 1 : kKept][kKept == 0 ? 1 : S][kKept == 0 ? 1 : 64 * kBwdWaves];
  const Place q = take_place(p.C, p.nchain, p.nct, p.nt, p.team, p.ch.ticket);
  if (q.chain < 0) return;
  const int tile = p.nt - 1 - q.tt;         // the last tokens come first
  const int C = p.C, t0 = tile * kBwdWaves * GDR_SCAN_BLOCK;
  const int rows = min(q.nw * GDR_SCAN_BLOCK, p.T - t0);
  const int r0 = q.wave * GDR_SCAN_BLOCK + q.grp * S;
  const size_t base = ((size_t)q.b * p.T + t0) * C;
  const auto view = [&](auto t, const void* array) {
    return View<decltype(t), VEC>(array, base, rows, C, r0, q.c, q.nv);
  };

  // a wait for a load waits for those before it too: what is needed first comes
  // first, and row by row
  float scale[V];
  if constexpr (KIND != 0) {
    const Four<float>::R r = View<float, VEC>(p.decay_a, 0, 1, C, 0, q.c, q.nv).load(0);
#pragma unroll
    for (int k = 0; k < V; ++k) scale[k] = Four<float>::get(r, k);
  }
  typename Four<X>::R rx[S];
  typename Four<T>::R ry[S];
  Four<float>::R ra[KIND == 0 ? S : 1];
  typename Four<T>::R rd[KIND == 0 ? 1 : S], rg[KIND == 2 ? S : 1];
  float xs[kCodes ? S : 1];
  {
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
    if constexpr (kCodes) {
      const int ng = (C + 127) / 128;
      const rsrc_t be = buffer(p.x_exp + ((size_t)q.b * p.T + t0) * ng, rows * ng);
      const int oe = q.nv > 0 ? r0 * ng + q.c / 128 : kNoLane;
#pragma unroll
      for (int i = 0; i < S; ++i)
        xs[i] = chan::scale_of(__builtin_amdgcn_raw_buffer_load_b8(be, oe + i * ng, 0, 0));
    }
    const auto vy = view(T{}, p.grad_y);
#pragma unroll
    for (int i = 0; i < S; ++i) ry[i] = vy.load(i);
  }
  const size_t nb = blocks_of(p.T), block = (size_t)tile * kBwdWaves + q.wave;
  const Four<float>::R rh =
      View<float, VEC>(p.ckpt, ((size_t)q.b * nb + (block < nb ? block : 0)) * C, block < nb ? 1 : 0, C, 0, q.c, q.nv).load(0);
  const int cc = q.c0 + q.lane;
  const int pos = q.nw - 1 - q.wave;        // the wave's place in the order of joining
  const Words<kBwdWaves> words = look_ahead<kBwdWaves>(p.ch, q, p.nt, pos);
  float k_in = 0.f;
  if (q.wave == 0 && q.tt < kSuper && p.grad_h && cc < C) k_in = p.grad_h[(size_t)q.b * C + cc];

  // a and v = b x; (P, H) forwards and (P, Q) backwards over the thread's run
  float a[S][V], v[S][V], gate[KIND == 2 ? S : 1][V], sp[KIND == 0 ? 1 : S][V], P[V], H[V], Q[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    P[k] = 1.f;
    H[k] = Q[k] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < S; ++i) {
    f32x4 kd, kn;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      if constexpr (KIND == 0) {
        a[i][k] = Four<float>::get(ra[i], k);
      } else {
        const Scale A(scale[k]);
        float sig;
        sp[i][k] = softplus(Four<T>::get(rd[i], k), sig);
        kd[k] = sig;
        a[i][k] = decay(A, sp[i][k]);
        if constexpr (KIND == 2) gate[i][k] = gate_pair(Four<T>::get(rg[i], k));
        if constexpr (NORM) kn[k] = __builtin_amdgcn_sqrtf(one_minus_sq(A, sp[i][k], a[i][k]));   // as the forward has it
      }
    }
    if constexpr (KIND != 0) kept[0][i][threadIdx.x] = kd;
    if constexpr (NORM) kept[1][i][threadIdx.x] = kn;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      v[i][k] = Four<X>::get(rx[i], k);
      if constexpr (kCodes) v[i][k] *= xs[i];
      if constexpr (KIND == 2) {
        v[i][k] *= gate_open(gate[i][k]);
        forget(gate[i][k]);   // one register, not s beside it
      }
      if constexpr (NORM) v[i][k] *= kn[k];
    }
#pragma unroll
    for (int k = 0; k < V; ++k) {
      P[k] *= a[i][k];
      H[k] = fmaf(a[i][k], H[k], v[i][k]);
    }
  }
  // behind the last token the state stays: x and grad_y read as 0 there
  const bool ragged = rows < q.nw * GDR_SCAN_BLOCK;
  if (ragged) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      P[k] = 1.f;
      H[k] = 0.f;
#pragma unroll
      for (int i = 0; i < S; ++i) {
        if (r0 + i >= rows) a[i][k] = 1.f;
        P[k] *= a[i][k];
        H[k] = fmaf(a[i][k], H[k], v[i][k]);
      }
    }
  }
#pragma unroll
  for (int i = S - 1; i >= 0; --i)
#pragma unroll
    for (int k = 0; k < V; ++k) Q[k] = a[i][k] * (Four<T>::get(ry[i], k) + Q[k]);
  float h[V], Pb[V], Qb[V];
  {
    float Pf[V], Pe[V], He[V];
#pragma unroll
    for (int k = 0; k < V; ++k) Pf[k] = P[k];
    join_groups<true>(Pf, H, Pe, He, q.grp);
#pragma unroll
    for (int k = 0; k < V; ++k) h[k] = fmaf(Pe[k], Four<float>::get(rh, k), He[k]);   // the state before the run
  }
  join_groups<false>(P, Q, Pb, Qb, q.grp);
  if (q.grp == 0) {
#pragma unroll
    for (int k = 0; k < V; ++k) j.run[pos][q.cl + k] = float2{P[k], Q[k]};
  }
  float k_end;
  join_tiles(j, p.ch, q, words, p.nt, pos, k_in, k_end);
  if (p.grad_h0 && q.tt + 1 == p.nt && q.wave == 0 && cc < C) p.grad_h0[(size_t)q.b * C + cc] = k_end;
  float K[V];
#pragma unroll
  for (int k = 0; k < V; ++k) K[k] = fmaf(Pb[k], j.from[pos][q.cl + k], Qb[k]);
  const auto gx = view(T{}, p.grad_x);
  const auto ga = view(float{}, p.grad_alpha);
  const auto gd = view(T{}, p.grad_decay_x), gg = view(T{}, p.grad_gate_x);
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.f;
  // the states before each token are held for half of the run at a time
  constexpr int HS = S / 2;
#pragma unroll
  for (int half = 1; half >= 0; --half) {
    float prev[HS][V];
#pragma unroll
    for (int i = 0; i < (half + 1) * HS; ++i) {
      forget(ry[i]);
    }
    {
      float t[V];
#pragma unroll
      for (int k = 0; k < V; ++k) t[k] = h[k];
#pragma unroll
      for (int i = 0; i < (half + 1) * HS - 1; ++i)
#pragma unroll
        for (int k = 0; k < V; ++k) {
          if (i >= half * HS) prev[i - half * HS][k] = t[k];
          t[k] = fmaf(a[i][k], t[k], v[i][k]);
        }
#pragma unroll
      for (int k = 0; k < V; ++k) prev[HS - 1][k] = t[k];
    }
#pragma unroll
    for (int i = (half + 1) * HS - 1; i >= half * HS; --i) {
      float ox_[V], od[V], og[V];
      f32x4 kd, kn;
      if constexpr (KIND != 0) kd = kept[0][i][threadIdx.x];
      if constexpr (NORM) kn = kept[1][i][threadIdx.x];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float G = Four<T>::get(ry[i], k) + K[k];
        const float ak = a[i][k];
        K[k] = ak * G;
        if constexpr (KIND == 0) {
          ox_[k] = G;
          od[k] = G * prev[i - half * HS][k];
        } else {
          float in = -prev[i - half * HS][k];
          ox_[k] = G;
          if constexpr (KIND == 2) {
            ox_[k] *= gate_open(gate[i][k]);
            og[k] = G * v[i][k] * gate_shut(gate[i][k]);
          }
          if constexpr (NORM) {
            ox_[k] *= kn[k];
            const float inv = __builtin_fminf(__builtin_amdgcn_rcpf(kn[k]), kMostInv);
            in = fmaf(v[i][k] * inv, ak * inv, in);   // v a / m
          }
          float du = K[k] * in;
          if (ragged && r0 + i >= rows) du = 0.f;   // no part of grad_decay_a, also where the state is NaN
          sum[k] = fmaf(du, sp[i][k], sum[k]);
          od[k] = du * scale[k] * kd[k];
        }
      }
      gx.store(i, ox_);
      if constexpr (KIND == 0) ga.store(i, od);
      else gd.store(i, od);
      if constexpr (KIND == 2) gg.store(i, og);
    }
  }
  if constexpr (KIND != 0) {
#pragma unroll
    for (int dist = kSide; dist < 64; dist *= 2)
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += __shfl_xor(sum[k], dist);
    // a row of `from` has been read by its own wave alone
    if (q.grp == 0) {
#pragma unroll
      for (int k = 0; k < V; ++k) j.from[pos][q.cl + k] = sum[k];
    }
    __syncthreads();
    if (q.wave == 0 && cc < C) {
      float s = 0.f;
      for (int w = 0; w < q.nw; ++w) s += j.from[w][q.lane];
      p.part[((size_t)tile * p.B + q.b) * C + cc] = s;
    }
  }
}

// grad_decay_a[c]: 64 threads per channel take every 64th partial row, then join.
__global__ __launch_bounds__(1024) void sum_kernel(const float* part, float* out, int rows, int C) {
  __shared__ float s[64][17];
  const int l = threadIdx.x & 15, y = threadIdx.x >> 4, c = blockIdx.x * 16 + l;
  float t = 0.f;
  if (c < C)
    for (int r = y; r < rows; r += 64) t += part[(size_t)r * C + c];
  s[y][l] = t;
  __syncthreads();
  const int w = threadIdx.x >> 6, lane = threadIdx.x & 63;   // a wave joins a channel
  t = chan::lane_sum<64>(s[lane][w]);
  if (lane == 0 && blockIdx.x * 16 + w < C) out[blockIdx.x * 16 + w] = t;
}

static size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// The hand-over words of the recomputed forward, if there is one, then the
// backward's, its states and its partial sums.
static size_t recomputed_bytes(int B, int T, int C, bool ckpt) { return ckpt ? 0 : chain_bytes(B, T, C, kFwdWaves); }

size_t bwd_workspace(int B, int T, int C, bool gated, bool ckpt) {
  return recomputed_bytes(B, T, C, ckpt) + chain_bytes(B, T, C, kBwdWaves) +
         (ckpt ? 0 : align256((size_t)B * blocks_of(T) * C * 4)) + (gated ? align256(tiles_t(T, kBwdWaves) * B * C * 4) : 0);
}

template <typename T, typename X, int KIND, bool NORM>
static hipError_t launch_v(const BwdP& p, bool vec, hipStream_t s) {
  const int nw = p.nt > 1 ? kBwdWaves : (int)blocks_of(p.T);
  const dim3 grid((unsigned)((size_t)p.nchain * p.nt)), block(64 * nw);
  if (vec) hipLaunchKernelGGL((scan_bwd_kernel<T, X, KIND, NORM, true>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((scan_bwd_kernel<T, X, KIND, NORM, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, typename X>
static hipError_t launch_kind(const BwdP& p, bool vec, hipStream_t s) {
  if (p.alpha) return launch_v<T, X, 0, false>(p, vec, s);
  if (p.gate_x) return p.normalise ? launch_v<T, X, 2, true>(p, vec, s) : launch_v<T, X, 2, false>(p, vec, s);
  return p.normalise ? launch_v<T, X, 1, true>(p, vec, s) : launch_v<T, X, 1, false>(p, vec, s);
}

hipError_t launch_scan_bwd(const gdr_scan_bwd_args& a, hipStream_t s) {
  char* ws = (char*)a.workspace;
  const size_t first = recomputed_bytes(a.B, a.T, a.C, a.ckpt != nullptr), words = first + chain_bytes(a.B, a.T, a.C, kBwdWaves);
  char* rest = ws + words;
  hipError_t e = clear_chains(ws, words, s);
  if (e != hipSuccess) return e;
  const float* ckpt = a.ckpt;
  if (!ckpt) {
    e = launch_ckpt(a, (float*)rest, ws, s);
    if (e != hipSuccess) return e;
    ckpt = (const float*)rest;
    rest += align256((size_t)a.B * blocks_of(a.T) * a.C * 4);
  }
  BwdP p{a.B, a.T, a.C, a.normalise, (int)chains_of(a.B, a.C), (a.C + kTileC - 1) / kTileC, (int)tiles_t(a.T, kBwdWaves),
         team_of(a.alpha != nullptr, a.io_dtype), a.x, a.x_exp, a.alpha, a.decay_x, a.decay_a, a.gate_x, ckpt, a.grad_y, a.grad_h, a.grad_x, a.grad_alpha,
         a.grad_decay_x, a.grad_gate_x, a.grad_h0, (float*)rest,
         chains_at(ws + first, a.B, a.T, a.C, kBwdWaves)};
  const int rows = p.nt * a.B;
  if (rows == 1) p.part = a.grad_decay_a;   // one partial row is the sum
  const size_t io = a.io_dtype == GDR_BF16 ? 2 : 4;
  const bool vec = a.C % 4 == 0 && vec4_ok(a.x, a.x_exp ? 1 : io) && vec4_ok(a.alpha, 4) && vec4_ok(a.decay_x, io) &&
                   vec4_ok(a.gate_x, io) && vec4_ok(a.grad_y, io) && vec4_ok(a.grad_x, io) && vec4_ok(a.grad_alpha, 4) &&
                   vec4_ok(a.grad_decay_x, io) && vec4_ok(a.grad_gate_x, io);
  if (a.io_dtype == GDR_BF16)
    e = a.x_exp ? launch_kind<__bf16, Code8>(p, vec, s) : launch_kind<__bf16, __bf16>(p, vec, s);
  else
    e = a.x_exp ? launch_kind<float, Code8>(p, vec, s) : launch_kind<float, float>(p, vec, s);
  if (e != hipSuccess || a.alpha || rows == 1) return e;
  hipLaunchKernelGGL(sum_kernel, dim3((a.C + 15) / 16), dim3(1024), 0, s, p.part, a.grad_decay_a, rows, a.C);
  return hipGetLastError();
}

}  // namespace scan
}  // namespace gdr
