// ssm_api.cpp -- C ABI of the selective state space scan: argument checks, then the
// launch.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include "../../include/gdr_ssm.h"
#include "api_span.h"
#include "ssm_kernels.h"

namespace {

using gdr::Span;

gdr_status check_sizes(int B, int T, int C, int N, int G, int io_dtype, int softplus) {
  if (io_dtype != GDR_F32 && io_dtype != GDR_BF16) return GDR_ERR_DTYPE;
  if (B <= 0 || T <= 0 || C <= 0 || N <= 0 || G <= 0 || C % G != 0) return GDR_ERR_SHAPE;
  if (C > (1 << 18) || N > gdr::ssm::kMaxN || (long long)G * N > (1 << 16)) return GDR_ERR_UNSUPPORTED;
  const long long bt = (long long)B * T;   // < 2^62
  if (bt >= (1LL << 30) || bt >= (1LL << 40) / C) return GDR_ERR_SHAPE;
  return softplus == 0 || softplus == 1 ? GDR_OK : GDR_ERR_ARG;
}

gdr_status check_fwd(const gdr_ssm_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->B, a->T, a->C, a->N, a->G, a->io_dtype, a->softplus);
  if (st != GDR_OK) return st;
  if (gdr::ssm::too_many_chains(a->B, a->C, a->G)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->dt || !a->A || !a->Bv || !a->Cv || !a->y) return GDR_ERR_NULL;
  if (a->reserved != 0) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, bt = (size_t)a->B * a->T, c = (size_t)a->C, n = bt * c;
  const size_t cn = c * a->N, vec = bt * a->G * a->N;
  const Span in[] = {{a->h0, a->B * cn * 4, 4}, {a->x, n * io, io}, {a->dt, n * io, io}, {a->A, cn * 4, 4},
                     {a->Bv, vec * io, io}, {a->Cv, vec * io, io}, {a->D, c * 4, 4}, {a->z, n * io, io},
                     {a->dt_bias, c * 4, 4}, {a->lens, (size_t)a->B * 4, 4}};
  const Span out[] = {{a->h_out, a->B * cn * 4, 4}, {a->y, n * io, io},
                      {a->ckpt, a->B * gdr::ssm::blocks_of(a->T) * cn * 4, 4}, {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_bwd(const gdr_ssm_bwd_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->B, a->T, a->C, a->N, a->G, a->io_dtype, a->softplus);
  if (st != GDR_OK) return st;
  if (gdr::ssm::too_many_chains(a->B, a->C, a->G)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->dt || !a->A || !a->Bv || !a->Cv || !a->grad_y) return GDR_ERR_NULL;
  if (!a->grad_x || !a->grad_dt || !a->grad_A || !a->grad_Bv || !a->grad_Cv) return GDR_ERR_NULL;
  if (a->reserved != 0 || (a->ckpt && a->h0)) return GDR_ERR_ARG;
  // each optional input's gradient, and no other
  if ((a->D && !a->grad_D) || (a->z && !a->grad_z) || (a->dt_bias && !a->grad_dt_bias)) return GDR_ERR_NULL;
  if ((!a->D && a->grad_D) || (!a->z && a->grad_z) || (!a->dt_bias && a->grad_dt_bias)) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, bt = (size_t)a->B * a->T, c = (size_t)a->C, n = bt * c;
  const size_t cn = c * a->N, vec = bt * a->G * a->N;
  const Span in[] = {{a->x, n * io, io}, {a->dt, n * io, io}, {a->A, cn * 4, 4}, {a->Bv, vec * io, io},
                     {a->Cv, vec * io, io}, {a->D, c * 4, 4}, {a->z, n * io, io}, {a->dt_bias, c * 4, 4},
                     {a->h0, a->B * cn * 4, 4}, {a->ckpt, a->B * gdr::ssm::blocks_of(a->T) * cn * 4, 4},
                     {a->lens, (size_t)a->B * 4, 4}, {a->grad_y, n * io, io}, {a->grad_h, a->B * cn * 4, 4}};
  const Span out[] = {{a->grad_x, n * io, io}, {a->grad_dt, n * io, io}, {a->grad_A, cn * 4, 4},
                      {a->grad_Bv, vec * io, io}, {a->grad_Cv, vec * io, io}, {a->grad_D, c * 4, 4},
                      {a->grad_z, n * io, io}, {a->grad_dt_bias, c * 4, 4}, {a->grad_h0, a->B * cn * 4, 4},
                      {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_step(const gdr_ssm_step_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->R, 1, a->C, a->N, a->G, a->io_dtype, a->softplus);
  if (st != GDR_OK) return st;
  if ((long long)a->R * a->C * a->N >= (1LL << 31)) return GDR_ERR_SHAPE;   // R C < 2^40 by now
  if (!a->x || !a->dt || !a->A || !a->Bv || !a->Cv || !a->h || !a->h_out || !a->y) return GDR_ERR_NULL;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, c = (size_t)a->C, n = (size_t)a->R * c, cn = c * a->N;
  const size_t vec = (size_t)a->R * a->G * a->N;
  const Span in[] = {{a->h, a->R * cn * 4, 4}, {a->x, n * io, io}, {a->dt, n * io, io}, {a->A, cn * 4, 4},
                     {a->Bv, vec * io, io}, {a->Cv, vec * io, io}, {a->D, c * 4, 4}, {a->z, n * io, io},
                     {a->dt_bias, c * 4, 4}};
  const Span out[] = {{a->h_out, a->R * cn * 4, 4}, {a->y, n * io, io}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

}  // namespace

extern "C" {

size_t gdr_ssm_fwd_workspace(const gdr_ssm_args* a) {
  if (check_fwd(a) != GDR_OK) return 0;
  return gdr::ssm::fwd_workspace(a->B, a->T, a->C, a->N, a->G);
}

gdr_status gdr_ssm_fwd(const gdr_ssm_args* a, void* stream) {
  const gdr_status st = check_fwd(a);
  if (st != GDR_OK) return st;
  const size_t need = gdr::ssm::fwd_workspace(a->B, a->T, a->C, a->N, a->G);
  if (need && (!a->workspace || a->workspace_bytes < need)) return GDR_ERR_WORKSPACE;
  return done(gdr::ssm::launch_ssm_fwd(*a, static_cast<hipStream_t>(stream)));
}

size_t gdr_ssm_bwd_workspace(const gdr_ssm_bwd_args* a) {
  if (check_bwd(a) != GDR_OK) return 0;
  return gdr::ssm::bwd_workspace(a->B, a->T, a->C, a->N, a->G, a->ckpt != nullptr);
}

gdr_status gdr_ssm_bwd(const gdr_ssm_bwd_args* a, void* stream) {
  const gdr_status st = check_bwd(a);
  if (st != GDR_OK) return st;
  if (!a->workspace ||
      a->workspace_bytes < gdr::ssm::bwd_workspace(a->B, a->T, a->C, a->N, a->G, a->ckpt != nullptr))
    return GDR_ERR_WORKSPACE;
  return done(gdr::ssm::launch_ssm_bwd(*a, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_ssm_step(const gdr_ssm_step_args* a, void* stream) {
  const gdr_status st = check_step(a);
  if (st != GDR_OK) return st;
  return done(gdr::ssm::launch_ssm_step(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
