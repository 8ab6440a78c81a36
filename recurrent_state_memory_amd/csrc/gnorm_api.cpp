// gnorm_api.cpp -- C ABI of the gated group norm: argument checks, then the launch.
// Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/gdr_gnorm.h"
#include "api_span.h"
#include "gnorm_kernels.h"

namespace {

using gdr::Span;

gdr_status check_sizes(int64_t R, int C, int G, int io_dtype) {
  if (io_dtype != GDR_F32 && io_dtype != GDR_BF16) return GDR_ERR_DTYPE;
  if (R <= 0 || C <= 0 || G <= 0 || C % G != 0) return GDR_ERR_SHAPE;
  if (C > (1 << 20) || C / G > gdr::gnorm::kMaxGroup) return GDR_ERR_UNSUPPORTED;
  if (R >= (1LL << 31) || R * G >= (1LL << 31) || R >= (1LL << 40) / C) return GDR_ERR_SHAPE;
  return GDR_OK;
}

gdr_status check_fwd(const gdr_gnorm_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->R, a->C, a->G, a->io_dtype);
  if (st != GDR_OK) return st;
  if (!a->x || !a->y) return GDR_ERR_NULL;
  if ((a->center != 0 && a->center != 1) || (a->silu != 0 && a->silu != 1)) return GDR_ERR_ARG;
  if (!std::isfinite(a->eps) || a->eps < 0.f || (a->mean && !a->center)) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->R * a->C, c = (size_t)a->C;
  const size_t rg = (size_t)a->R * a->G;
  const Span in[] = {{a->x, n * io, io}, {a->z, n * io, io}, {a->weight, c * 4, 4}, {a->bias, c * 4, 4}};
  const Span out[] = {{a->y, n * io, io}, {a->mean, rg * 4, 4}, {a->rstd, rg * 4, 4}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_bwd(const gdr_gnorm_bwd_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->R, a->C, a->G, a->io_dtype);
  if (st != GDR_OK) return st;
  if (!a->x || !a->rstd || !a->grad_y || !a->grad_x) return GDR_ERR_NULL;
  if (a->z && !a->grad_z) return GDR_ERR_NULL;
  if ((!a->z && a->grad_z) || (a->silu != 0 && a->silu != 1)) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->R * a->C, c = (size_t)a->C;
  const size_t rg = (size_t)a->R * a->G;
  const Span in[] = {{a->x, n * io, io}, {a->z, n * io, io}, {a->mean, rg * 4, 4}, {a->rstd, rg * 4, 4},
                     {a->weight, c * 4, 4}, {a->bias, c * 4, 4}, {a->grad_y, n * io, io}};
  const Span out[] = {{a->grad_x, n * io, io}, {a->grad_z, n * io, io}, {a->grad_weight, c * 4, 4},
                      {a->grad_bias, c * 4, 4}, {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

// The columns' sums pass through the workspace; none is needed without them.
size_t bwd_need(const gdr_gnorm_bwd_args* a) {
  return a->grad_weight || a->grad_bias ? gdr::gnorm::bwd_workspace(a->R, a->C, a->G, a->io_dtype) : 0;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

}  // namespace

extern "C" {

gdr_status gdr_gnorm_fwd(const gdr_gnorm_args* a, void* stream) {
  const gdr_status st = check_fwd(a);
  if (st != GDR_OK) return st;
  return done(gdr::gnorm::launch_gnorm_fwd(*a, static_cast<hipStream_t>(stream)));
}

size_t gdr_gnorm_bwd_workspace(const gdr_gnorm_bwd_args* a) {
  if (check_bwd(a) != GDR_OK) return 0;
  return bwd_need(a);
}

gdr_status gdr_gnorm_bwd(const gdr_gnorm_bwd_args* a, void* stream) {
  const gdr_status st = check_bwd(a);
  if (st != GDR_OK) return st;
  const size_t need = bwd_need(a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return GDR_ERR_WORKSPACE;
  return done(gdr::gnorm::launch_gnorm_bwd(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
