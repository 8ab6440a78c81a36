// norm_api.cpp -- C ABI of the layer norm and the 8-bit checkpoints: argument
// checks, then the launch.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include <cmath>

#include "../../include/gdr_ckpt8.h"
#include "../../include/gdr_norm.h"
#include "api_span.h"
#include "norm_kernels.h"

namespace {

using gdr::Span;

gdr_status check_rows(int64_t R, int D, int io_dtype, int most_d) {
  if (io_dtype != GDR_F32 && io_dtype != GDR_BF16) return GDR_ERR_DTYPE;
  if (R <= 0 || D <= 0) return GDR_ERR_SHAPE;
  if (D > most_d) return GDR_ERR_UNSUPPORTED;
  if (R >= (1LL << 31) || R >= (1LL << 40) / D) return GDR_ERR_SHAPE;
  return GDR_OK;
}

size_t groups_of(int D) { return ((size_t)D + GDR_CKPT8_GROUP - 1) / GDR_CKPT8_GROUP; }

gdr_status check_norm(const gdr_norm_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_rows(a->R, a->D, a->io_dtype, 65536);
  if (st != GDR_OK) return st;
  if (!a->x || !a->y) return GDR_ERR_NULL;
  if ((a->x_code != nullptr) != (a->x_exp != nullptr)) return GDR_ERR_NULL;
  if (a->reserved != 0 || !std::isfinite(a->eps) || a->eps < 0.f) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->R * a->D, r = (size_t)a->R, d = (size_t)a->D;
  const Span in[] = {{a->x, n * io, io}, {a->weight, d * 4, 4}, {a->bias, d * 4, 4}};
  const Span out[] = {{a->y, n * io, io}, {a->mean, r * 4, 4}, {a->rstd, r * 4, 4}, {a->x_code, n, 1},
                      {a->x_exp, r * groups_of(a->D), 1}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_norm_bwd(const gdr_norm_bwd_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_rows(a->R, a->D, a->io_dtype, 65536);
  if (st != GDR_OK) return st;
  if (!a->x || !a->mean || !a->rstd || !a->grad_y || !a->grad_x) return GDR_ERR_NULL;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->R * a->D, r = (size_t)a->R, d = (size_t)a->D;
  const size_t xs = a->x_exp ? 1 : io;
  const Span in[] = {{a->x, n * xs, xs}, {a->x_exp, r * groups_of(a->D), 1}, {a->mean, r * 4, 4},
                     {a->rstd, r * 4, 4}, {a->weight, d * 4, 4}, {a->grad_y, n * io, io}};
  const Span out[] = {{a->grad_x, n * io, io}, {a->grad_weight, d * 4, 4}, {a->grad_bias, d * 4, 4},
                      {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

// The columns' sums pass through the workspace; none is needed without them.
size_t norm_bwd_need(const gdr_norm_bwd_args* a) {
  return a->grad_weight || a->grad_bias ? gdr::norm::bwd_workspace(a->R, a->D) : 0;
}

gdr_status check_ckpt8(int64_t R, int D, int io_dtype, const void* in_p, const void* code, const void* exp,
                       const void* out_p) {
  const gdr_status st = check_rows(R, D, io_dtype, 1 << 30);
  if (st != GDR_OK) return st;
  if (!code || !exp || (!in_p && !out_p)) return GDR_ERR_NULL;
  const size_t io = io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)R * D;
  const Span x{in_p ? in_p : out_p, n * io, io}, c{code, n, 1}, e{exp, (size_t)R * groups_of(D), 1};
  if (!gdr::aligned_to(x.p, io)) return GDR_ERR_ALIGN;
  if (gdr::spans_clash(x, c) || gdr::spans_clash(x, e)) return GDR_ERR_ARG;
  if (in_p && gdr::spans_clash(c, e)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

}  // namespace

extern "C" {

gdr_status gdr_norm_fwd(const gdr_norm_args* a, void* stream) {
  const gdr_status st = check_norm(a);
  if (st != GDR_OK) return st;
  return done(gdr::norm::launch_norm_fwd(*a, static_cast<hipStream_t>(stream)));
}

size_t gdr_norm_bwd_workspace(const gdr_norm_bwd_args* a) {
  if (check_norm_bwd(a) != GDR_OK) return 0;
  return norm_bwd_need(a);
}

gdr_status gdr_norm_bwd(const gdr_norm_bwd_args* a, void* stream) {
  const gdr_status st = check_norm_bwd(a);
  if (st != GDR_OK) return st;
  const size_t need = norm_bwd_need(a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return GDR_ERR_WORKSPACE;
  return done(gdr::norm::launch_norm_bwd(*a, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_ckpt8_pack(const gdr_ckpt8_pack_args* a, void* stream) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_ckpt8(a->R, a->D, a->io_dtype, a->x, a->code, a->exp, nullptr);
  if (st != GDR_OK) return st;
  return done(gdr::ckpt8::launch_pack(*a, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_ckpt8_unpack(const gdr_ckpt8_unpack_args* a, void* stream) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_ckpt8(a->R, a->D, a->io_dtype, nullptr, a->code, a->exp, a->x);
  if (st != GDR_OK) return st;
  return done(gdr::ckpt8::launch_unpack(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
