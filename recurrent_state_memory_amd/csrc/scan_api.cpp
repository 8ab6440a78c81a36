// scan_api.cpp -- C ABI of the channelwise recurrence: argument checks, then the
// launch.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include "../../include/gdr_ckpt8.h"
#include "../../include/gdr_scan.h"
#include "api_span.h"
#include "scan_kernels.h"

namespace {

using gdr::Span;

gdr_status check_sizes(int B, int T, int C, int io_dtype) {
  if (io_dtype != GDR_F32 && io_dtype != GDR_BF16) return GDR_ERR_DTYPE;
  if (B <= 0 || T <= 0 || C <= 0) return GDR_ERR_SHAPE;
  if (C > (1 << 18)) return GDR_ERR_UNSUPPORTED;
  const long long bt = (long long)B * T;   // < 2^62
  if (bt >= (1LL << 31) || bt >= (1LL << 40) / C) return GDR_ERR_SHAPE;
  return GDR_OK;
}

// alpha, or decay_x with decay_a; gate_x and normalise only with the latter.
gdr_status check_decay(const float* alpha, const void* decay_x, const float* decay_a, const void* gate_x,
                       int normalise) {
  if (normalise != 0 && normalise != 1) return GDR_ERR_ARG;
  if (alpha) return decay_x || decay_a || gate_x || normalise ? GDR_ERR_ARG : GDR_OK;
  return decay_x && decay_a ? GDR_OK : GDR_ERR_NULL;
}

gdr_status check_fwd(const gdr_scan_args* a) {
  if (!a) return GDR_ERR_NULL;
  gdr_status st = check_sizes(a->B, a->T, a->C, a->io_dtype);
  if (st != GDR_OK) return st;
  if (gdr::scan::too_many_tiles(a->B, a->T, a->C)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->y) return GDR_ERR_NULL;
  if (a->reserved != 0) return GDR_ERR_ARG;
  st = check_decay(a->alpha, a->decay_x, a->decay_a, a->gate_x, a->normalise);
  if (st != GDR_OK) return st;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->B * a->T * a->C, bc = (size_t)a->B * a->C;
  const Span in[] = {{a->h0, bc * 4, 4}, {a->x, n * io, io}, {a->alpha, n * 4, 4}, {a->decay_x, n * io, io},
                     {a->decay_a, (size_t)a->C * 4, 4}, {a->gate_x, n * io, io}};
  const Span out[] = {{a->h_out, bc * 4, 4}, {a->y, n * io, io},
                      {a->ckpt, (size_t)a->B * gdr::scan::blocks_of(a->T) * a->C * 4, 4},
                      {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_bwd(const gdr_scan_bwd_args* a) {
  if (!a) return GDR_ERR_NULL;
  gdr_status st = check_sizes(a->B, a->T, a->C, a->io_dtype);
  if (st != GDR_OK) return st;
  if (gdr::scan::too_many_tiles(a->B, a->T, a->C)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->grad_y || !a->grad_x) return GDR_ERR_NULL;
  if (a->reserved != 0) return GDR_ERR_ARG;
  st = check_decay(a->alpha, a->decay_x, a->decay_a, a->gate_x, a->normalise);
  if (st != GDR_OK) return st;
  if (a->ckpt && a->h0) return GDR_ERR_ARG;
  // each input's gradient, and no other
  if (a->alpha ? !a->grad_alpha : !a->grad_decay_x || !a->grad_decay_a) return GDR_ERR_NULL;
  if (a->gate_x && !a->grad_gate_x) return GDR_ERR_NULL;
  if (a->alpha ? a->grad_decay_x || a->grad_decay_a : a->grad_alpha != nullptr) return GDR_ERR_ARG;
  if (!a->gate_x && a->grad_gate_x) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->B * a->T * a->C, bc = (size_t)a->B * a->C;
  const size_t xs = a->x_exp ? 1 : io, groups = ((size_t)a->C + GDR_CKPT8_GROUP - 1) / GDR_CKPT8_GROUP;
  const Span in[] = {{a->x, n * xs, xs}, {a->x_exp, (size_t)a->B * a->T * groups, 1}, {a->alpha, n * 4, 4},
                     {a->decay_x, n * io, io}, {a->decay_a, (size_t)a->C * 4, 4}, {a->gate_x, n * io, io},
                     {a->h0, bc * 4, 4}, {a->ckpt, (size_t)a->B * gdr::scan::blocks_of(a->T) * a->C * 4, 4},
                     {a->grad_y, n * io, io}, {a->grad_h, bc * 4, 4}};
  const Span out[] = {{a->grad_x, n * io, io}, {a->grad_alpha, n * 4, 4}, {a->grad_decay_x, n * io, io},
                      {a->grad_decay_a, (size_t)a->C * 4, 4}, {a->grad_gate_x, n * io, io}, {a->grad_h0, bc * 4, 4},
                      {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_step(const gdr_scan_step_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->N, 1, a->C, a->io_dtype);
  if (st != GDR_OK) return st;
  if ((long long)a->N * a->C >= (1LL << 31)) return GDR_ERR_SHAPE;
  if (!a->x || !a->h || !a->h_out || !a->y) return GDR_ERR_NULL;
  const gdr_status sd = check_decay(a->alpha, a->decay_x, a->decay_a, a->gate_x, a->normalise);
  if (sd != GDR_OK) return sd;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->N * a->C;
  const Span in[] = {{a->h, n * 4, 4}, {a->x, n * io, io}, {a->alpha, n * 4, 4}, {a->decay_x, n * io, io},
                     {a->decay_a, (size_t)a->C * 4, 4}, {a->gate_x, n * io, io}};
  const Span out[] = {{a->h_out, n * 4, 4}, {a->y, n * io, io}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

}  // namespace

extern "C" {

size_t gdr_scan_fwd_workspace(const gdr_scan_args* a) {
  if (check_fwd(a) != GDR_OK) return 0;
  return gdr::scan::fwd_workspace(a->B, a->T, a->C);
}

gdr_status gdr_scan_fwd(const gdr_scan_args* a, void* stream) {
  const gdr_status st = check_fwd(a);
  if (st != GDR_OK) return st;
  const size_t need = gdr::scan::fwd_workspace(a->B, a->T, a->C);
  if (need && (!a->workspace || a->workspace_bytes < need)) return GDR_ERR_WORKSPACE;
  return done(gdr::scan::launch_scan_fwd(*a, static_cast<hipStream_t>(stream)));
}

size_t gdr_scan_bwd_workspace(const gdr_scan_bwd_args* a) {
  if (check_bwd(a) != GDR_OK) return 0;
  return gdr::scan::bwd_workspace(a->B, a->T, a->C, a->alpha == nullptr, a->ckpt != nullptr);
}

gdr_status gdr_scan_bwd(const gdr_scan_bwd_args* a, void* stream) {
  const gdr_status st = check_bwd(a);
  if (st != GDR_OK) return st;
  const size_t need = gdr::scan::bwd_workspace(a->B, a->T, a->C, a->alpha == nullptr, a->ckpt != nullptr);
  if (need && (!a->workspace || a->workspace_bytes < need)) return GDR_ERR_WORKSPACE;
  return done(gdr::scan::launch_scan_bwd(*a, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_scan_step(const gdr_scan_step_args* a, void* stream) {
  const gdr_status st = check_step(a);
  if (st != GDR_OK) return st;
  return done(gdr::scan::launch_scan_step(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
