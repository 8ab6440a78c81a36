// conv_api.cpp -- C ABI of the short causal convolution: argument checks, then the
// launch.  Every check runs on the host before any HIP call.
#include <hip/hip_runtime.h>

#include "../../include/gdr_conv.h"
#include "api_span.h"
#include "conv_kernels.h"

namespace {

using gdr::Span;

gdr_status check_sizes(int B, int T, int C, int K, int io_dtype, int silu) {
  if (io_dtype != GDR_F32 && io_dtype != GDR_BF16) return GDR_ERR_DTYPE;
  if (B <= 0 || T <= 0 || C <= 0 || K <= 0) return GDR_ERR_SHAPE;
  if (K < gdr::conv::kMinK || K > gdr::conv::kMaxK || C > (1 << 18)) return GDR_ERR_UNSUPPORTED;
  const long long bt = (long long)B * T;   // < 2^62
  if (bt >= (1LL << 30) || bt >= (1LL << 40) / C) return GDR_ERR_SHAPE;
  return silu == 0 || silu == 1 ? GDR_OK : GDR_ERR_ARG;
}

gdr_status check_fwd(const gdr_conv_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->B, a->T, a->C, a->K, a->io_dtype, a->silu);
  if (st != GDR_OK) return st;
  if (gdr::conv::too_many_tiles(a->B, a->T, a->C)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->weight || !a->y) return GDR_ERR_NULL;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->B * a->T * a->C, c = (size_t)a->C;
  const size_t edge = (size_t)a->B * (a->K - 1) * c;
  const Span in[] = {{a->state, edge * io, io}, {a->x, n * io, io}, {a->weight, c * a->K * 4, 4}, {a->bias, c * 4, 4},
                     {a->lens, (size_t)a->B * 4, 4}};
  const Span out[] = {{a->state_out, edge * io, io}, {a->y, n * io, io}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_bwd(const gdr_conv_bwd_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->B, a->T, a->C, a->K, a->io_dtype, a->silu);
  if (st != GDR_OK) return st;
  if (gdr::conv::too_many_tiles(a->B, a->T, a->C)) return GDR_ERR_UNSUPPORTED;
  if (!a->x || !a->weight || !a->grad_y || !a->grad_x || !a->grad_weight) return GDR_ERR_NULL;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->B * a->T * a->C, c = (size_t)a->C;
  const size_t edge = (size_t)a->B * (a->K - 1) * c;
  const Span in[] = {{a->x, n * io, io}, {a->weight, c * a->K * 4, 4}, {a->bias, c * 4, 4}, {a->state, edge * io, io},
                     {a->lens, (size_t)a->B * 4, 4}, {a->grad_y, n * io, io}, {a->grad_state_out, edge * io, io}};
  const Span out[] = {{a->grad_x, n * io, io}, {a->grad_weight, c * a->K * 4, 4}, {a->grad_bias, c * 4, 4},
                      {a->grad_state, edge * io, io}, {a->workspace, a->workspace_bytes, 16}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status check_step(const gdr_conv_step_args* a) {
  if (!a) return GDR_ERR_NULL;
  const gdr_status st = check_sizes(a->N, 1, a->C, a->K, a->io_dtype, a->silu);
  if (st != GDR_OK) return st;
  if ((long long)a->N * a->C * (a->K - 1) >= (1LL << 31)) return GDR_ERR_SHAPE;   // N C < 2^40 by now
  if (!a->x || !a->weight || !a->state || !a->state_out || !a->y) return GDR_ERR_NULL;
  if (a->reserved != 0) return GDR_ERR_ARG;
  const size_t io = a->io_dtype == GDR_BF16 ? 2 : 4, n = (size_t)a->N * a->C, c = (size_t)a->C;
  const Span in[] = {{a->state, n * (a->K - 1) * io, io}, {a->x, n * io, io}, {a->weight, c * a->K * 4, 4},
                     {a->bias, c * 4, 4}};
  const Span out[] = {{a->state_out, n * (a->K - 1) * io, io}, {a->y, n * io, io}};
  if (!gdr::spans_aligned(in, out)) return GDR_ERR_ALIGN;
  if (!gdr::spans_apart(in, out, 0, 0)) return GDR_ERR_ARG;
  return GDR_OK;
}

gdr_status done(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_ERR_HIP; }

}  // namespace

extern "C" {

gdr_status gdr_conv_fwd(const gdr_conv_args* a, void* stream) {
  const gdr_status st = check_fwd(a);
  if (st != GDR_OK) return st;
  return done(gdr::conv::launch_conv_fwd(*a, static_cast<hipStream_t>(stream)));
}

size_t gdr_conv_bwd_workspace(const gdr_conv_bwd_args* a) {
  if (check_bwd(a) != GDR_OK) return 0;
  return gdr::conv::bwd_workspace(a->B, a->T, a->C, a->K);
}

gdr_status gdr_conv_bwd(const gdr_conv_bwd_args* a, void* stream) {
  const gdr_status st = check_bwd(a);
  if (st != GDR_OK) return st;
  if (!a->workspace || a->workspace_bytes < gdr::conv::bwd_workspace(a->B, a->T, a->C, a->K))
    return GDR_ERR_WORKSPACE;
  return done(gdr::conv::launch_conv_bwd(*a, static_cast<hipStream_t>(stream)));
}

gdr_status gdr_conv_step(const gdr_conv_step_args* a, void* stream) {
  const gdr_status st = check_step(a);
  if (st != GDR_OK) return st;
  return done(gdr::conv::launch_conv_step(*a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
