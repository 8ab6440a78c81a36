/* gdr_scan.h -- C ABI of the channelwise gated linear recurrence (gfx950):
 * forward, backward and single-token step.
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  It is the diagonal member of the family whose matrix-state members
 * are gdr_chunk_fwd and gdr_step_decode: each of C channels carries one number.
 *
 * Per batch row b, channel c and token t:
 *
 *     h_t = a_t h_{t-1} + b_t x_t,    y_t = h_t
 *
 *   alpha given:    a_t = alpha_t,  b_t = 1
 *   decay_x given:  u_t = decay_a[c] softplus(decay_x_t),  a_t = exp(-u_t),
 *                   b_t = [sigmoid(gate_x_t) if gate_x]
 *                         [sqrt(1 - a_t^2)   if normalise]
 * (the decay's form is the gated delta rule's, gdr_chunk_fwd_gated; with
 * normalise the state of a white input keeps its variance whatever the decay).
 *
 * Decays: alpha in [0, 1] and decay_a >= 0 are not checked.  A decay of 0
 * (alpha = 0, decay_x = +Inf) is an exact reset: it starts a new sequence packed
 * behind another.  alpha = 1 with x = 0, or decay_x = -Inf with normalise and a finite x,
 * leaves the state as it is (padding).  NaN, and Inf in x, h0 and the gradients, propagate
 * along their channel: what depends on them is not finite, through a reset (0 times Inf)
 * as well.  An Inf may come out as NaN: states pass on through products of many decays,
 * which may underflow.
 *
 * Sizes: any B, C and T >= 1 with B * T * C < 2^40, C <= 2^18 and
 * B * ceil(C/64) * ceil(T/128) < 2^23.  Every pointer is
 * aligned to its element; channels move 4 at a time, fastest where C is a multiple of 4
 * and the buffers are aligned to 4 elements.  Outputs overlap neither inputs nor
 * each other (GDR_ERR_ARG), except that h_out may equal h0 (and the step's
 * h_out its h).  All arithmetic and states are fp32; y and the gradients of the
 * activations are rounded once (RNE) to io_dtype; exponentials below fp32's least normal
 * number (of a pre-activation below -87) count as 0.  Results do not depend on
 * timing: no atomics add numbers.
 */
#ifndef GDR_SCAN_H
#define GDR_SCAN_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between two saved states (ckpt[b][j] is the state before token 32 j). */
#define GDR_SCAN_BLOCK 32

typedef struct gdr_scan_args {
  int32_t B, T, C;
  int32_t io_dtype;     /* gdr_dtype of x, decay_x, gate_x and y               */
  const void *x;        /* [B,T,C] io_dtype                                    */
  const float *alpha;   /* [B,T,C] fp32, or NULL: then decay_x and decay_a     */
  const void *decay_x;  /* [B,T,C] io_dtype                                    */
  const float *decay_a; /* [C] fp32                                            */
  const void *gate_x;   /* [B,T,C] io_dtype or NULL (only with decay_x)        */
  int32_t normalise;    /* 0 or 1 (1 only with decay_x)                        */
  int32_t reserved;     /* 0                                                   */
  const float *h0;      /* [B,C] fp32 start state, or NULL for zero            */
  void *y;              /* [B,T,C] io_dtype                                    */
  float *h_out;         /* [B,C] fp32 final state, or NULL; may equal h0       */
  float *ckpt;          /* [B,ceil(T/32),C] fp32 block-start states, or NULL   */
  void *workspace;      /* gdr_scan_fwd_workspace bytes, 16-byte aligned; its  */
  size_t workspace_bytes; /* contents need not be set and are not kept         */
} gdr_scan_args;

/* Bytes gdr_scan_fwd needs at `workspace` (0: none).  Also 0 for arguments that
 * gdr_scan_fwd refuses. */
size_t gdr_scan_fwd_workspace(const gdr_scan_args *args);

/* Forward on `stream`; GDR_ERR_* as in gdr.h, all checked before any HIP call.
 * Workgroups hand states to each other through the workspace, which the call clears
 * itself: it serves one call at a time (calls on one stream, or a graph replayed on
 * it, may share one). */
gdr_status gdr_scan_fwd(const gdr_scan_args *args, void *stream);

/* Gradients of a loss L through y and h_out.  With G_t = dL/dh_t (everything
 * that follows t included), G_t = grad_y_t + a_{t+1} G_{t+1}:
 *   grad_x = b G,  grad_alpha = G h_{t-1},  grad_h0 = a_1 G_1,
 *   grad_gate_x = G b x (1 - sigmoid(gate_x)),
 *   dL/du = G a (b x a / (1 - a^2) [if normalise] - h_{t-1}),
 *   grad_decay_x = dL/du decay_a sigmoid(decay_x),
 *   grad_decay_a = sum over (b, t) of dL/du softplus(decay_x).
 * 1 - sigmoid is formed without the difference, so grad_gate_x is accurate relative to
 * itself for open gates too (from gate_x = 87 on it counts as 2^-126).
 * b has the forward's own sqrt(1 - a^2).  Where 1 - a^2 is below fp32's least normal
 * number 2^-126, the quotient is taken with 2^63 for the inverse of that root, so it is 0
 * where the root is (the term vanishes with it; at decay_a = 0 it has no limit).
 * States inside a block of 32 tokens are computed again from ckpt (as
 * gdr_scan_fwd wrote it); without ckpt the whole recurrence is run again from
 * h0, and ckpt and h0 are not given together.  x may be 8-bit: then x_exp holds
 * the exponents of its groups (gdr_ckpt8.h), x is [B,T,C] codes and x_exp
 * [B,T,ceil(C/128)]. */
typedef struct gdr_scan_bwd_args {
  int32_t B, T, C;
  int32_t io_dtype;     /* gdr_dtype of x (unless x_exp), decay_x, gate_x,     */
                        /* grad_y, grad_x, grad_decay_x and grad_gate_x        */
  const void *x;
  const uint8_t *x_exp; /* NULL, or x is 8-bit codes                           */
  const float *alpha;
  const void *decay_x;
  const float *decay_a;
  const void *gate_x;
  int32_t normalise;
  int32_t reserved;
  const float *h0;      /* as the forward's; NULL with ckpt                    */
  const float *ckpt;    /* as the forward wrote it, or NULL                    */
  const void *grad_y;   /* [B,T,C] io_dtype                                    */
  const float *grad_h;  /* [B,C] fp32, or NULL for zero                        */
  void *grad_x;         /* [B,T,C] io_dtype                                    */
  float *grad_alpha;    /* [B,T,C] fp32 (with alpha), else NULL                */
  void *grad_decay_x;   /* [B,T,C] io_dtype (with decay_x), else NULL          */
  float *grad_decay_a;  /* [C] fp32 (with decay_x), else NULL                  */
  void *grad_gate_x;    /* [B,T,C] io_dtype (with gate_x), else NULL           */
  float *grad_h0;       /* [B,C] fp32, or NULL                                 */
  void *workspace;      /* gdr_scan_bwd_workspace bytes, 16-byte aligned       */
  size_t workspace_bytes;
} gdr_scan_bwd_args;

size_t gdr_scan_bwd_workspace(const gdr_scan_bwd_args *args);
gdr_status gdr_scan_bwd(const gdr_scan_bwd_args *args, void *stream);

/* One token on N states. */
typedef struct gdr_scan_step_args {
  int32_t N, C;         /* N * C < 2^31                                        */
  int32_t io_dtype;
  int32_t normalise;
  const void *x;        /* [N,C] io_dtype                                      */
  const float *alpha;   /* [N,C] fp32, or NULL                                 */
  const void *decay_x;  /* [N,C] io_dtype                                      */
  const float *decay_a; /* [C] fp32                                            */
  const void *gate_x;   /* [N,C] io_dtype, or NULL                             */
  const float *h;       /* [N,C] fp32                                          */
  float *h_out;         /* [N,C] fp32; may equal h                             */
  void *y;              /* [N,C] io_dtype                                      */
} gdr_scan_step_args;

gdr_status gdr_scan_step(const gdr_scan_step_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_SCAN_H */
