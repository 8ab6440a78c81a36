/* gdr_ssm.h -- C ABI of the selective state space scan (gfx950): forward, backward
 * and single-token step.
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  It stands between the channelwise recurrence (gdr_scan.h, one number a
 * channel) and the delta rule's matrix states: each of C channels has N numbers, driven
 * and read through vectors B_t and C_t that all channels of a group share.  Per batch
 * row, channel c of group g and token t:
 *
 *     d_t = softplus(dt_t + dt_bias) (without softplus: dt_t + dt_bias)
 *     h_t[n] = exp(d_t A[c][n]) h_{t-1}[n] + d_t x_t B_t[g][n]
 *     u_t = sum over n of C_t[g][n] h_t[n] + D[c] x_t
 *     y_t = u_t z_t sigmoid(z_t) with z, else u_t
 *
 * Channels of a group are neighbours: channel c belongs to group c / (C / G).  A <= 0
 * is the stable case and not checked; its values are held to [-2^64, 2^64], so that -Inf,
 * or fp32's lowest value, is a state that every time step from 2^-56 on resets.
 *
 * A batch may be padded: row b has lens[b] tokens (its value is held to [0, T]), NULL
 * means T.  Tokens behind them are not read; their y and gradients are 0, the state
 * stays what it is, and so do the saved states there.
 *
 * Sizes: 1 <= N <= 64, C a multiple of G, C <= 2^18, G * N <= 2^16, any B and T >= 1
 * with B * T < 2^30, B * T * C < 2^40 and B * G * ceil(C/G/64) < 2^22.  Every pointer is
 * aligned to its element.  Outputs overlap neither inputs nor each other (GDR_ERR_ARG),
 * except that h_out may equal h0 (and the step's h_out its h).  All arithmetic and states
 * are fp32; y and the gradients of io_dtype are rounded once (RNE); exponentials below
 * fp32's least normal number count as 0.  Sums run in an order that the sizes fix: no atomics
 * add numbers.  NaN propagates along its channel (in the backward also to the gradients
 * of the vectors and of A, D and dt_bias that it enters); an Inf may come out as NaN.
 */
#ifndef GDR_SSM_H
#define GDR_SSM_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between two saved states (ckpt[b][j] is the state before token 32 j). */
#define GDR_SSM_BLOCK 32

typedef struct gdr_ssm_args {
  int32_t B, T, C, N, G;
  int32_t io_dtype;     /* gdr_dtype of x, dt, Bv, Cv, z and y                 */
  int32_t softplus;     /* 0 or 1                                              */
  int32_t reserved;     /* 0                                                   */
  const void *x;        /* [B,T,C] io_dtype                                    */
  const void *dt;       /* [B,T,C] io_dtype                                    */
  const float *A;       /* [C,N] fp32                                          */
  const void *Bv;       /* [B,T,G,N] io_dtype                                  */
  const void *Cv;       /* [B,T,G,N] io_dtype                                  */
  const float *D;       /* [C] fp32, or NULL for zeros                         */
  const void *z;        /* [B,T,C] io_dtype, or NULL: no gate                  */
  const float *dt_bias; /* [C] fp32, or NULL for zeros                         */
  const float *h0;      /* [B,C,N] fp32 start state, or NULL for zero          */
  const int32_t *lens;  /* [B], or NULL for T                                  */
  void *y;              /* [B,T,C] io_dtype                                    */
  float *h_out;         /* [B,C,N] fp32 final state, or NULL; may equal h0     */
  float *ckpt;          /* [B,ceil(T/32),N,C] fp32 block-start states, or NULL */
  void *workspace;      /* gdr_ssm_fwd_workspace bytes, 16-byte aligned; its   */
  size_t workspace_bytes; /* contents need not be set and are not kept         */
} gdr_ssm_args;

/* Bytes gdr_ssm_fwd needs at `workspace` (0: none, or refused arguments); a
 * workspace serves one call at a time (calls on one stream, or a graph replayed on it,
 * may share one). */
size_t gdr_ssm_fwd_workspace(const gdr_ssm_args *args);
gdr_status gdr_ssm_fwd(const gdr_ssm_args *args, void *stream);

/* Gradients of a loss through y and h_out.  With g_t = dL/du_t (grad_y_t, times
 * z sigmoid(z) with z), s = sigmoid, a_t = exp(d_t A) and H_t = dL/dh_t:
 *   H_t = C_t g_t + a_{t+1} H_{t+1},   q_t = H_t a_t h_{t-1},   p_t = sum over n of B_t H_t
 *   grad_x  = d p + D g,               grad_Bv = sum over the group's channels of H d x,
 *   grad_dt = (sum over n of A q + x p) s(dt + dt_bias) (that slope only with softplus),
 *   grad_Cv = sum over the group's channels of g h,     grad_A = sum over (b, t) of d q,
 *   grad_z  = grad_y u s(z) (1 + z (1 - s(z))),         grad_D = sum over (b, t) of g x,
 *   grad_dt_bias = sum over (b, t) of grad_dt,          grad_h0 = a_1 H_1.
 * States inside a block of 32 tokens are computed again from ckpt (as gdr_ssm_fwd
 * wrote it); without ckpt the whole recurrence is run again from h0, and ckpt and h0
 * are not given together. */
typedef struct gdr_ssm_bwd_args {
  int32_t B, T, C, N, G;
  int32_t io_dtype;     /* gdr_dtype of the forward's, grad_y and the          */
                        /* gradients of x, dt, Bv, Cv and z                    */
  int32_t softplus;
  int32_t reserved;     /* 0                                                   */
  const void *x;
  const void *dt;
  const float *A;
  const void *Bv;
  const void *Cv;
  const float *D;
  const void *z;
  const float *dt_bias;
  const float *h0;      /* as the forward's; NULL with ckpt                    */
  const float *ckpt;    /* as the forward wrote it, or NULL                    */
  const int32_t *lens;
  const void *grad_y;   /* [B,T,C] io_dtype                                    */
  const float *grad_h;  /* [B,C,N] fp32, or NULL for zero                      */
  void *grad_x;         /* [B,T,C] io_dtype                                    */
  void *grad_dt;        /* [B,T,C] io_dtype                                    */
  float *grad_A;        /* [C,N] fp32                                          */
  void *grad_Bv;        /* [B,T,G,N] io_dtype                                  */
  void *grad_Cv;        /* [B,T,G,N] io_dtype                                  */
  float *grad_D;        /* [C] fp32 (with D), else NULL                        */
  void *grad_z;         /* [B,T,C] io_dtype (with z), else NULL                */
  float *grad_dt_bias;  /* [C] fp32 (with dt_bias), else NULL                  */
  float *grad_h0;       /* [B,C,N] fp32, or NULL                               */
  void *workspace;      /* gdr_ssm_bwd_workspace bytes, 16-byte aligned        */
  size_t workspace_bytes;
} gdr_ssm_bwd_args;

size_t gdr_ssm_bwd_workspace(const gdr_ssm_bwd_args *args);
gdr_status gdr_ssm_bwd(const gdr_ssm_bwd_args *args, void *stream);

/* One token on R states: R * C * N < 2^31. */
typedef struct gdr_ssm_step_args {
  int32_t R, C, N, G;
  int32_t io_dtype;
  int32_t softplus;
  const void *x;        /* [R,C] io_dtype                                      */
  const void *dt;       /* [R,C] io_dtype                                      */
  const float *A;       /* [C,N] fp32                                          */
  const void *Bv;       /* [R,G,N] io_dtype                                    */
  const void *Cv;       /* [R,G,N] io_dtype                                    */
  const float *D;       /* [C] fp32, or NULL                                   */
  const void *z;        /* [R,C] io_dtype, or NULL                             */
  const float *dt_bias; /* [C] fp32, or NULL                                   */
  const float *h;       /* [R,C,N] fp32                                        */
  float *h_out;         /* [R,C,N] fp32; may equal h                           */
  void *y;              /* [R,C] io_dtype                                      */
} gdr_ssm_step_args;

gdr_status gdr_ssm_step(const gdr_ssm_step_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_SSM_H */
