/* gdr_conv.h -- C ABI of the short causal convolution (gfx950): forward, backward
 * and single-token step.
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  It is what a recurrent layer puts ahead of its recurrence: each channel
 * sees its own last K tokens,
 *
 *     u_t = bias + sum over j < K of weight[c][j] x_{t-K+1+j},
 *     y_t = u_t sigmoid(u_t) if silu, else u_t
 *
 * where the K - 1 tokens before a row's first are those of `state`, oldest first
 * (zero without it), and state_out holds the last K - 1 of the row, so that calls
 * on consecutive pieces of a sequence give what one call on all of it gives.
 *
 * A batch may be padded: row b has lens[b] tokens (its value is held to [0, T]), NULL
 * means T.  Tokens behind them are not read; their y and gradients are 0, and a row of
 * length 0 passes its state on.
 *
 * Sizes: 2 <= K <= 8, 1 <= C <= 2^18, any B and T >= 1 with B * T < 2^30, B * T * C < 2^40
 * and B * ceil(C/256) * ceil(T/256) < 2^22.  Every pointer is aligned to its element;
 * channels move 16 bytes at a time, fastest where rows begin at multiples of 16 bytes.
 * Outputs overlap neither inputs nor each other (GDR_ERR_ARG), except that state_out may
 * equal state.  All arithmetic is fp32; y, grad_x and grad_state are rounded once (RNE) to
 * io_dtype, states are copied.  The sums of grad_weight and grad_bias run in an order that
 * the sizes fix.  NaN and Inf stay within the K tokens of their channel that they reach
 * (backward: x through silu's slope reaches grad_x of K - 1 tokens on either side), and
 * grad_weight and grad_bias of that channel.
 */
#ifndef GDR_CONV_H
#define GDR_CONV_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdr_conv_args {
  int32_t B, T, C, K;
  int32_t io_dtype;     /* gdr_dtype of x, state, y and state_out              */
  int32_t silu;         /* 0 or 1                                              */
  const void *x;        /* [B,T,C] io_dtype                                    */
  const float *weight;  /* [C,K] fp32; weight[c][K-1] meets the token itself   */
  const float *bias;    /* [C] fp32, or NULL for zeros                         */
  const void *state;    /* [B,K-1,C] io_dtype, or NULL for zeros               */
  const int32_t *lens;  /* [B], or NULL for T                                  */
  void *y;              /* [B,T,C] io_dtype                                    */
  void *state_out;      /* [B,K-1,C] io_dtype, or NULL; may equal state        */
} gdr_conv_args;

gdr_status gdr_conv_fwd(const gdr_conv_args *args, void *stream);

/* Gradients of a loss through y and state_out.  With d_t = grad_y_t (times the
 * slope s (1 + u (1 - s)), s = sigmoid(u), if silu):
 *   grad_x_t = sum over j of weight[c][j] d_{t+K-1-j} (+ grad_state_out, for the
 *              tokens that state_out holds),
 *   grad_state: the same for the tokens before the first,
 *   grad_weight[c][j] = sum over (b, t) of d_t x_{t-K+1+j},  grad_bias = sum of d_t. */
typedef struct gdr_conv_bwd_args {
  int32_t B, T, C, K;
  int32_t io_dtype;     /* gdr_dtype of x, state, grad_y, grad_x and the       */
                        /* states' gradients                                   */
  int32_t silu;
  const void *x;
  const float *weight;
  const float *bias;
  const void *state;
  const int32_t *lens;
  const void *grad_y;          /* [B,T,C] io_dtype                             */
  const void *grad_state_out;  /* [B,K-1,C] io_dtype, or NULL for zeros        */
  void *grad_x;                /* [B,T,C] io_dtype                             */
  float *grad_weight;          /* [C,K] fp32                                   */
  float *grad_bias;            /* [C] fp32, or NULL                            */
  void *grad_state;            /* [B,K-1,C] io_dtype, or NULL                  */
  void *workspace;             /* gdr_conv_bwd_workspace bytes, 16-byte aligned */
  size_t workspace_bytes;
} gdr_conv_bwd_args;

/* Bytes gdr_conv_bwd needs at `workspace` (0 for arguments that it refuses).  Its
 * contents need not be set and are not kept; it serves one call at a time. */
size_t gdr_conv_bwd_workspace(const gdr_conv_bwd_args *args);
gdr_status gdr_conv_bwd(const gdr_conv_bwd_args *args, void *stream);

/* One token on N states: N * (K-1) * C < 2^31. */
typedef struct gdr_conv_step_args {
  int32_t N, C, K;
  int32_t io_dtype;
  int32_t silu;
  int32_t reserved;     /* 0                                                   */
  const void *x;        /* [N,C] io_dtype                                      */
  const float *weight;  /* [C,K] fp32                                          */
  const float *bias;    /* [C] fp32, or NULL                                   */
  const void *state;    /* [N,K-1,C] io_dtype                                  */
  void *state_out;      /* [N,K-1,C] io_dtype; may equal state                 */
  void *y;              /* [N,C] io_dtype                                      */
} gdr_conv_step_args;

gdr_status gdr_conv_step(const gdr_conv_step_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_CONV_H */
