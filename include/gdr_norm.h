/* gdr_norm.h -- C ABI of the layer norm, forward and backward (gfx950).
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  Rows of D values: the channels of a token before a layer, or one
 * head's d_v outputs of the delta rule after it.  Per row x:
 *
 *     mean = sum(x) / D,   rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
 *     xh   = (x - mean) rstd,   y = xh weight + bias
 *
 * and with g = grad_y weight:
 *     grad_x      = rstd (g - sum(g)/D - xh sum(g xh)/D)
 *     grad_weight = sum over rows of grad_y xh,  grad_bias = sum over rows of grad_y
 *
 * Sizes: any R >= 1 rows of 1 <= D <= 65536, R * D < 2^40, R < 2^31.  Every
 * pointer is aligned to its element; rows move 16 bytes at a time, fastest where they
 * begin at multiples of 16 bytes.  Outputs overlap neither
 * inputs nor each other (GDR_ERR_ARG).  Sums are fp32, in an order that depends
 * on the sizes alone; y and grad_x are rounded once (RNE) to io_dtype.  NaN and
 * Inf stay within their row (and reach grad_weight and grad_bias).
 */
#ifndef GDR_NORM_H
#define GDR_NORM_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdr_norm_args {
  int64_t R;
  int32_t D;
  int32_t io_dtype;     /* gdr_dtype of x and y                                */
  float eps;            /* finite, >= 0                                        */
  int32_t reserved;     /* 0                                                   */
  const void *x;        /* [R,D] io_dtype                                      */
  const float *weight;  /* [D] fp32, or NULL for ones                          */
  const float *bias;    /* [D] fp32, or NULL for zeros                         */
  void *y;              /* [R,D] io_dtype                                      */
  float *mean;          /* [R] fp32, or NULL                                   */
  float *rstd;          /* [R] fp32, or NULL                                   */
  uint8_t *x_code;      /* [R,D] 8-bit copy of x for the backward, or NULL     */
  uint8_t *x_exp;       /* [R,ceil(D/128)] its exponents (with x_code; both as */
                        /* gdr_ckpt8_pack writes them)                         */
} gdr_norm_args;

gdr_status gdr_norm_fwd(const gdr_norm_args *args, void *stream);

typedef struct gdr_norm_bwd_args {
  int64_t R;
  int32_t D;
  int32_t io_dtype;     /* gdr_dtype of grad_y, grad_x and x (unless x_exp)    */
  const void *x;        /* [R,D] io_dtype, or 8-bit codes                      */
  const uint8_t *x_exp; /* NULL, or the exponents of x's codes                 */
  const float *mean;    /* [R] fp32, as the forward wrote them                 */
  const float *rstd;    /* [R] fp32                                            */
  const float *weight;  /* [D] fp32, or NULL for ones                          */
  const void *grad_y;   /* [R,D] io_dtype                                      */
  void *grad_x;         /* [R,D] io_dtype                                      */
  float *grad_weight;   /* [D] fp32, or NULL                                   */
  float *grad_bias;     /* [D] fp32, or NULL                                   */
  void *workspace;      /* gdr_norm_bwd_workspace bytes, 16-byte aligned       */
  size_t workspace_bytes;
} gdr_norm_bwd_args;

/* Bytes gdr_norm_bwd needs at `workspace` (0: none, or refused arguments). */
size_t gdr_norm_bwd_workspace(const gdr_norm_bwd_args *args);
gdr_status gdr_norm_bwd(const gdr_norm_bwd_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_NORM_H */
