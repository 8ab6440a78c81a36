/* gdr_gnorm.h -- C ABI of the group norm with its activation or gate, forward and
 * backward (gfx950).
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  It is what stands between a recurrence and a layer's last projection: a
 * token's C channels fall into G groups (heads) of D = C / G, each group is normalised
 * by itself, each channel has its own weight and bias, and the result is gated:
 *
 *     mean = sum(x) / D if center, else 0
 *     rstd = 1 / sqrt(sum((x - mean)^2) / D + eps)
 *     xh   = (x - mean) rstd,   u = xh weight + bias
 *     y    = u act(z) with z given, else act(u);   act(v) = v sigmoid(v) if silu, else v
 *
 * and with du = grad_y act(z) (grad_y act'(u) without z), g = du weight:
 *     grad_z = grad_y u act'(z)
 *     grad_x = rstd (g - [sum(g)/D if center] - xh sum(g xh)/D)
 *     grad_weight = sum over rows of du xh,   grad_bias = sum over rows of du
 *
 * Sizes: any R >= 1 rows, 1 <= G with C a multiple of G, C / G <= 16384, C <= 2^20,
 * R * G < 2^31, R * C < 2^40.  Every pointer is aligned to its element; rows move 16
 * bytes at a time, fastest where groups begin at multiples of 16 bytes.  Outputs
 * overlap neither inputs nor each other (GDR_ERR_ARG).  Sums are fp32, in an order
 * that depends on the sizes alone (where the squares of a group pass fp32, its values
 * being some 2^60, rstd is 0); y, grad_x and grad_z are rounded once (RNE) to
 * io_dtype.  NaN and Inf stay within their group of their row (and reach grad_weight
 * and grad_bias).
 */
#ifndef GDR_GNORM_H
#define GDR_GNORM_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct gdr_gnorm_args {
  int64_t R;
  int32_t C, G;
  int32_t io_dtype;     /* gdr_dtype of x, z and y                             */
  int32_t center, silu; /* 0 or 1                                              */
  float eps;            /* finite, >= 0                                        */
  const void *x;        /* [R,C] io_dtype                                      */
  const void *z;        /* [R,C] io_dtype, or NULL                             */
  const float *weight;  /* [C] fp32, or NULL for ones                          */
  const float *bias;    /* [C] fp32, or NULL for zeros                         */
  void *y;              /* [R,C] io_dtype                                      */
  float *mean;          /* [R,G] fp32, or NULL (NULL without center)           */
  float *rstd;          /* [R,G] fp32, or NULL                                 */
} gdr_gnorm_args;

gdr_status gdr_gnorm_fwd(const gdr_gnorm_args *args, void *stream);

typedef struct gdr_gnorm_bwd_args {
  int64_t R;
  int32_t C, G;
  int32_t io_dtype;     /* gdr_dtype of x, z, grad_y, grad_x and grad_z        */
  int32_t silu;
  const void *x;
  const void *z;
  const float *mean;    /* [R,G] fp32, as the forward wrote them; NULL without */
                        /* center                                              */
  const float *rstd;    /* [R,G] fp32                                          */
  const float *weight;  /* [C] fp32, or NULL for ones                          */
  const float *bias;    /* [C] fp32, or NULL for zeros                         */
  const void *grad_y;   /* [R,C] io_dtype                                      */
  void *grad_x;         /* [R,C] io_dtype                                      */
  void *grad_z;         /* [R,C] io_dtype (with z), else NULL                  */
  float *grad_weight;   /* [C] fp32, or NULL                                   */
  float *grad_bias;     /* [C] fp32, or NULL                                   */
  void *workspace;      /* gdr_gnorm_bwd_workspace bytes, 16-byte aligned      */
  size_t workspace_bytes;
} gdr_gnorm_bwd_args;

/* Bytes gdr_gnorm_bwd needs at `workspace` (0: none, or refused arguments).  Its
 * contents need not be set and are not kept; it serves one call at a time. */
size_t gdr_gnorm_bwd_workspace(const gdr_gnorm_bwd_args *args);
gdr_status gdr_gnorm_bwd(const gdr_gnorm_bwd_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_GNORM_H */
