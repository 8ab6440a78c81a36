/* gdr_ckpt8.h -- C ABI of the 8-bit activation checkpoints (gfx950).
 *
 * Part of libgdr.so (status codes, stream convention and ownership rules as in
 * gdr.h).  An activation that only the backward reads again is kept as one byte
 * a value: rows of D values, each run of 128 (the last one of a row may be
 * shorter) with one power of two as its scale,
 *
 *     exp   = the least E in [1, 254] with  max|x| <= 448 * 2^(E - 127)
 *     code  = x * 2^(127 - E) rounded (RNE) to e4m3 (4 exponent bits, bias 7,
 *             3 fraction bits, largest value 448)
 *     value = code * 2^(E - 127)
 *
 * so that scaling is exact and each value is off by at most 2^-4 of itself, or
 * 2^-10 of the scale.  NaN and Inf become NaN codes; the maximum is that of the
 * finite values (0 when there are none: E = 1).  A magnitude within 2^-5 of 2^128
 * rounds up to it and is unpacked as Inf.  gdr_norm_fwd writes such a
 * copy of its input while it has it, and gdr_norm_bwd and gdr_scan_bwd read one
 * in place of x.
 *
 * Sizes: any R >= 1 and D >= 1, R < 2^31, D <= 2^30, R * D < 2^40.  Pointers
 * are aligned to their element; outputs do not overlap inputs (GDR_ERR_ARG).
 */
#ifndef GDR_CKPT8_H
#define GDR_CKPT8_H

#include "gdr.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Values that share one exponent. */
#define GDR_CKPT8_GROUP 128

typedef struct gdr_ckpt8_pack_args {
  int64_t R;
  int32_t D;
  int32_t io_dtype;   /* gdr_dtype of x                                        */
  const void *x;      /* [R,D] io_dtype                                        */
  uint8_t *code;      /* [R,D]                                                 */
  uint8_t *exp;       /* [R,ceil(D/128)]                                       */
} gdr_ckpt8_pack_args;

gdr_status gdr_ckpt8_pack(const gdr_ckpt8_pack_args *args, void *stream);

typedef struct gdr_ckpt8_unpack_args {
  int64_t R;
  int32_t D;
  int32_t io_dtype;   /* gdr_dtype of x                                        */
  const uint8_t *code;
  const uint8_t *exp;
  void *x;            /* [R,D] io_dtype: the codes' values                     */
} gdr_ckpt8_unpack_args;

gdr_status gdr_ckpt8_unpack(const gdr_ckpt8_unpack_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_CKPT8_H */
