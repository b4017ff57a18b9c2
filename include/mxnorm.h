/*
 * mxnorm.h -- C ABI of the root-mean-square norm with the residual's addition
 * on AMD Instinct MI355X (gfx950).  Part of libmxconv.so; statuses and
 * conventions are those of mxlinear.h.
 *
 *     total = x + residual                      (rounded to its type, which is x's)
 *     rstd  = 1 / sqrt(mean over the features of total^2 + eps)
 *     y     = total * rstd * weight
 * for each token, and the gradients of both lines:
 *     h  = total * rstd,  g = dy * weight
 *     dx = rstd * (g - h * mean(g * h)) + dtotal      (x's and the residual's gradient alike)
 *     dweight = sum over the tokens of dy * h
 * Sums, h and g are fp32 or more, each result is rounded once.  Sums have a
 * fixed order: results are bit-reproducible.  Squares are summed in fp64, which
 * holds those of all finite values: rows of any size are normed alike.  rstd is
 * rounded to fp32: a subnormal of fewer bits where the root is over 2^126, and
 * Inf, and y with it, where it is 2^-128 or less.  A row with an Inf has an rstd
 * of 0.
 *
 * Matrices are [tokens][features] with a row stride in elements, of any
 * alignment that the type has.  total may be x or the residual, and dx may be
 * dy or dtotal, exactly (same address, stride and type); nothing else may
 * overlap.  With tokens = 0 the matrices are empty and dweight is zero.
 */
#ifndef MXNORM_H
#define MXNORM_H

#include "mxlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t tokens;   /* >= 0 */
  int32_t features; /* > 0 */
  float eps;        /* >= 0 and finite */
} mx_norm_desc;
/* MX_ERR_SHAPE: a value outside these, or sizes whose padded matrix is not one
 * of mxlinear.h's (an activation of as many in features). */

/* The norm.
 *   residual  NULL: total = x, and total is not needed then
 *   dtype     type of x, residual and total
 *   weight    [features], contiguous, of its own type
 *   total     NULL: not stored
 *   y         NULL: not stored
 *   yq        NULL, or a tensor whose row form takes y in 8 bits, the
 *             activation of mx_linear8_fwd on a layer without experts (E4M3,
 *             1x128 blocks; its column form is ignored).  Its codes are those of
 *             total * rstd * weight with rstd in fp64, rounded once; quantizing a
 *             stored y, which has been rounded, may give others next to ties
 *   rstd      NULL, or fp32 [tokens], for the gradients
 * One of total, y, yq and rstd is needed. */
mx_status mx_norm_fwd(const mx_norm_desc* desc, const void* x, int64_t ldx, const void* residual, int64_t ldr, mx_dtype dtype,
                      const void* weight, mx_dtype w_dtype, void* total, int64_t ldt, void* y, mx_dtype y_dtype, int64_t ldy,
                      const mx_linear_qtensor* yq, float* rstd, hipStream_t stream);

/* Bytes of workspace of mx_norm_bwd (0 on an invalid descriptor).  A workspace
 * serves one call at a time, in captured graphs too. */
size_t mx_norm_workspace_bytes(const mx_norm_desc* desc);

/* The gradients.
 *   total, rstd  of mx_norm_fwd (total is x where there was no residual)
 *   dtotal       NULL, or the gradient that reaches total past the norm
 *   dtype        type of total, dtotal and dx
 *   dweight      NULL, or fp32 [features]; the workspace is needed for it alone
 *   dx           NULL: not stored */
mx_status mx_norm_bwd(const mx_norm_desc* desc, const void* dy, mx_dtype dy_dtype, int64_t lddy, const void* total, int64_t ldt,
                      const void* dtotal, int64_t lddt, mx_dtype dtype, const void* weight, mx_dtype w_dtype,
                      const float* rstd, void* dx, int64_t lddx, float* dweight, void* workspace, size_t ws_bytes,
                      hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXNORM_H */
