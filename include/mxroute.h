/*
 * mxroute.h -- C ABI of the tokens' way to their experts and back on AMD
 * Instinct MI355X (gfx950).  Part of libmxconv.so; statuses and conventions
 * are those of mxlinear.h.
 *
 * A token t has `choices` experts, expert[t][j], with weights weight[t][j].  A
 * choice outside 0..experts-1 is dropped: a padded token's, or one that finds
 * its expert full.  The others are sorted by expert, and an expert's in the
 * order of (t, j):
 *     rows[t][j]   the choice's place in that order, -1 if it was dropped
 *     offsets      where each expert's rows begin, as mx_linear_* take them; the
 *                  last one is the number of rows that are in use
 *     order[i]     t * choices + j of place i, -1 behind the last one in use
 * and the rows of tokens x choices matrices follow the tokens there and back:
 *     gather       out[rows[t][j]] = x[t]
 *     gather_bwd   dx[t] = sum_j dout[rows[t][j]]
 *     combine      out[t] = sum_j weight[t][j] * y[rows[t][j]]
 *     combine_bwd  dy[rows[t][j]] = weight[t][j] * dout[t],
 *                  dweight[t][j] = <dout[t], y[rows[t][j]]>
 * Dropped choices add nothing and have a dweight of 0, a token whose choices
 * were all dropped gets zeros, and rows that no choice has are neither read
 * nor written.  Sums are fp32 in the order of j (dweight: a fixed order), each
 * result is rounded once; no atomics: results are bit-reproducible.
 *
 * Matrices have a row stride in elements and any alignment that their type
 * has; expert, rows and weights are contiguous [tokens][choices].  Sources and
 * destinations must not overlap.  Nothing can check device data before a call:
 * an entry of rows outside 0..tokens*choices-1 counts as dropped, and one that
 * occurs twice gives undefined values in its row, but no access out of bounds.
 */
#ifndef MXROUTE_H
#define MXROUTE_H

#include "mxlinear.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MX_ROUTE_MAX_CHOICES 64

typedef struct {
  int32_t tokens;   /* >= 0 */
  int32_t choices;  /* 1..MX_ROUTE_MAX_CHOICES */
  int32_t experts;  /* 1..MX_LINEAR_MAX_EXPERTS */
  int32_t features; /* > 0 (mx_route_sort does not read it) */
} mx_route_desc;
/* MX_ERR_SHAPE: a value outside these, or tokens * choices of 2^30 or more. */

/* Bytes of workspace of mx_route_sort (0 on an invalid descriptor, or where
 * none is needed).  A workspace serves one call at a time, in captured graphs
 * too. */
size_t mx_route_workspace_bytes(const mx_route_desc* desc);

/* expert [tokens][choices] -> offsets [experts + 1], rows [tokens][choices] and,
 * unless NULL, order [tokens * choices]; all int32. */
mx_status mx_route_sort(const mx_route_desc* desc, const int32_t* expert, int32_t* offsets, int32_t* rows, int32_t* order,
                        void* workspace, size_t ws_bytes, hipStream_t stream);

/* x [tokens][features] -> out [tokens * choices][features], of one type. */
mx_status mx_route_gather(const mx_route_desc* desc, const void* x, int64_t ldx, const int32_t* rows, void* out, int64_t ldo,
                          mx_dtype dtype, hipStream_t stream);
mx_status mx_route_gather_bwd(const mx_route_desc* desc, const void* dout, int64_t ldo, const int32_t* rows, void* dx,
                              int64_t ldx, mx_dtype dtype, hipStream_t stream);

/* y [tokens * choices][features] and fp32 weight -> out [tokens][features]; y
 * and out of one type. */
mx_status mx_route_combine(const mx_route_desc* desc, const void* y, int64_t ldy, const int32_t* rows, const float* weight,
                           void* out, int64_t ldo, mx_dtype dtype, hipStream_t stream);
/* dout, y and dy of one type; dweight fp32.  dy or dweight may be NULL. */
mx_status mx_route_combine_bwd(const mx_route_desc* desc, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                               const int32_t* rows, const float* weight, void* dy, int64_t lddy, float* dweight,
                               mx_dtype dtype, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXROUTE_H */
