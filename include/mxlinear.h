/*
 * mxlinear.h -- C ABI of the microscaled linear layers (token-major, one
 * layer or a group of experts) and of the gradient clip, on AMD Instinct
 * MI355X (gfx950).  Part of libmxconv.so; statuses, roles and rounding modes
 * are those of mxconv.h.
 *
 * A linear layer multiplies tokens by a weight:
 *     X  [tokens][in_features]     the activation           MX_ROLE_ACT
 *     W  [out_features][in_features]  the weight            MX_ROLE_WEIGHT
 *     dY [tokens][out_features]    the output gradient      MX_ROLE_GRAD
 *     Y = X W^T,  dX = dY W,  dW = dY^T X
 * on operands in 4-bit microscaled floating point: E2M1 elements with one
 * E8M0 (power of two) scale per block, the format that block = 32 selects
 * for convolutions, by the same rule (mxconv.h, mx_quantize_cbf).
 *
 * Experts.  With experts = E >= 1, W holds E matrices, the tokens are sorted
 * by expert and `offsets`, E+1 int32 in device memory, gives the rows of X,
 * Y and dY that are expert e's: offsets[e] .. offsets[e+1]-1.  Any count may
 * be zero.  Offsets must not decrease and must lie in 0..tokens; nothing can
 * check device data before the call, so the kernels read them as their
 * running maximum clamped to that range: a wrong array gives wrong results
 * but no access out of bounds.  Rows that belong to no expert are neither
 * read nor written.  With experts = 0 offsets is ignored (pass NULL).
 *
 * Blocks.  block = 1: one scale per row and 32 consecutive features; a
 * token's codes depend on that token alone.  It has the row form only.
 * block = 32: one scale per 32 rows x 32 features, counted from the expert's
 * first row; the same codes then serve both contraction directions, so each
 * tensor is quantized once for its two products.
 *
 * Forms.  A quantized tensor is kept in up to two forms, each in the order
 * in which the matrix units take it when the product runs along
 *   MX_FORM_ROWS  the features:  X and W for Y = X W^T, dY for dX = dY W
 *   MX_FORM_COLS  the tokens (X and dY for dW) or W's output features (W for dX)
 * A form holds a matrix of R rows (the lines that stay) and C columns (the
 * contracted ones), both padded to multiples of 128, in tiles of 32 x 64:
 *   codes   tile (r/32, c/64) at ((r/32) * (C/64) + c/64) * 1024, in it
 *           (c/32%2) * 512 + (r%32) * 16 + (c%32)/2, even c in the low nibble
 *   scales  byte ((r/128) * (C/64) + c/64) * 256 + (c/32%2) * 128
 *           + (r%32) * 4 + (r/32)%4
 * An expert's tokens start at a multiple of 128 in the padded order, W's
 * experts follow each other as matrices of their own.  Padding holds zeros.
 *
 * Conventions
 * - Pointers are device pointers, except the descriptor, the tensor structs
 *   and the arrays of mx_grad_list.  The library allocates nothing and keeps
 *   nothing between calls.
 * - Matrices are row-major with a row stride `ld` in elements, at least the
 *   number of columns.  The element type is an mx_dtype.  Any alignment that
 *   the type has is taken; rows at multiples of 16 bytes are read fastest, at
 *   multiples of 64 written fastest.  W and dW are contiguous between experts:
 *   expert e starts at e * out_features * ld.
 * - Codes, scales and workspace are 16-byte aligned.  Sources and
 *   destinations must not overlap (the clip's may be the same tensors).
 * - Arguments are checked on the host before anything is enqueued; a
 *   negative mx_status is returned and nothing runs.  On MX_OK the work has
 *   been enqueued on `stream`.  Everything can be captured in a HIP graph.
 * - Results are bit-reproducible: no atomics, every sum has a fixed order.
 * - Products of dequantized elements are exact, sums are fp32, and one
 *   rounding to the output's type follows.
 * - tokens may be 0: Y and dX are then empty and dW is zero, as is the dW of
 *   an expert without tokens.
 */
#ifndef MXLINEAR_H
#define MXLINEAR_H

#include "mxconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element type of an unquantized matrix. */
typedef enum { MX_F32 = 0, MX_BF16 = 1, MX_F16 = 2 } mx_dtype;

typedef enum { MX_FORM_ROWS = 0, MX_FORM_COLS = 1 } mx_form;

#define MX_LINEAR_MAX_EXPERTS 1024

typedef struct {
  int32_t tokens;       /* rows of X, Y and dY, over all experts */
  int32_t out_features; /* rows of W */
  int32_t in_features;  /* columns of W */
  int32_t experts;      /* 0: one layer; else the number of experts */
  int32_t block;        /* 1 or 32 */
} mx_linear_desc;
/* MX_ERR_SHAPE: tokens < 0, a feature count <= 0, experts outside
 * 0..MX_LINEAR_MAX_EXPERTS, a padded size of 2^31 rows or more, or ld below
 * the number of columns.  MX_ERR_BLOCK: block other than 1 or 32, or a call
 * on the column form with block 1.  MX_ERR_FORMAT: unknown mx_dtype or
 * mx_form. */

/* A quantized tensor.  rows / cols: the codes of the two forms; either may
 * be NULL where no call needs that form, and its scales with it. */
typedef struct {
  void* rows;
  uint8_t* row_scales;
  void* cols;
  uint8_t* col_scales;
} mx_linear_qtensor;

/* Bytes of one form's codes and scales (0 on an invalid argument, or for a
 * form without elements). */
size_t mx_linear_code_bytes(const mx_linear_desc* desc, mx_role role, mx_form form);
size_t mx_linear_scale_bytes(const mx_linear_desc* desc, mx_role role, mx_form form);

/* Quantize a matrix of `role` into the forms that dst has.
 *   rounding, seed   as mx_quantize_cbf: MX_SR draws from SplitMix64 with the
 *                    element's index row * columns + column in the whole
 *                    source matrix (W: over all experts), whatever ld is
 * A block that holds an Inf or a NaN takes scale code 0xFF (NaN) and zero
 * codes; every output that the block enters is NaN then. */
mx_status mx_linear_quantize(const mx_linear_desc* desc, mx_role role, const void* src, mx_dtype dtype, int64_t ld,
                             const int32_t* offsets, const mx_linear_qtensor* dst, mx_round rounding, uint64_t seed,
                             hipStream_t stream);

/* The values that one form holds, in the matrix' own order. */
mx_status mx_linear_dequantize(const mx_linear_desc* desc, mx_role role, mx_form form, const mx_linear_qtensor* q,
                               void* dst, mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t stream);

/* Bytes of workspace that mx_linear_fwd, _dgrad, _wgrad and _apply on this
 * descriptor need at most (0 on an invalid descriptor, or where none do):
 * partial sums of a product that is split along its contraction, and
 * _apply's quantized tokens. */
size_t mx_linear_workspace_bytes(const mx_linear_desc* desc);

/* Y = X W^T from the row forms of W and X. */
mx_status mx_linear_fwd(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                        mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                        hipStream_t stream);

/* dX = dY W from the column form of W and the row form of dY (block 32). */
mx_status mx_linear_dgrad(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* dyq, void* dx,
                          mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                          hipStream_t stream);

/* dW = dY^T X from the column forms of dY and X (block 32). */
mx_status mx_linear_wgrad(const mx_linear_desc* desc, const mx_linear_qtensor* dyq, const mx_linear_qtensor* xq, void* dw,
                          mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                          hipStream_t stream);

/* Serving: quantize X with block 1 (whatever desc->block is: the weight's
 * row form is laid out alike for both) and multiply, Y = X W^T.  The result
 * is that of mx_linear_quantize and mx_linear_fwd; for few tokens it is one
 * launch that quantizes them on the way. */
mx_status mx_linear_apply(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype,
                          int64_t ldx, void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, void* workspace,
                          size_t ws_bytes, hipStream_t stream);

/* Gradients of many tensors, contiguous each, as arrays of `count` entries
 * in HOST memory (read during the call only).  Their elements, counted with
 * 8192 more for each tensor, must not pass 2^43 (MX_ERR_SHAPE). */
typedef struct {
  int32_t count;
  const void* const* grads;
  void* const* out;       /* clipped gradients, of the gradient's type; may be the gradients themselves, NULL for the norm alone */
  const int64_t* numel;   /* >= 0 */
  const int32_t* dtypes;  /* mx_dtype */
} mx_grad_list;

/* Bytes of workspace for a list of `count` tensors (0 for count <= 0). */
size_t mx_grad_workspace_bytes(int32_t count);

/* *norm = sqrt(sum of all squares), summed in fp64, one fp32 in device
 * memory. */
mx_status mx_grad_norm(const mx_grad_list* list, float* norm, void* workspace, size_t ws_bytes, hipStream_t stream);

/* The norm as above, then out = grad * min(1, max_norm / (norm + 1e-6)), the
 * factor and the product in fp32, rounded once to the tensor's type.  With a
 * factor of 1 tensors that are their own output are left untouched.  A norm
 * of Inf gives the factor 0, a NaN norm a NaN factor: callers that want to
 * skip such a step look at *norm.  max_norm must be >= 0 (MX_ERR_SHAPE).
 * A tensor that aliases another one gives undefined values. */
mx_status mx_grad_clip(const mx_grad_list* list, float max_norm, float* norm, void* workspace, size_t ws_bytes,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MXLINEAR_H */
