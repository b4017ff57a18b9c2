// Internal interface of the linear layers in 8 bits: the tile layout and the
// launchers behind the C ABI (linear8_capi.cpp).  Padded geometry, forms and
// experts' segments are those of linear.h.  Arguments reaching a launcher have
// been validated on the host.
#pragma once

#include "linear.h"
#include "mxlinear8.h"

namespace mx {

// A tile of 32 rows x 64 contracted columns is 2 KiB: two planes of 1 KiB, of
// each of which lane l of a wave takes 16 bytes (row l%32, columns 32 * plane +
// 16 * (l/32) .. +15).  The two together are an operand of
// v_mfma_scale_f32_32x32x64_f8f6f4: it contracts corresponding places of its two
// operands, so any order of columns will do that both have, and one scale
// covers all 64.  The scales of 4 tiles on top of each other are interleaved,
// so that one dword per lane serves 4 MFMA operands through the byte select.
constexpr int k8TileBytes = 2048;
constexpr int k8ScaleBytes = 128;  // of 128 rows x 128 columns

hipError_t launch_lin8_quantize(const LinGeom& g, mx_role role, int block, const void* src, mx_dtype dtype, int64_t ld,
                                const int32_t* offsets, const mx_linear_qtensor* dst, hipStream_t s);
hipError_t launch_lin8_dequantize(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                  mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t s);

// The three products.  a: the operand whose rows are the output's rows.
size_t lin8_product_workspace(const LinGeom& g, LinOp op);
hipError_t launch_lin8_product(const LinGeom& g, LinOp op, const mx_linear_qtensor* aq, const mx_linear_qtensor* bq,
                               void* out, mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace,
                               hipStream_t s);
// fwd and dgrad with few tokens, where lin8_few() says so.
bool lin8_few(const LinGeom& g);
hipError_t launch_lin8_few(const LinGeom& g, bool dgrad, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                           mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s);
// Quantize-and-multiply in one launch, where lin8_fused() says so.
bool lin8_fused(const LinGeom& g);
hipError_t launch_lin8_fused(const LinGeom& g, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                             void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s);

// What a call launches, for the tests (linear.h's LinVariant).
LinVariant lin8_product_variant(const LinGeom& g, LinOp op, mx_dtype dtype);
bool lin8_product_streams(const LinGeom& g, LinOp op, const void* out, mx_dtype dtype, int64_t ld);
LinVariant lin8_few_variant(const LinGeom& g, bool dgrad, bool fused);

}  // namespace mx
