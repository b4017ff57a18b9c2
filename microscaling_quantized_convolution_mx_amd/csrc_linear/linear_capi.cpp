// C ABI of the microscaled linear layers and the gradient clip: host-side
// validation and dispatch.  The arguments are documented in
// include/mxlinear.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <limits>

#include "linear.h"

namespace {

using mx::LinGeom;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
mx_status launched(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

bool known_dtype(int t) { return t == MX_F32 || t == MX_BF16 || t == MX_F16; }
uintptr_t dtype_bytes(int t) { return t == MX_F32 ? 4 : 2; }

// Padded rows, column tiles and workgroups are 32-bit in the kernels.
constexpr int64_t kMaxLines = std::numeric_limits<int32_t>::max();

mx_status check_desc(const mx_linear_desc* d) {
  if (!d) return MX_ERR_NULL;
  if (d->block != 1 && d->block != 32) return MX_ERR_BLOCK;
  if (d->tokens < 0 || d->out_features <= 0 || d->in_features <= 0) return MX_ERR_SHAPE;
  if (d->experts < 0 || d->experts > MX_LINEAR_MAX_EXPERTS) return MX_ERR_SHAPE;
  // (in this order no product below overflows: every factor fits 32 bits)
  if (d->tokens > kMaxLines - 128 - 128 * static_cast<int64_t>(MX_LINEAR_MAX_EXPERTS) ||
      d->out_features > kMaxLines - 128 || d->in_features > kMaxLines - 128)
    return MX_ERR_SHAPE;
  const LinGeom g = mx::make_lin_geom(d);
  if (g.np * g.ew > kMaxLines || g.kp * g.ew > kMaxLines) return MX_ERR_SHAPE;
  // 128x128 blocks and output tiles of every matrix: one launch each
  const int64_t mb = g.mp / 128, nb = g.np / 128, kb = g.kp / 128;
  const int64_t most = kMaxLines / 256;
  if (mb * nb > most || mb * kb > most || nb * kb > most / g.ew) return MX_ERR_SHAPE;
  return MX_OK;
}

mx_status check_role(mx_role r) {
  return (r == MX_ROLE_ACT || r == MX_ROLE_WEIGHT || r == MX_ROLE_GRAD) ? MX_OK : MX_ERR_ROLE;
}

int64_t form_tiles(const LinGeom& g, mx_role role, mx_form form) {
  int64_t r, c;
  mx::form_dims(g, role, form, r, c);
  return (r / mx::kTileR) * (c / mx::kTileC) * mx::form_matrices(g, role);
}

// The form's buffers, where it has elements.
mx_status check_form(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q) {
  if (!q) return MX_ERR_NULL;
  const void* codes = form == MX_FORM_ROWS ? q->rows : q->cols;
  const void* scales = form == MX_FORM_ROWS ? q->row_scales : q->col_scales;
  if (form_tiles(g, role, form) > 0 && (!codes || !scales)) return MX_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scales, 16)) return MX_ERR_ALIGN;
  return MX_OK;
}

// An unquantized matrix of rows x cols.
mx_status check_matrix(const void* p, int dtype, int64_t ld, int64_t rows, int64_t cols) {
  if (!known_dtype(dtype)) return MX_ERR_FORMAT;
  if (ld < cols || ld > std::numeric_limits<int64_t>::max() / 8 / (rows > 0 ? rows : 1)) return MX_ERR_SHAPE;
  if (rows > 0 && !p) return MX_ERR_NULL;
  if (!aligned(p, dtype_bytes(dtype))) return MX_ERR_ALIGN;
  return MX_OK;
}

mx_status check_offsets(const LinGeom& g, const int32_t* offsets) {
  if (g.e > 0 && !offsets) return MX_ERR_NULL;
  return aligned(offsets, 4) || g.e == 0 ? MX_OK : MX_ERR_ALIGN;
}

void matrix_dims(const LinGeom& g, mx_role role, int64_t& rows, int64_t& cols) {
  rows = role == MX_ROLE_WEIGHT ? g.n * g.ew : g.m;
  cols = role == MX_ROLE_GRAD ? g.n : g.k;
}

mx_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need > 0 && (!ws || bytes < need)) return MX_ERR_WORKSPACE;
  return aligned(ws, 16) ? MX_OK : MX_ERR_ALIGN;
}

// What _apply keeps of the quantized tokens in its workspace, before the
// product's partial sums.
size_t apply_code_bytes(const LinGeom& g) { return static_cast<size_t>(g.mp / mx::kTileR * (g.kp / mx::kTileC)) * mx::kTileBytes; }
size_t apply_scale_bytes(const LinGeom& g) { return static_cast<size_t>(g.mp / mx::kPad * (g.kp / mx::kTileC)) * mx::kScaleBytes; }
size_t apply_workspace(const LinGeom& g) {
  if (g.m == 0 || mx::lin_fused(g)) return 0;
  return apply_code_bytes(g) + apply_scale_bytes(g) + mx::lin_product_workspace(g, mx::LIN_FWD);
}

mx_status product(const mx_linear_desc* desc, mx::LinOp op, const mx_linear_qtensor* aq, const mx_linear_qtensor* bq, void* out,
                  mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes, hipStream_t stream) {
  mx_status st = check_desc(desc);
  if (st != MX_OK) return st;
  if (op != mx::LIN_FWD && desc->block != 32) return MX_ERR_BLOCK;
  const LinGeom g = mx::make_lin_geom(desc);
  const mx_role ra = op == mx::LIN_FWD ? MX_ROLE_ACT : MX_ROLE_GRAD, rb = op == mx::LIN_WGRAD ? MX_ROLE_ACT : MX_ROLE_WEIGHT;
  if ((st = check_form(g, ra, op == mx::LIN_WGRAD ? MX_FORM_COLS : MX_FORM_ROWS, aq)) != MX_OK) return st;
  if ((st = check_form(g, rb, op == mx::LIN_FWD ? MX_FORM_ROWS : MX_FORM_COLS, bq)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, op == mx::LIN_FWD ? MX_ROLE_GRAD : op == mx::LIN_DGRAD ? MX_ROLE_ACT : MX_ROLE_WEIGHT, rows, cols);
  if ((st = check_matrix(out, dtype, ld, rows, cols)) != MX_OK) return st;
  if ((st = check_offsets(g, offsets)) != MX_OK) return st;
  if ((st = check_workspace(workspace, ws_bytes, mx::lin_product_workspace(g, op))) != MX_OK) return st;
  return launched(mx::launch_lin_product(g, op, aq, bq, out, dtype, ld, offsets, workspace, stream));
}

mx_status check_list(const mx_grad_list* l, bool clip) {
  if (!l) return MX_ERR_NULL;
  if (l->count < 0) return MX_ERR_SHAPE;
  if (l->count > 0 && (!l->grads || !l->numel || !l->dtypes || (clip && !l->out))) return MX_ERR_NULL;
  int64_t total = 0;
  for (int32_t i = 0; i < l->count; ++i) {
    if (!known_dtype(l->dtypes[i])) return MX_ERR_FORMAT;
    // one chunk at least for each, so that all chunks fit an int32
    if (l->numel[i] < 0 || l->numel[i] > mx::kMaxGradElems) return MX_ERR_SHAPE;
    if ((total += l->numel[i] + 8192) > mx::kMaxGradElems) return MX_ERR_SHAPE;
    if (l->numel[i] == 0) continue;
    if (!l->grads[i] || (clip && !l->out[i])) return MX_ERR_NULL;
    const uintptr_t a = dtype_bytes(l->dtypes[i]);
    if (!aligned(l->grads[i], a) || (clip && !aligned(l->out[i], a))) return MX_ERR_ALIGN;
  }
  return MX_OK;
}

mx_status grad(const mx_grad_list* l, bool clip, float max_norm, float* norm, void* workspace, size_t ws_bytes, hipStream_t stream) {
  mx_status st = check_list(l, clip);
  if (st != MX_OK) return st;
  if (clip && !(max_norm >= 0.0f)) return MX_ERR_SHAPE;
  if (!norm) return MX_ERR_NULL;
  if (!aligned(norm, 4)) return MX_ERR_ALIGN;
  if ((st = check_workspace(workspace, ws_bytes, mx_grad_workspace_bytes(l->count))) != MX_OK) return st;
  return launched(mx::launch_grad_clip(l, clip, max_norm, norm, workspace, stream));
}

}  // namespace

extern "C" {

size_t mx_linear_code_bytes(const mx_linear_desc* desc, mx_role role, mx_form form) {
  if (check_desc(desc) != MX_OK || check_role(role) != MX_OK || (form != MX_FORM_ROWS && form != MX_FORM_COLS)) return 0;
  if (form == MX_FORM_COLS && desc->block != 32) return 0;
  return static_cast<size_t>(form_tiles(mx::make_lin_geom(desc), role, form)) * mx::kTileBytes;
}

size_t mx_linear_scale_bytes(const mx_linear_desc* desc, mx_role role, mx_form form) {
  // 4 tiles of 1 KiB share 256 bytes of scales
  return mx_linear_code_bytes(desc, role, form) / (4 * mx::kTileBytes) * mx::kScaleBytes;
}

size_t mx_linear_workspace_bytes(const mx_linear_desc* desc) {
  if (check_desc(desc) != MX_OK) return 0;
  const LinGeom g = mx::make_lin_geom(desc);
  size_t need = apply_workspace(g);
  for (mx::LinOp op : {mx::LIN_FWD, mx::LIN_DGRAD, mx::LIN_WGRAD}) {
    const size_t b = mx::lin_product_workspace(g, op);
    need = b > need ? b : need;
  }
  return need;
}

mx_status mx_linear_quantize(const mx_linear_desc* desc, mx_role role, const void* src, mx_dtype dtype, int64_t ld,
                             const int32_t* offsets, const mx_linear_qtensor* dst, mx_round rounding, uint64_t seed,
                             hipStream_t stream) {
  mx_status st = check_desc(desc);
  if (st != MX_OK) return st;
  if ((st = check_role(role)) != MX_OK) return st;
  if (rounding != MX_RNE && rounding != MX_SR) return MX_ERR_ROUND;
  if (!dst) return MX_ERR_NULL;
  const LinGeom g = mx::make_lin_geom(desc);
  if (dst->cols && desc->block != 32) return MX_ERR_BLOCK;
  // the forms that dst has, one at least where there is something to store
  if (dst->rows || !dst->cols) {
    if ((st = check_form(g, role, MX_FORM_ROWS, dst)) != MX_OK) return st;
  }
  if (dst->cols && (st = check_form(g, role, MX_FORM_COLS, dst)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, role, rows, cols);
  if ((st = check_matrix(src, dtype, ld, rows, cols)) != MX_OK) return st;
  if (role != MX_ROLE_WEIGHT && (st = check_offsets(g, offsets)) != MX_OK) return st;
  return launched(mx::launch_lin_quantize(g, role, desc->block, src, dtype, ld, offsets, dst, rounding, seed, stream));
}

mx_status mx_linear_dequantize(const mx_linear_desc* desc, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                               mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t stream) {
  mx_status st = check_desc(desc);
  if (st != MX_OK) return st;
  if ((st = check_role(role)) != MX_OK) return st;
  if (form != MX_FORM_ROWS && form != MX_FORM_COLS) return MX_ERR_FORMAT;
  if (form == MX_FORM_COLS && desc->block != 32) return MX_ERR_BLOCK;
  const LinGeom g = mx::make_lin_geom(desc);
  if ((st = check_form(g, role, form, q)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, role, rows, cols);
  if ((st = check_matrix(dst, dtype, ld, rows, cols)) != MX_OK) return st;
  if (role != MX_ROLE_WEIGHT && (st = check_offsets(g, offsets)) != MX_OK) return st;
  return launched(mx::launch_lin_dequantize(g, role, form, q, dst, dtype, ld, offsets, stream));
}

mx_status mx_linear_fwd(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                        mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                        hipStream_t stream) {
  return product(desc, mx::LIN_FWD, xq, wq, y, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear_dgrad(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* dyq, void* dx,
                          mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                          hipStream_t stream) {
  return product(desc, mx::LIN_DGRAD, dyq, wq, dx, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear_wgrad(const mx_linear_desc* desc, const mx_linear_qtensor* dyq, const mx_linear_qtensor* xq, void* dw,
                          mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                          hipStream_t stream) {
  return product(desc, mx::LIN_WGRAD, dyq, xq, dw, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear_apply(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                          void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, void* workspace, size_t ws_bytes,
                          hipStream_t stream) {
  mx_status st = check_desc(desc);
  if (st != MX_OK) return st;
  const LinGeom g = mx::make_lin_geom(desc);
  if ((st = check_form(g, MX_ROLE_WEIGHT, MX_FORM_ROWS, wq)) != MX_OK) return st;
  if ((st = check_matrix(x, x_dtype, ldx, g.m, g.k)) != MX_OK) return st;
  if ((st = check_matrix(y, y_dtype, ldy, g.m, g.n)) != MX_OK) return st;
  if ((st = check_offsets(g, offsets)) != MX_OK) return st;
  if ((st = check_workspace(workspace, ws_bytes, apply_workspace(g))) != MX_OK) return st;
  if (g.m == 0) return MX_OK;
  if (mx::lin_fused(g)) return launched(mx::launch_lin_fused(g, wq, x, x_dtype, ldx, y, y_dtype, ldy, offsets, stream));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const mx_linear_qtensor xq{ws, ws + apply_code_bytes(g), nullptr, nullptr};
  const hipError_t e = mx::launch_lin_quantize(g, MX_ROLE_ACT, 1, x, x_dtype, ldx, offsets, &xq, MX_RNE, 0, stream);
  if (e != hipSuccess) return MX_ERR_LAUNCH;
  return launched(mx::launch_lin_product(g, mx::LIN_FWD, &xq, wq, y, y_dtype, ldy, offsets,
                                         ws + apply_code_bytes(g) + apply_scale_bytes(g), stream));
}

// Not part of the ABI: the kernel, size, pieces, threads and workgroups of
// linear.h's LinVariant for mx_linear_fwd (0), _dgrad (1), _wgrad (2) or
// _apply's product (3) on this descriptor.  Launches nothing.
mx_status mx_internal_linear_variant(const mx_linear_desc* desc, int call, int64_t* out) {
  const mx_status st = check_desc(desc);
  if (st != MX_OK) return st;
  if (!out) return MX_ERR_NULL;
  const LinGeom g = mx::make_lin_geom(desc);
  const mx::LinVariant v = call == 3 && g.m > 0 && mx::lin_fused(g)
                               ? mx::lin_few_variant(g, false, true)
                               : mx::lin_product_variant(g, call == 1 ? mx::LIN_DGRAD : call == 2 ? mx::LIN_WGRAD : mx::LIN_FWD);
  out[0] = v.kernel;
  out[1] = v.size;
  out[2] = v.splits;
  out[3] = v.threads;
  out[4] = v.workgroups;
  return MX_OK;
}

// Not part of the ABI: whether mx_linear_fwd (0), _dgrad (1), _wgrad (2) or
// _dequantize (4, from the row form) would write this output past the caches.
int mx_internal_linear_streams(const mx_linear_desc* desc, int call, const void* out, mx_dtype dtype, int64_t ld) {
  if (call == 4) return mx::lin_dequantize_streams(out, dtype, ld) ? 1 : 0;
  const mx::LinOp op = call == 1 ? mx::LIN_DGRAD : call == 2 ? mx::LIN_WGRAD : mx::LIN_FWD;
  return check_desc(desc) == MX_OK && mx::lin_product_streams(mx::make_lin_geom(desc), op, out, dtype, ld) ? 1 : 0;
}

size_t mx_grad_workspace_bytes(int32_t count) { return count > 0 ? mx::grad_workspace_bytes(count) : 0; }

mx_status mx_grad_norm(const mx_grad_list* list, float* norm, void* workspace, size_t ws_bytes, hipStream_t stream) {
  return grad(list, false, 0.0f, norm, workspace, ws_bytes, stream);
}

mx_status mx_grad_clip(const mx_grad_list* list, float max_norm, float* norm, void* workspace, size_t ws_bytes,
                       hipStream_t stream) {
  return grad(list, true, max_norm, norm, workspace, ws_bytes, stream);
}

}  // extern "C"
