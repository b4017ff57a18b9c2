// C ABI of the linear layers in 8 bits: host-side validation and dispatch.
// The arguments are documented in include/mxlinear8.h.
#include "linear8.h"
#include "linear_checks.h"

namespace {

using namespace mx;

// What _apply keeps of the quantized tokens in its workspace, before the
// product's partial sums.
size_t apply_code_bytes(const LinGeom& g) { return static_cast<size_t>(g.mp / kTileR * (g.kp / kTileC)) * k8TileBytes; }
size_t apply_scale_bytes(const LinGeom& g) { return static_cast<size_t>(g.mp / kPad * (g.kp / kPad)) * k8ScaleBytes; }
size_t apply_workspace(const LinGeom& g) {
  if (g.m == 0 || lin8_fused(g)) return 0;
  return apply_code_bytes(g) + apply_scale_bytes(g) + lin8_product_workspace(g, LIN_FWD);
}

mx_status product8(const mx_linear_desc* desc, LinOp op, const mx_linear_qtensor* aq, const mx_linear_qtensor* bq, void* out,
                   mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes, hipStream_t stream) {
  mx_status st = check_desc(desc, kPad);
  if (st != MX_OK) return st;
  const LinGeom g = make_lin_geom(desc);
  const mx_role ra = op == LIN_FWD ? MX_ROLE_ACT : MX_ROLE_GRAD, rb = op == LIN_WGRAD ? MX_ROLE_ACT : MX_ROLE_WEIGHT;
  if ((st = check_form(g, ra, op == LIN_WGRAD ? MX_FORM_COLS : MX_FORM_ROWS, aq)) != MX_OK) return st;
  if ((st = check_form(g, rb, op == LIN_FWD ? MX_FORM_ROWS : MX_FORM_COLS, bq)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, op == LIN_FWD ? MX_ROLE_GRAD : op == LIN_DGRAD ? MX_ROLE_ACT : MX_ROLE_WEIGHT, rows, cols);
  if ((st = check_matrix(out, dtype, ld, rows, cols)) != MX_OK) return st;
  if ((st = check_offsets(g, offsets)) != MX_OK) return st;
  if ((st = check_workspace(workspace, ws_bytes, lin8_product_workspace(g, op))) != MX_OK) return st;
  return launched(launch_lin8_product(g, op, aq, bq, out, dtype, ld, offsets, workspace, stream));
}

bool known_form(mx_form f) { return f == MX_FORM_ROWS || f == MX_FORM_COLS; }

}  // namespace

extern "C" {

size_t mx_linear8_code_bytes(const mx_linear_desc* desc, mx_role role, mx_form form) {
  if (check_desc(desc, kPad) != MX_OK || check_role(role) != MX_OK || !known_form(form)) return 0;
  return static_cast<size_t>(form_tiles(make_lin_geom(desc), role, form)) * k8TileBytes;
}

size_t mx_linear8_scale_bytes(const mx_linear_desc* desc, mx_role role, mx_form form) {
  // 8 tiles, 128 x 128, share 128 bytes of scales
  return mx_linear8_code_bytes(desc, role, form) / (8 * k8TileBytes) * k8ScaleBytes;
}

size_t mx_linear8_workspace_bytes(const mx_linear_desc* desc) {
  if (check_desc(desc, kPad) != MX_OK) return 0;
  const LinGeom g = make_lin_geom(desc);
  size_t need = apply_workspace(g);
  for (LinOp op : {LIN_FWD, LIN_DGRAD, LIN_WGRAD}) {
    const size_t b = lin8_product_workspace(g, op);
    need = b > need ? b : need;
  }
  return need;
}

mx_status mx_linear8_quantize(const mx_linear_desc* desc, mx_role role, const void* src, mx_dtype dtype, int64_t ld,
                              const int32_t* offsets, const mx_linear_qtensor* dst, hipStream_t stream) {
  mx_status st = check_desc(desc, kPad);
  if (st != MX_OK) return st;
  if ((st = check_role(role)) != MX_OK) return st;
  if (!dst) return MX_ERR_NULL;
  const LinGeom g = make_lin_geom(desc);
  // the forms that dst has, one at least where there is something to store
  if (dst->rows || !dst->cols) {
    if ((st = check_form(g, role, MX_FORM_ROWS, dst)) != MX_OK) return st;
  }
  if (dst->cols && (st = check_form(g, role, MX_FORM_COLS, dst)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, role, rows, cols);
  if ((st = check_matrix(src, dtype, ld, rows, cols)) != MX_OK) return st;
  if (role != MX_ROLE_WEIGHT && (st = check_offsets(g, offsets)) != MX_OK) return st;
  return launched(launch_lin8_quantize(g, role, desc->block, src, dtype, ld, offsets, dst, stream));
}

mx_status mx_linear8_dequantize(const mx_linear_desc* desc, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t stream) {
  mx_status st = check_desc(desc, kPad);
  if (st != MX_OK) return st;
  if ((st = check_role(role)) != MX_OK) return st;
  if (!known_form(form)) return MX_ERR_FORMAT;
  const LinGeom g = make_lin_geom(desc);
  if ((st = check_form(g, role, form, q)) != MX_OK) return st;
  int64_t rows, cols;
  matrix_dims(g, role, rows, cols);
  if ((st = check_matrix(dst, dtype, ld, rows, cols)) != MX_OK) return st;
  if (role != MX_ROLE_WEIGHT && (st = check_offsets(g, offsets)) != MX_OK) return st;
  return launched(launch_lin8_dequantize(g, role, form, q, dst, dtype, ld, offsets, stream));
}

mx_status mx_linear8_fwd(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                         mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                         hipStream_t stream) {
  return product8(desc, LIN_FWD, xq, wq, y, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear8_dgrad(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const mx_linear_qtensor* dyq, void* dx,
                           mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
  return product8(desc, LIN_DGRAD, dyq, wq, dx, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear8_wgrad(const mx_linear_desc* desc, const mx_linear_qtensor* dyq, const mx_linear_qtensor* xq, void* dw,
                           mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
  return product8(desc, LIN_WGRAD, dyq, xq, dw, dtype, ld, offsets, workspace, ws_bytes, stream);
}

mx_status mx_linear8_apply(const mx_linear_desc* desc, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                           void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, void* workspace, size_t ws_bytes,
                           hipStream_t stream) {
  mx_status st = check_desc(desc, kPad);
  if (st != MX_OK) return st;
  const LinGeom g = make_lin_geom(desc);
  if ((st = check_form(g, MX_ROLE_WEIGHT, MX_FORM_ROWS, wq)) != MX_OK) return st;
  if ((st = check_matrix(x, x_dtype, ldx, g.m, g.k)) != MX_OK) return st;
  if ((st = check_matrix(y, y_dtype, ldy, g.m, g.n)) != MX_OK) return st;
  if ((st = check_offsets(g, offsets)) != MX_OK) return st;
  if ((st = check_workspace(workspace, ws_bytes, apply_workspace(g))) != MX_OK) return st;
  if (g.m == 0) return MX_OK;
  if (lin8_fused(g)) return launched(launch_lin8_fused(g, wq, x, x_dtype, ldx, y, y_dtype, ldy, offsets, stream));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const mx_linear_qtensor xq{ws, ws + apply_code_bytes(g), nullptr, nullptr};
  const hipError_t e = launch_lin8_quantize(g, MX_ROLE_ACT, 1, x, x_dtype, ldx, offsets, &xq, stream);
  if (e != hipSuccess) return MX_ERR_LAUNCH;
  return launched(launch_lin8_product(g, LIN_FWD, &xq, wq, y, y_dtype, ldy, offsets, ws + apply_code_bytes(g) + apply_scale_bytes(g), stream));
}

// Not part of the ABI: mx_internal_linear_variant of the layers in 8 bits, which
// depends on the output's type.
mx_status mx_internal_linear8_variant(const mx_linear_desc* desc, int call, mx_dtype dtype, int64_t* out) {
  const mx_status st = check_desc(desc, kPad);
  if (st != MX_OK) return st;
  if (!out) return MX_ERR_NULL;
  const LinGeom g = make_lin_geom(desc);
  const LinVariant v = call == 3 && g.m > 0 && lin8_fused(g)
                           ? lin8_few_variant(g, false, true)
                           : lin8_product_variant(g, call == 1 ? LIN_DGRAD : call == 2 ? LIN_WGRAD : LIN_FWD, dtype);
  out[0] = v.kernel;
  out[1] = v.size;
  out[2] = v.splits;
  out[3] = v.threads;
  out[4] = v.workgroups;
  return MX_OK;
}

}  // extern "C"
