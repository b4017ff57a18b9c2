// Host-side checks of arguments that the C ABIs of the linear layers, the norm
// and the routing share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <limits>

#include "linear.h"

namespace mx {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline mx_status launched(hipError_t e) { return e == hipSuccess ? MX_OK : MX_ERR_LAUNCH; }

inline bool known_dtype(int t) { return t == MX_F32 || t == MX_BF16 || t == MX_F16; }
inline uintptr_t dtype_bytes(int t) { return t == MX_F32 ? 4 : 2; }

// Padded rows, column tiles and workgroups are 32-bit in the kernels.
constexpr int64_t kMaxLines = std::numeric_limits<int32_t>::max();

// square: the side of the square blocks, which is the other block size than 1.
inline mx_status check_desc(const mx_linear_desc* d, int square = 32) {
  if (!d) return MX_ERR_NULL;
  if (d->block != 1 && d->block != square) return MX_ERR_BLOCK;
  if (d->tokens < 0 || d->out_features <= 0 || d->in_features <= 0) return MX_ERR_SHAPE;
  if (d->experts < 0 || d->experts > MX_LINEAR_MAX_EXPERTS) return MX_ERR_SHAPE;
  // (in this order no product below overflows: every factor fits 32 bits)
  if (d->tokens > kMaxLines - 128 - 128 * static_cast<int64_t>(MX_LINEAR_MAX_EXPERTS) ||
      d->out_features > kMaxLines - 128 || d->in_features > kMaxLines - 128)
    return MX_ERR_SHAPE;
  const LinGeom g = make_lin_geom(d);
  if (g.np * g.ew > kMaxLines || g.kp * g.ew > kMaxLines) return MX_ERR_SHAPE;
  // 128x128 blocks and output tiles of every matrix: one launch each
  const int64_t mb = g.mp / 128, nb = g.np / 128, kb = g.kp / 128;
  const int64_t most = kMaxLines / 256;
  if (mb * nb > most || mb * kb > most || nb * kb > most / g.ew) return MX_ERR_SHAPE;
  return MX_OK;
}

inline mx_status check_role(mx_role r) {
  return (r == MX_ROLE_ACT || r == MX_ROLE_WEIGHT || r == MX_ROLE_GRAD) ? MX_OK : MX_ERR_ROLE;
}

inline int64_t form_tiles(const LinGeom& g, mx_role role, mx_form form) {
  int64_t r, c;
  form_dims(g, role, form, r, c);
  return (r / kTileR) * (c / kTileC) * form_matrices(g, role);
}

// The form's buffers, where it has elements.
inline mx_status check_form(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q) {
  if (!q) return MX_ERR_NULL;
  const void* codes = form == MX_FORM_ROWS ? q->rows : q->cols;
  const void* scales = form == MX_FORM_ROWS ? q->row_scales : q->col_scales;
  if (form_tiles(g, role, form) > 0 && (!codes || !scales)) return MX_ERR_NULL;
  if (!aligned(codes, 16) || !aligned(scales, 16)) return MX_ERR_ALIGN;
  return MX_OK;
}

// An unquantized matrix of rows x cols.
inline mx_status check_matrix(const void* p, int dtype, int64_t ld, int64_t rows, int64_t cols) {
  if (!known_dtype(dtype)) return MX_ERR_FORMAT;
  if (ld < cols || ld > std::numeric_limits<int64_t>::max() / 8 / (rows > 0 ? rows : 1)) return MX_ERR_SHAPE;
  if (rows > 0 && !p) return MX_ERR_NULL;
  if (!aligned(p, dtype_bytes(dtype))) return MX_ERR_ALIGN;
  return MX_OK;
}

inline mx_status check_offsets(const LinGeom& g, const int32_t* offsets) {
  if (g.e > 0 && !offsets) return MX_ERR_NULL;
  return aligned(offsets, 4) || g.e == 0 ? MX_OK : MX_ERR_ALIGN;
}

inline void matrix_dims(const LinGeom& g, mx_role role, int64_t& rows, int64_t& cols) {
  rows = role == MX_ROLE_WEIGHT ? g.n * g.ew : g.m;
  cols = role == MX_ROLE_GRAD ? g.n : g.k;
}

inline mx_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need > 0 && (!ws || bytes < need)) return MX_ERR_WORKSPACE;
  return aligned(ws, 16) ? MX_OK : MX_ERR_ALIGN;
}

}  // namespace mx
