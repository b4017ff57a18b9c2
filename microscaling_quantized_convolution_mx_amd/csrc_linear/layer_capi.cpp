// C ABI of the norm and the routing: host-side validation and dispatch.  The
// arguments are documented in include/mxnorm.h and include/mxroute.h.
#include "layer.h"
#include "linear_checks.h"

namespace {

using namespace mx;

bool overlaps_allowed(const void* a, int64_t lda, const void* b, int64_t ldb) { return a != b || lda == ldb; }

mx_status check_norm(const mx_norm_desc* d) {
  if (!d) return MX_ERR_NULL;
  if (!(d->eps >= 0.0f) || d->eps > std::numeric_limits<float>::max()) return MX_ERR_SHAPE;
  const mx_linear_desc act{d->tokens, 1, d->features, 0, 1};
  return check_desc(&act);
}

mx_status check_route(const mx_route_desc* d) {
  if (!d) return MX_ERR_NULL;
  if (d->tokens < 0 || d->choices < 1 || d->choices > MX_ROUTE_MAX_CHOICES || d->experts < 1 || d->experts > MX_LINEAR_MAX_EXPERTS)
    return MX_ERR_SHAPE;
  return static_cast<int64_t>(d->tokens) * d->choices < (int64_t{1} << 30) ? MX_OK : MX_ERR_SHAPE;
}

// The descriptor and rows of a move, its tokens' matrix and its rows' matrix.
mx_status check_move(const mx_route_desc* d, const int32_t* rows, const void* tokens, int64_t ldt, const void* matrix, int64_t ldm,
                     mx_dtype dtype) {
  mx_status st = check_route(d);
  if (st != MX_OK) return st;
  if (d->features < 1) return MX_ERR_SHAPE;
  if (d->tokens > 0 && !rows) return MX_ERR_NULL;
  if (!aligned(rows, 4)) return MX_ERR_ALIGN;
  if ((st = check_matrix(tokens, dtype, ldt, d->tokens, d->features)) != MX_OK) return st;
  return check_matrix(matrix, dtype, ldm, static_cast<int64_t>(d->tokens) * d->choices, d->features);
}

mx_status check_weight(const mx_route_desc* d, const float* weight) {
  if (d->tokens > 0 && !weight) return MX_ERR_NULL;
  return aligned(weight, 4) ? MX_OK : MX_ERR_ALIGN;
}

}  // namespace

extern "C" {

mx_status mx_norm_fwd(const mx_norm_desc* desc, const void* x, int64_t ldx, const void* residual, int64_t ldr, mx_dtype dtype,
                      const void* weight, mx_dtype w_dtype, void* total, int64_t ldt, void* y, mx_dtype y_dtype, int64_t ldy,
                      const mx_linear_qtensor* yq, float* rstd, hipStream_t stream) {
  mx_status st = check_norm(desc);
  if (st != MX_OK) return st;
  const int64_t m = desc->tokens, k = desc->features;
  if (m > 0 && !total && !y && !yq && !rstd) return MX_ERR_NULL;
  if ((st = check_matrix(x, dtype, ldx, m, k)) != MX_OK) return st;
  if (residual && (st = check_matrix(residual, dtype, ldr, m, k)) != MX_OK) return st;
  if ((st = check_matrix(weight, w_dtype, k, 1, k)) != MX_OK) return st;
  if (total && (st = check_matrix(total, dtype, ldt, m, k)) != MX_OK) return st;
  if (!known_dtype(y_dtype)) return MX_ERR_FORMAT;
  if (y && (st = check_matrix(y, y_dtype, ldy, m, k)) != MX_OK) return st;
  // total in the place of x or the residual has their rows
  if (total && (!overlaps_allowed(total, ldt, x, ldx) || !overlaps_allowed(total, ldt, residual, ldr))) return MX_ERR_SHAPE;
  NormFwd a{};
  if (yq) {
    const mx_linear_desc act{desc->tokens, 1, desc->features, 0, 1};
    if ((st = check_form(make_lin_geom(&act), MX_ROLE_ACT, MX_FORM_ROWS, yq)) != MX_OK) return st;
    a.codes = static_cast<uint8_t*>(yq->rows);
    a.scales = yq->row_scales;
  }
  if (!aligned(rstd, 4)) return MX_ERR_ALIGN;
  a.x = x;
  a.ldx = ldx;
  a.residual = residual;
  a.ldr = ldr;
  a.dtype = dtype;
  a.weight = weight;
  a.w_dtype = w_dtype;
  a.total = total;
  a.ldt = ldt;
  a.y = y;
  a.y_dtype = y_dtype;
  a.ldy = ldy;
  a.rstd = rstd;
  return launched(launch_norm_fwd(*desc, a, stream));
}

size_t mx_norm_workspace_bytes(const mx_norm_desc* desc) { return check_norm(desc) == MX_OK ? norm_workspace(*desc) : 0; }

mx_status mx_norm_bwd(const mx_norm_desc* desc, const void* dy, mx_dtype dy_dtype, int64_t lddy, const void* total, int64_t ldt,
                      const void* dtotal, int64_t lddt, mx_dtype dtype, const void* weight, mx_dtype w_dtype,
                      const float* rstd, void* dx, int64_t lddx, float* dweight, void* workspace, size_t ws_bytes,
                      hipStream_t stream) {
  mx_status st = check_norm(desc);
  if (st != MX_OK) return st;
  const int64_t m = desc->tokens, k = desc->features;
  if (m > 0 && !dx && !dweight) return MX_ERR_NULL;
  if ((st = check_matrix(dy, dy_dtype, lddy, m, k)) != MX_OK) return st;
  if ((st = check_matrix(total, dtype, ldt, m, k)) != MX_OK) return st;
  if (dtotal && (st = check_matrix(dtotal, dtype, lddt, m, k)) != MX_OK) return st;
  if ((st = check_matrix(weight, w_dtype, k, 1, k)) != MX_OK) return st;
  if (m > 0 && !rstd) return MX_ERR_NULL;
  if (dx && (st = check_matrix(dx, dtype, lddx, m, k)) != MX_OK) return st;
  if (!aligned(rstd, 4) || !aligned(dweight, 4)) return MX_ERR_ALIGN;
  if (dx && dx == dy && (dtype != dy_dtype || lddx != lddy)) return MX_ERR_SHAPE;
  if (dx && !overlaps_allowed(dx, lddx, dtotal, lddt)) return MX_ERR_SHAPE;
  if ((st = check_workspace(workspace, ws_bytes, dweight ? norm_workspace(*desc) : 0)) != MX_OK) return st;
  NormBwd a{};
  a.dy = dy;
  a.dy_dtype = dy_dtype;
  a.lddy = lddy;
  a.total = total;
  a.ldt = ldt;
  a.dtotal = dtotal;
  a.lddt = lddt;
  a.dtype = dtype;
  a.weight = weight;
  a.w_dtype = w_dtype;
  a.rstd = rstd;
  a.dx = dx;
  a.lddx = lddx;
  a.dweight = dweight;
  return launched(launch_norm_bwd(*desc, a, workspace, stream));
}

size_t mx_route_workspace_bytes(const mx_route_desc* desc) { return check_route(desc) == MX_OK ? route_workspace(*desc) : 0; }

mx_status mx_route_sort(const mx_route_desc* desc, const int32_t* expert, int32_t* offsets, int32_t* rows, int32_t* order,
                        void* workspace, size_t ws_bytes, hipStream_t stream) {
  mx_status st = check_route(desc);
  if (st != MX_OK) return st;
  if (!offsets || (desc->tokens > 0 && (!expert || !rows))) return MX_ERR_NULL;
  if (!aligned(expert, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(order, 4)) return MX_ERR_ALIGN;
  if ((st = check_workspace(workspace, ws_bytes, route_workspace(*desc))) != MX_OK) return st;
  return launched(launch_route_sort(*desc, expert, offsets, rows, order, workspace, stream));
}

mx_status mx_route_gather(const mx_route_desc* desc, const void* x, int64_t ldx, const int32_t* rows, void* out, int64_t ldo,
                          mx_dtype dtype, hipStream_t stream) {
  const mx_status st = check_move(desc, rows, x, ldx, out, ldo, dtype);
  return st != MX_OK ? st : launched(launch_route_gather(*desc, x, ldx, rows, out, ldo, dtype, stream));
}

mx_status mx_route_gather_bwd(const mx_route_desc* desc, const void* dout, int64_t ldo, const int32_t* rows, void* dx,
                              int64_t ldx, mx_dtype dtype, hipStream_t stream) {
  const mx_status st = check_move(desc, rows, dx, ldx, dout, ldo, dtype);
  return st != MX_OK ? st : launched(launch_route_combine(*desc, dout, ldo, rows, nullptr, dx, ldx, dtype, stream));
}

mx_status mx_route_combine(const mx_route_desc* desc, const void* y, int64_t ldy, const int32_t* rows, const float* weight,
                           void* out, int64_t ldo, mx_dtype dtype, hipStream_t stream) {
  mx_status st = check_move(desc, rows, out, ldo, y, ldy, dtype);
  if (st != MX_OK || (st = check_weight(desc, weight)) != MX_OK) return st;
  return launched(launch_route_combine(*desc, y, ldy, rows, weight, out, ldo, dtype, stream));
}

mx_status mx_route_combine_bwd(const mx_route_desc* desc, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                               const int32_t* rows, const float* weight, void* dy, int64_t lddy, float* dweight,
                               mx_dtype dtype, hipStream_t stream) {
  mx_status st = check_move(desc, rows, dout, ldo, y, ldy, dtype);
  if (st != MX_OK || (st = check_weight(desc, weight)) != MX_OK) return st;
  if (desc->tokens > 0 && !dy && !dweight) return MX_ERR_NULL;
  if (dy && (st = check_matrix(dy, dtype, lddy, static_cast<int64_t>(desc->tokens) * desc->choices, desc->features)) != MX_OK) return st;
  if (!aligned(dweight, 4)) return MX_ERR_ALIGN;
  return launched(launch_route_combine_bwd(*desc, dout, ldo, y, ldy, rows, weight, dy, lddy, dweight, dtype, stream));
}

}  // extern "C"
