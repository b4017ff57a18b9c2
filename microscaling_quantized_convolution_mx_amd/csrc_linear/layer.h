// Internal interface of the norm and the routing: launchers behind the C ABIs
// (layer_capi.cpp).  Arguments reaching a launcher have been validated on the
// host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "linear8.h"
#include "mxnorm.h"
#include "mxroute.h"

namespace mx {

struct NormFwd {
  const void *x, *residual, *weight;
  void *total, *y;
  int64_t ldx, ldr, ldt, ldy;
  mx_dtype dtype, w_dtype, y_dtype;
  uint8_t *codes, *scales;  // of the 8-bit row form, or NULL
  float* rstd;
};
struct NormBwd {
  const void *dy, *total, *dtotal, *weight;
  const float* rstd;
  void* dx;
  float* dweight;
  int64_t lddy, ldt, lddt, lddx;
  mx_dtype dy_dtype, dtype, w_dtype;
};
hipError_t launch_norm_fwd(const mx_norm_desc& d, const NormFwd& a, hipStream_t s);
size_t norm_workspace(const mx_norm_desc& d);
hipError_t launch_norm_bwd(const mx_norm_desc& d, const NormBwd& a, void* workspace, hipStream_t s);

size_t route_workspace(const mx_route_desc& d);
hipError_t launch_route_sort(const mx_route_desc& d, const int32_t* expert, int32_t* offsets, int32_t* rows, int32_t* order,
                             void* workspace, hipStream_t s);
hipError_t launch_route_gather(const mx_route_desc& d, const void* x, int64_t ldx, const int32_t* rows, void* out, int64_t ldo,
                               mx_dtype dtype, hipStream_t s);
// weight NULL: all are 1
hipError_t launch_route_combine(const mx_route_desc& d, const void* y, int64_t ldy, const int32_t* rows, const float* weight,
                                void* out, int64_t ldo, mx_dtype dtype, hipStream_t s);
hipError_t launch_route_combine_bwd(const mx_route_desc& d, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                                    const int32_t* rows, const float* weight, void* dy, int64_t lddy, float* dweight,
                                    mx_dtype dtype, hipStream_t s);

}  // namespace mx
