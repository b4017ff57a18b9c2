// Internal interface of the microscaled linear layers: padded geometry, the
// tile layout of quantized matrices, the experts' segments, and the launchers
// behind the C ABI (linear_capi.cpp).  Arguments reaching a launcher have
// been validated on the host.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxlinear.h"

namespace mx {

// A form is stored in tiles of 32 rows x 64 contracted columns: 1 KiB of
// codes that one wave reads as 64 lanes x 16 bytes, which is the operand of
// v_mfma_scale_f32_32x32x64_f8f6f4 as it stands (lane l: row l%32, columns
// 32*(l/32) .. +31).  Scales of 4 tiles on top of each other (128 rows) are
// interleaved, so that one dword per lane serves 4 MFMA operands through the
// instruction's byte select.
constexpr int kTileR = 32, kTileC = 64;
constexpr int kTileBytes = 1024;
constexpr int kScaleBytes = 256;  // of 128 rows x 64 columns
constexpr int kPad = 128;         // rows and columns of a form are padded to this
constexpr int kStepTiles = 2;     // column tiles per step of a product's loop

inline int64_t pad128(int64_t v) { return (v + kPad - 1) / kPad * kPad; }

struct LinGeom {
  int64_t m, n, k;     // tokens, out and in features
  int e;               // experts (0: one layer)
  int64_t mp, np, kp;  // padded; mp holds every expert's padded tokens
  int ew;              // weight matrices: max(e, 1)
};

inline LinGeom make_lin_geom(const mx_linear_desc* d) {
  LinGeom g;
  g.m = d->tokens;
  g.n = d->out_features;
  g.k = d->in_features;
  g.e = d->experts;
  g.ew = d->experts > 0 ? d->experts : 1;
  g.np = pad128(g.n);
  g.kp = pad128(g.k);
  // each expert with tokens adds less than 128 rows of padding
  const int64_t used = g.m < g.ew ? g.m : g.ew;
  g.mp = g.e > 0 ? pad128(g.m + (kPad - 1) * used) : pad128(g.m);
  return g;
}

// Padded rows (the lines that stay) and columns (contracted) of one form.
// W: of one expert's matrix.
inline void form_dims(const LinGeom& g, mx_role role, mx_form form, int64_t& r, int64_t& c) {
  const int64_t a = role == MX_ROLE_WEIGHT ? g.np : g.mp;
  const int64_t b = role == MX_ROLE_GRAD ? g.np : g.kp;
  r = form == MX_FORM_ROWS ? a : b;
  c = form == MX_FORM_ROWS ? b : a;
}
inline int64_t form_matrices(const LinGeom& g, mx_role role) { return role == MX_ROLE_WEIGHT ? g.ew : 1; }

// The tokens of one expert.
struct Segment {
  int e;         // expert
  int len;       // tokens
  int64_t row0;  // first row in X, Y, dY
  int64_t prow;  // first padded row of the quantized forms
  int unit;      // the target's number within the expert
};

#ifdef __HIPCC__
// Inclusive scans over the wave's 64 lanes (of values >= 0 for the maximum):
// within rows of 16 lanes, then each row's last value into the next row, then
// the first half's into the second.
template <class Op>
__device__ __forceinline__ int wave_scan(int v, Op op) {
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false));  // row_shr:1
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false));  // row_shr:2
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false));  // row_shr:4
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false));  // row_shr:8
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false));  // row_bcast:15
  v = op(v, __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false));  // row_bcast:31
  return v;
}
__device__ __forceinline__ int wave_scan_max(int v) {
  return wave_scan(v, [](int a, int b) { return max(a, b); });
}
__device__ __forceinline__ int wave_scan_add(int v) {
  return wave_scan(v, [](int a, int b) { return a + b; });
}

// Finds the expert that holds unit `target` when expert e's tokens make
// ceil(len / per) units, and fills seg; false if there are fewer units.  By
// expert number instead (per = 0): target is the expert.  `total` receives
// the number of units of all experts when target is negative.  All 64 lanes
// of a wave call it together; the result is the same in each.  Offsets are
// read as their running maximum clamped to [0, m] (see mxlinear.h), so the
// lengths add up to m at most and padded rows stay inside the buffers.
__device__ __forceinline__ bool find_segment(const int32_t* __restrict__ off, int experts, int m, int target, int per,
                                    Segment& seg, int* total = nullptr) {
  const int lane = threadIdx.x & 63;
  int start = min(max(off[0], 0), m);  // first row of the chunk's first expert
  int units = 0, pads = 0;             // of the experts before the chunk; pads in units of 128 rows
  for (int base = 0; base < experts; base += 64) {
    const int e = base + lane;
    const int raw = e < experts ? min(max(off[e + 1], 0), m) : 0;
    const int end = max(wave_scan_max(raw), start);
    const int first = __builtin_amdgcn_update_dpp(start, end, 0x138, 0xF, 0xF, false);  // wave_shr:1
    const int len = end - first;
    const int u = per > 0 ? (len + per - 1) / per : (e < experts ? 1 : 0);
    const int p = (len + kPad - 1) / kPad;
    const int us = wave_scan_add(u), ps = wave_scan_add(p);
    const uint64_t hit = __ballot(target >= units + us - u && target < units + us);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      seg.e = base + l;
      seg.len = __builtin_amdgcn_readlane(len, l);
      seg.row0 = __builtin_amdgcn_readlane(first, l);
      seg.prow = static_cast<int64_t>(pads + __builtin_amdgcn_readlane(ps - p, l)) * kPad;
      seg.unit = target - (units + __builtin_amdgcn_readlane(us - u, l));
      return true;
    }
    units += __builtin_amdgcn_readlane(us, 63);
    pads += __builtin_amdgcn_readlane(ps, 63);
    start = __builtin_amdgcn_readlane(end, 63);
  }
  if (total) *total = units;
  return false;
}

// 16 bytes at an address of any alignment: the GPU takes 16-byte accesses that
// are not aligned, so rows need not start at multiples of 16 bytes.
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef i32x4 i32x4_any __attribute__((aligned(1)));
__device__ __forceinline__ i32x4 load16(const void* p) { return *static_cast<const i32x4_any*>(p); }
__device__ __forceinline__ void store16(void* p, i32x4 v) { *static_cast<i32x4_any*>(p) = v; }
// ... past the caches.  Results that no kernel reads soon are written so: a
// 16384x8192 dequantization to bf16 takes 50 us instead of 75, one of 1024x4096
// 4.0 instead of 4.1.
__device__ __forceinline__ void stream16(void* p, i32x4 v) { __builtin_nontemporal_store(v, static_cast<i32x4_any*>(p)); }

// The scaled MFMA's results and its operands, of which E2M1 uses the first half.
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ i32x8 operand(i32x4 v) { return i32x8{v.x, v.y, v.z, v.w, 0, 0, 0, 0}; }

// An element of a matrix of type T as fp32, and back (round to nearest even).
struct bf16_t { uint16_t v; };
struct f16_t { _Float16 v; };
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return __uint_as_float(static_cast<uint32_t>(v.v) << 16); }
__device__ __forceinline__ float to_f32(f16_t v) { return static_cast<float>(v.v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ bf16_t from_f32<bf16_t>(float v) {
  return {__builtin_bit_cast(uint16_t, static_cast<__bf16>(v))};
}
template <> __device__ __forceinline__ f16_t from_f32<f16_t>(float v) { return {static_cast<_Float16>(v)}; }
#endif

hipError_t launch_lin_quantize(const LinGeom& g, mx_role role, int block, const void* src, mx_dtype dtype, int64_t ld,
                               const int32_t* offsets, const mx_linear_qtensor* dst, mx_round rounding, uint64_t seed,
                               hipStream_t s);
hipError_t launch_lin_dequantize(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                 mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t s);

// The three products.  a: the operand whose rows are the output's rows.
enum LinOp { LIN_FWD, LIN_DGRAD, LIN_WGRAD };
size_t lin_product_workspace(const LinGeom& g, LinOp op);
hipError_t launch_lin_product(const LinGeom& g, LinOp op, const mx_linear_qtensor* aq, const mx_linear_qtensor* bq,
                              void* out, mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace,
                              hipStream_t s);
// fwd and dgrad with few tokens, where lin_few() says so.
bool lin_few(const LinGeom& g);
hipError_t launch_lin_few(const LinGeom& g, bool dgrad, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                          mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s);
// Quantize-and-multiply in one launch, where lin_fused() says so.
bool lin_fused(const LinGeom& g);
hipError_t launch_lin_fused(const LinGeom& g, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                            void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s);

// What a call launches, as the same rules choose it: for the tests, which say
// of each case which kernel it is meant for.
struct LinVariant {
  int32_t kernel;  // 0: none, 1: k_lin_few, 2: k_lin_few that quantizes, 3: k_lin_product
  int32_t size;    // stripes of a workgroup of k_lin_few, rows of a tile of k_lin_product
  int32_t splits;  // pieces of the contraction
  int32_t threads;
  int64_t workgroups;
};
LinVariant lin_product_variant(const LinGeom& g, LinOp op);
LinVariant lin_few_variant(const LinGeom& g, bool dgrad, bool fused);
bool lin_dequantize_streams(const void* dst, mx_dtype dtype, int64_t ld);
// Whether the rows of a matrix start at multiples of 64 bytes.
inline bool whole_lines(const void* p, int64_t row_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(row_bytes)) & 63) == 0;
}
bool lin_product_streams(const LinGeom& g, LinOp op, const void* out, mx_dtype dtype, int64_t ld);

// grad_clip.hip: the list's elements are at most kMaxGradElems.
constexpr int64_t kMaxGradElems = int64_t{1} << 43;
size_t grad_workspace_bytes(int32_t count);
hipError_t launch_grad_clip(const mx_grad_list* l, bool clip, float max_norm, float* norm, void* workspace, hipStream_t s);

}  // namespace mx
