// Quantizer and dequantizer of the linear layers in 8 bits (E4M3 elements, one
// E8M0 scale per 1x128 or 128x128 block; rounding and layout in mxlinear8.h).
//
// One workgroup takes 128 rows x 128 columns: every block in it is whole, of
// either size and form.  A lane holds 8 rows x 8 columns, its wave 32 rows x 128
// columns: 16 lanes side by side load 256 bytes of a row.  A row's maximum is
// 16 lanes', a column's goes through LDS.  The codes of both forms are put
// together in LDS, the column form's transposed by the lanes' 8 rows, and
// written as whole stripes.
//
// Bound by memory traffic: 16384x8192 bf16 74 us for the row form (5.4 TB/s, a
// large copy's rate), 79 for the column form, 107 for both (5.0); dequantizing
// the row form to bf16 64 (6.3 TB/s, most of it stores past the caches), to fp32
// 8192x8192 94.  The column form dequantizes at 3.3 TB/s: its bytes go through
// LDS one by one.  A lane's 8 loads are issued before the first is converted;
// each next to its conversion, in the branch for the row's end, both forms took
// 133 us.
#include <type_traits>

#include "linear8_codes.h"

namespace mx {
namespace {

struct Quant8Params {
  const void* src;
  int64_t ld;
  int64_t rows, cols;  // of the source matrix (W: of one expert's)
  int64_t mat;         // padded rows of one matrix (W: of one expert's)
  int experts;         // > 0: ragged token segments by offsets
  int weights;         // weight matrices, else 0
  const int32_t* offsets;
  uint8_t *rcodes, *rscales, *ccodes, *cscales;
  int64_t rkt, ckt;    // column tiles of a stripe in the two forms
  int64_t cmat;        // padded rows of one matrix in the column form
  uint32_t ncb;        // column blocks: block b takes column block b % ncb of 128-row block b / ncb
};

// The workgroup's 128 rows.
struct Rows {
  int64_t row0, left;  // first source row, rows from there on (of its matrix or expert)
  int64_t prow;        // first padded row in the row form
  int64_t pr0, crow0;  // first contracted column, and the matrix' first line, in the column form
};

__device__ __forceinline__ bool find_rows(const Quant8Params& p, uint32_t by, Rows& o) {
  const int64_t pb = static_cast<int64_t>(by) * kPad;
  if (p.experts > 0) {
    Segment s;
    if (!find_segment(p.offsets, p.experts, static_cast<int>(p.rows), static_cast<int>(by), kPad, s)) return false;
    o.row0 = s.row0 + static_cast<int64_t>(s.unit) * kPad;
    o.left = s.len - static_cast<int64_t>(s.unit) * kPad;
    o.prow = o.pr0 = s.prow + static_cast<int64_t>(s.unit) * kPad;
    o.crow0 = 0;
  } else {
    const int64_t e = p.weights > 0 ? pb / p.mat : 0;
    o.pr0 = pb - e * p.mat;
    o.row0 = e * p.rows + o.pr0;
    o.left = p.rows - o.pr0;
    o.prow = pb;
    o.crow0 = e * p.cmat;
  }
  return true;
}

constexpr int kBlockBytes = kPad * kPad;

// Place in LDS of the 16-byte piece of line r of a 128x128 block (of either
// form) and contracted columns 16j..: as in memory, with the lines of 8 permuted
// so that the writes of one instruction meet all banks.
__device__ __forceinline__ int piece_row(int r, int j) { return (r / 32) * 4096 + j * 512 + ((r & 31) ^ j) * 16; }
__device__ __forceinline__ int piece_col(int r, int j) { return (r / 32) * 4096 + j * 512 + ((r & 31) ^ (r >> 3 & 7)) * 16; }

template <class T, bool SQUARE, bool ROWS, bool COLS>
__global__ __launch_bounds__(256) void k_lin8_quantize(const Quant8Params p) {
  __shared__ __attribute__((aligned(16))) uint8_t rtile[ROWS ? kBlockBytes : 16], ctile[COLS ? kBlockBytes : 16];
  __shared__ __attribute__((aligned(16))) uint8_t rsc[kPad], csc[kPad];
  __shared__ uint32_t part[4][COLS || SQUARE ? kPad : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, q = lane & 15;
  const uint32_t by = blockIdx.x / p.ncb, bx = blockIdx.x - by * p.ncb;
  Rows at;
  if (!find_rows(p, by, at)) return;
  const int r0 = 32 * wave + 8 * g;
  const int64_t c = static_cast<int64_t>(bx) * kPad + 8 * q;
  Raw8<T> raw[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    raw[i] = load_raw8(static_cast<const T*>(p.src) + (at.row0 + r0 + i) * p.ld, c, r0 + i < at.left ? p.cols : 0);
  float x[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) unpack8(raw[i], x[i]);
  uint32_t rcode[8], ccode[8];
  if constexpr (SQUARE) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, amax8(x[i]));
    m = row16_max(m);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
    if (lane == 0) part[wave][0] = m;
    __syncthreads();
    const uint32_t code = block8_code(max(max(part[0][0], part[1][0]), max(part[2][0], part[3][0])));
#pragma unroll
    for (int i = 0; i < 8; ++i) rcode[i] = ccode[i] = code;
  } else {
    if constexpr (ROWS) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rcode[i] = block8_code(row16_max(amax8(x[i])));
    }
    if constexpr (COLS) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i][j]) & 0x7FFFFFFFu);
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
        m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
        if (g == 0) part[wave][8 * q + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        ccode[j] = block8_code(max(max(part[0][8 * q + j], part[1][8 * q + j]), max(part[2][8 * q + j], part[3][8 * q + j])));
    }
  }
  if constexpr (ROWS) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      *reinterpret_cast<uint2*>(rtile + piece_row(r0 + i, q / 2) + 8 * (q & 1)) = encode8x8(x[i], rcode[i]);
      if (q == 0) rsc[((r0 + i) & 31) * 4 + wave] = static_cast<uint8_t>(rcode[i]);
    }
  }
  if constexpr (COLS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = x[i][j];
      *reinterpret_cast<uint2*>(ctile + piece_col(8 * q + j, r0 / 16) + 8 * (g & 1)) = encode8x8(v, ccode[j]);
      if (wave == 0 && g == 0) csc[((8 * q + j) & 31) * 4 + q / 4] = static_cast<uint8_t>(ccode[j]);
    }
  }
  __syncthreads();
  // a stripe's two tiles of this block follow each other in memory
  if constexpr (ROWS) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(rtile + piece_row(32 * s + (tid & 31), tid >> 5));
      *reinterpret_cast<i32x4*>(p.rcodes + ((at.prow / kTileR + s) * p.rkt + 2 * static_cast<int64_t>(bx)) * k8TileBytes + 16 * tid) = v;
    }
    if (tid < 32)
      reinterpret_cast<uint32_t*>(p.rscales + (at.prow / kPad * (p.rkt / 2) + bx) * k8ScaleBytes)[tid] = reinterpret_cast<const uint32_t*>(rsc)[tid];
  }
  if constexpr (COLS) {
    const int64_t line = at.crow0 + static_cast<int64_t>(bx) * kPad;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const i32x4 v = *reinterpret_cast<const i32x4*>(ctile + piece_col(32 * s + (tid & 31), tid >> 5));
      *reinterpret_cast<i32x4*>(p.ccodes + ((line / kTileR + s) * p.ckt + at.pr0 / kTileC) * k8TileBytes + 16 * tid) = v;
    }
    if (tid >= 64 && tid < 96)
      reinterpret_cast<uint32_t*>(p.cscales + (line / kPad * (p.ckt / 2) + at.pr0 / kPad) * k8ScaleBytes)[tid - 64] =
          reinterpret_cast<const uint32_t*>(csc)[tid - 64];
  }
}

// The row form alone in 1x128 blocks: nothing joins the rows, so a workgroup
// takes a stripe of 32 and a lane 2 of them.  A launch that leaves CUs idle lasts
// as long as one lane's work, and large ones have more waves to hide memory with:
// 33x1024 2.6 us in a HIP graph, 3.9 by whole blocks; 301x1999 fp32 3.1 and 5.8;
// 2048x4096 bf16 5.3 and 5.7; 8192^2 bf16 30.6 and 31.2, fp32 58.5 and 61.8.
template <class T>
__global__ __launch_bounds__(256) void k_lin8_quantize_stripes(const Quant8Params p) {
  __shared__ __attribute__((aligned(16))) uint8_t rtile[4096];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, q = lane & 15;
  const uint32_t stripe = blockIdx.y, by = blockIdx.x / p.ncb, bx = blockIdx.x - by * p.ncb;
  Rows at;
  if (!find_rows(p, by, at)) return;
  const int r0 = 8 * wave + 2 * g;  // of the stripe
  const int64_t c = static_cast<int64_t>(bx) * kPad + 8 * q, first = 32 * static_cast<int64_t>(stripe) + r0;
  Raw8<T> raw[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    raw[i] = load_raw8(static_cast<const T*>(p.src) + (at.row0 + first + i) * p.ld, c, first + i < at.left ? p.cols : 0);
  uint8_t* scales = p.rscales + (at.prow / kPad * (p.rkt / 2) + bx) * k8ScaleBytes + stripe;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float x[8];
    unpack8(raw[i], x);
    const uint32_t code = block8_code(row16_max(amax8(x)));
    *reinterpret_cast<uint2*>(rtile + piece_row(r0 + i, q / 2) + 8 * (q & 1)) = encode8x8(x, code);
    if (q == 0) scales[(r0 + i) * 4] = static_cast<uint8_t>(code);
  }
  __syncthreads();
  *reinterpret_cast<i32x4*>(p.rcodes + ((at.prow / kTileR + stripe) * p.rkt + 2 * static_cast<int64_t>(bx)) * k8TileBytes + 16 * tid) =
      *reinterpret_cast<const i32x4*>(rtile + piece_row(tid & 31, tid >> 5));
}

// Workgroups, waves and lanes as in the quantizer, but a wave's rows in the
// order of memory: a load takes 4 rows that share their lines.  COLS: from the
// column form, byte by byte through LDS.  STREAM: past the caches, rows at
// multiples of 64 bytes.
template <class T, bool COLS, bool STREAM>
__global__ __launch_bounds__(256) void k_lin8_dequantize(const Quant8Params p, T* __restrict__ dst) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[COLS ? kBlockBytes : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, g = lane >> 4, q = lane & 15;
  const uint32_t by = blockIdx.x / p.ncb, bx = blockIdx.x - by * p.ncb;
  Rows at;
  if (!find_rows(p, by, at)) return;
  const int64_t c = static_cast<int64_t>(bx) * kPad + 8 * q;
  const int64_t line = at.crow0 + static_cast<int64_t>(bx) * kPad;
  const uint8_t* sc;
  if constexpr (COLS) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      *reinterpret_cast<i32x4*>(tile + 4096 * s + 16 * tid) =
          *reinterpret_cast<const i32x4*>(p.ccodes + ((line / kTileR + s) * p.ckt + at.pr0 / kTileC) * k8TileBytes + 16 * tid);
    __syncthreads();
    sc = p.cscales + (line / kPad * (p.ckt / 2) + at.pr0 / kPad) * k8ScaleBytes;
  } else {
    sc = p.rscales + (at.prow / kPad * (p.rkt / 2) + bx) * k8ScaleBytes;
  }
  if (c >= p.cols) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = 32 * wave + 4 * i + g;
    if (r >= at.left) continue;
    uint32_t w[2];
    float scale[COLS ? 8 : 1];
    if constexpr (COLS) {
      uint8_t b[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int l = 8 * q + j;
        b[j] = tile[(l / 32) * 4096 + (r / 16) * 512 + (l & 31) * 16 + (r & 15)];
        scale[j] = scale_value8(sc[(l & 31) * 4 + l / 32]);
      }
      __builtin_memcpy(w, b, 8);
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p.rcodes + ((at.prow / kTileR + wave) * p.rkt + 2 * static_cast<int64_t>(bx)) * k8TileBytes +
                                                      (q / 2) * 512 + (r & 31) * 16 + 8 * (q & 1));
      w[0] = v.x;
      w[1] = v.y;
      scale[0] = scale_value8(sc[(r & 31) * 4 + wave]);
    }
    float y[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w[h]), true);
      const float v[4] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
      for (int j = 0; j < 4; ++j) y[4 * h + j] = v[j] * scale[COLS ? 4 * h + j : 0];
    }
    store_row8<STREAM>(dst + (at.row0 + r) * p.ld, c, p.cols, y);
  }
}

Quant8Params make_params(const LinGeom& g, mx_role role, int64_t ld, const int32_t* offsets, const mx_linear_qtensor* q) {
  Quant8Params p{};
  int64_t r, c;
  form_dims(g, role, MX_FORM_ROWS, r, c);
  p.ld = ld;
  p.rows = role == MX_ROLE_WEIGHT ? g.n : g.m;
  p.cols = role == MX_ROLE_GRAD ? g.n : g.k;
  p.mat = r;
  p.cmat = c;
  p.experts = role == MX_ROLE_WEIGHT ? 0 : g.e;
  p.weights = role == MX_ROLE_WEIGHT ? g.ew : 0;
  p.offsets = offsets;
  p.rcodes = static_cast<uint8_t*>(q->rows);
  p.rscales = q->row_scales;
  p.ccodes = static_cast<uint8_t*>(q->cols);
  p.cscales = q->col_scales;
  p.rkt = c / kTileC;
  p.ckt = r / kTileC;
  p.ncb = static_cast<uint32_t>(c / kPad);
  return p;
}

// Workgroups of 128 x 128 over the padded matrix (of all experts).
unsigned groups(const LinGeom& g, mx_role role) {
  int64_t r, c;
  form_dims(g, role, MX_FORM_ROWS, r, c);
  return static_cast<unsigned>(c / kPad * (r * form_matrices(g, role) / kPad));
}

}  // namespace

hipError_t launch_lin8_quantize(const LinGeom& g, mx_role role, int block, const void* src, mx_dtype dtype, int64_t ld,
                                const int32_t* offsets, const mx_linear_qtensor* dst, hipStream_t s) {
  Quant8Params p = make_params(g, role, ld, offsets, dst);
  p.src = src;
  const unsigned n = groups(g, role);
  if (n == 0) return hipSuccess;
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(n), dim3(256), 0, s, p); };
  auto with = [&](auto t, auto square) {
    using T = decltype(t);
    constexpr bool S = decltype(square)::value;
    if (p.rcodes && p.ccodes) go(k_lin8_quantize<T, S, true, true>);
    else if (p.ccodes) go(k_lin8_quantize<T, S, false, true>);
    else if constexpr (S) go(k_lin8_quantize<T, true, true, false>);
    else hipLaunchKernelGGL(k_lin8_quantize_stripes<T>, dim3(n, 4), dim3(256), 0, s, p);
  };
  auto as = [&](auto t) { block == kPad ? with(t, std::true_type{}) : with(t, std::false_type{}); };
  switch (dtype) {
    case MX_BF16: as(bf16_t{}); break;
    case MX_F16: as(f16_t{}); break;
    default: as(float{}); break;
  }
  return hipGetLastError();
}

hipError_t launch_lin8_dequantize(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                  mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t s) {
  const Quant8Params p = make_params(g, role, ld, offsets, q);
  const unsigned n = groups(g, role);
  if (n == 0) return hipSuccess;
  auto as = [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(n), dim3(256), 0, s, p, static_cast<T*>(dst)); };
    auto with = [&](auto stream) {
      constexpr bool S = decltype(stream)::value;
      form == MX_FORM_COLS ? go(k_lin8_dequantize<T, true, S>) : go(k_lin8_dequantize<T, false, S>);
    };
    // (fp32: a lane's 32 bytes are two stores of half lines, which the caches join)
    sizeof(T) == 2 && lin_dequantize_streams(dst, dtype, ld) ? with(std::true_type{}) : with(std::false_type{});
  };
  switch (dtype) {
    case MX_BF16: as(bf16_t{}); break;
    case MX_F16: as(f16_t{}); break;
    default: as(float{}); break;
  }
  return hipGetLastError();
}

}  // namespace mx
