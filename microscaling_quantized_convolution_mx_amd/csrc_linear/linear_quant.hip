// Quantizer and dequantizer of the microscaled linear layers (E2M1 elements,
// one E8M0 scale per 1x32 or 32x32 block; layout in mxlinear.h).
//
//   e = clamp(floor(log2 amax_block) - 2, -127, 127),  code = Round(|x| 2^-e)
//
// The multiplication by a power of two is exact, so the only rounding is the
// one onto the E2M1 grid.
//
// One workgroup takes 128 rows x 128 columns, or 64 for SR, a wave a tile of
// 32 x 64.  (16384x8192 bf16, row form: RNE 67 us, 77 with 64 columns; SR 131,
// 139 with 128, whose 8 waves of ~90 registers fill a CU less evenly.)
// Lane l holds row l%32 and 32 consecutive columns
// (l/32): a 1x32 block is one lane's, so its maximum needs no exchange, its
// 32 codes are one 16-byte store, and the wave's 64 stores are the 1 KiB tile
// in order.  A 32x32 block is half a wave's: five exchanges.  The column form
// needs the codes of a column: the wave writes its tile to LDS and reads it
// back through the transposing 4-bit LDS read.  Scale bytes are gathered in
// LDS, since 128 rows share a dword.
//
// Bound by memory traffic for RNE: 16384x8192 bf16 67 us for the row form (5.0
// TB/s, a large copy's rate), 83 for both.  SR adds a 64-bit multiplicative hash
// per two elements and is bound by those integer operations, 1.0e12 elements/s:
// 131 us; neither other ways to encode nor half as many registers change that.
// Dequantizing to bf16 takes 50 us (6.8 TB/s).
#include <type_traits>

#include "linear.h"
#include "linear_codes.h"

namespace mx {
namespace {

typedef int i32x2v __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2v lds_i32x2v;

struct QuantParams {
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
  uint64_t seed;
};

// Column tiles of the quantizer's workgroup.
constexpr int tile_columns(bool sr) { return sr ? 1 : 2; }

constexpr int kStageRow = kTileC + 1;  // elements between rows in LDS: a column's rows lie in different banks

// ALIGNED: rows start at multiples of 16 bytes, and a lane loads its elements
// itself.  Where they do not, those loads would straddle cache lines (8192x8191
// bf16: 83 us); then a lane takes a column, so that a load covers a piece of
// one row, and the elements reach the lane that encodes them through LDS
// (36 us; 8192x8192 takes 34).
template <class T, bool SQUARE, bool SR, bool ALIGNED>
__global__ __launch_bounds__(256 * tile_columns(SR)) void k_lin_quantize(const QuantParams p) {
  constexpr int NT = tile_columns(SR);
  __shared__ __attribute__((aligned(16))) uint8_t tiles[SQUARE ? 4 * NT : 1][kTileBytes];
  __shared__ __attribute__((aligned(16))) uint8_t rsc[NT * kScaleBytes], csc[NT * kScaleBytes];
  __shared__ T stage[ALIGNED ? 1 : 4 * NT][ALIGNED ? 1 : 32 * kStageRow];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6 & 3, t = threadIdx.x >> 8;
  // the workgroup's 128 rows: source row and count, padded row, and the
  // matrix' base in the column form
  int64_t row0, prow, crow0 = 0, pr0 = 0;  // pr0: padded row inside the column form's matrix
  int64_t left;
  const uint32_t by = blockIdx.x / p.ncb, bx = blockIdx.x - by * p.ncb;
  const int64_t pb = static_cast<int64_t>(by) * kPad;
  if (p.experts > 0) {
    Segment s;
    if (!find_segment(p.offsets, p.experts, static_cast<int>(p.rows), static_cast<int>(by), kPad, s)) return;
    row0 = s.row0 + static_cast<int64_t>(s.unit) * kPad;
    left = s.len - static_cast<int64_t>(s.unit) * kPad;
    prow = s.prow + static_cast<int64_t>(s.unit) * kPad;
    pr0 = prow;
  } else if (p.weights > 0) {
    const int64_t e = pb / p.mat;
    pr0 = pb - e * p.mat;
    row0 = e * p.rows + pr0;
    left = p.rows - pr0;
    prow = pb;
    crow0 = e * p.cmat;
  } else {
    row0 = prow = pr0 = pb;
    left = p.rows - pb;
  }
  const int r = lane & 31, half = lane >> 5;
  const int64_t row = row0 + 32 * wave + r;
  const T* src = static_cast<const T*>(p.src) + (row0 + 32 * wave) * p.ld;
  const int nr = static_cast<int>(min<int64_t>(left - 32 * wave, 32));  // rows of the wave, if any
  const int64_t ct = static_cast<int64_t>(bx) * NT + t;  // column tile
  const int64_t c = ct * kTileC + 32 * half;
  float x[32];
  if constexpr (ALIGNED) {
    if (r < nr && c < p.cols) {
      load32(src + r * p.ld, c, p.cols, x);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    }
  } else {
    T* ls = stage[4 * t + wave];
    const int64_t lc = ct * kTileC + lane;
    const bool in = lc < p.cols && nr > 0;
    const T* col = src + (in ? lc : 0);
    T e[32]{};
    if (nr > 0) {
#pragma unroll
      for (int i = 0; i < 32; ++i) e[i] = col[min(i, nr - 1) * p.ld];
    }
#pragma unroll
    for (int i = 0; i < 32; ++i) ls[i * kStageRow + lane] = in && i < nr ? e[i] : T{};
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = to_f32(ls[r * kStageRow + 32 * half + i]);
  }
  uint32_t m = amax32(x);
  if constexpr (SQUARE) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  }
  const uint32_t code = block_code(m);
  const uint4 w = encode32<SR>(x, code, p.seed, static_cast<uint64_t>(row) * static_cast<uint64_t>(p.cols) + c,
                                (p.cols & 1) != 0);
  if (p.rcodes) {
    reinterpret_cast<uint4*>(p.rcodes + ((prow / kTileR + wave) * p.rkt + ct) * kTileBytes)[lane] = w;
    rsc[t * kScaleBytes + lane * 4 + wave] = static_cast<uint8_t>(code);
  }
  if constexpr (SQUARE) {
    if (p.ccodes) {
      // rows of the tile's two 32x32 blocks in LDS, columns out of it:
      // each transposing read takes 16 rows for 16 lanes' columns
      uint8_t* lt = tiles[4 * t + wave];
      reinterpret_cast<uint4*>(lt)[lane] = w;
      __builtin_amdgcn_wave_barrier();
      const uint8_t* b = lt + half * 512 + (lane & 15) * 16 + ((lane >> 4) & 1) * 8;
      const i32x2v q0 = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2v*)(b));
      const i32x2v q1 = __builtin_amdgcn_ds_read_tr4_b64_v2i32((lds_i32x2v*)(b + 256));
      // column tile of the column form: stripe = 32 source columns, its
      // columns = the padded rows
      const int64_t stripe = (crow0 + ct * kTileC) / kTileR + half;
      const int64_t pr = pr0 + 32 * wave;
      uint8_t* dst = p.ccodes + (stripe * p.ckt + pr / kTileC) * kTileBytes + ((pr / 32) & 1) * 512 + r * 16;
      *reinterpret_cast<int4*>(dst) = make_int4(q0.x, q0.y, q1.x, q1.y);
      // its scale: row r of the tile's stripe `half`, column half wave%2 of
      // column tile wave/2
      csc[((wave >> 1) * 64 + (wave & 1) * 32 + r) * 2 * NT + 2 * t + half] = static_cast<uint8_t>(code);
    }
  }
  __syncthreads();
  const int q = threadIdx.x;
  if (q < 64 * NT) {
    if (p.rcodes)
      reinterpret_cast<uint32_t*>(p.rscales + ((prow / kPad) * p.rkt + static_cast<int64_t>(bx) * NT) * kScaleBytes)[q] =
          reinterpret_cast<const uint32_t*>(rsc)[q];
  } else if (SQUARE && p.ccodes && q < 64 * NT + 128) {
    const int i = q - 64 * NT;
    const int64_t line = crow0 + static_cast<int64_t>(bx) * NT * kTileC;
    uint8_t* d = p.cscales + ((line / kPad) * p.ckt + pr0 / kTileC) * kScaleBytes + 4 * i;
    if constexpr (NT == 2) *reinterpret_cast<uint32_t*>(d) = reinterpret_cast<const uint32_t*>(csc)[i];
    else *reinterpret_cast<uint16_t*>(d + (line / kTileR & 3)) = reinterpret_cast<const uint16_t*>(csc)[i];  // two of a dword's four stripes
  }
}

// 2^(code - 127): 2^-127 is an fp32 subnormal, 0xFF is NaN
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code == 0xFFu ? __uint_as_float(0x7FC00000u) : (code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23));
}

// N consecutive codes as values in T: the hardware conversion gives the E2M1
// values, the scale is applied in fp32, where the product is exact, and the
// result is rounded to T.
template <class T, int N>
__device__ __forceinline__ void decode(uint32_t w, float scale, T* y) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  f32x2 v[(N + 1) / 2];
  v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
  v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
  if constexpr (N > 4) v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
  if constexpr (N > 4) v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
#pragma unroll
  for (int i = 0; i < N; ++i) y[i] = from_f32<T>(v[i / 2][i % 2] * scale);
}

// Workgroups of 128 rows x 128 columns as in the quantizer; wave w takes 16
// rows, a lane 16 bytes of them at a time, so that a store covers whole rows.
// COLS: from the column form, where a lane's 16 bytes are a column of 32 rows
// and a store writes one element of 64 columns (16384x8192 bf16 71 us, fp32
// 117; from the row form 50 and 98).  ALIGNED: rows start at
// multiples of 64 bytes; others are written through the caches, which join the
// lines that two stores share (8192x8191 bf16: 33 us, 67 past them; 16384x8200
// 97 and 120; 16384x8224, whole 64 bytes, 85 and 51).
template <class T, bool COLS, bool ALIGNED>
__global__ __launch_bounds__(512) void k_lin_dequantize(const QuantParams p, T* __restrict__ dst) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t row0, prow, crow0 = 0, pr0;
  int64_t left;
  const uint32_t by = blockIdx.x / p.ncb, bx = blockIdx.x - by * p.ncb;
  const int64_t pb = static_cast<int64_t>(by) * kPad;
  if (p.experts > 0) {
    Segment s;
    if (!find_segment(p.offsets, p.experts, static_cast<int>(p.rows), static_cast<int>(by), kPad, s)) return;
    row0 = s.row0 + static_cast<int64_t>(s.unit) * kPad;
    left = s.len - static_cast<int64_t>(s.unit) * kPad;
    prow = pr0 = s.prow + static_cast<int64_t>(s.unit) * kPad;
  } else {
    const int64_t e = p.weights > 0 ? pb / p.mat : 0;
    pr0 = pb - e * p.mat;
    row0 = e * p.rows + pr0;
    left = p.rows - pr0;
    prow = pb;
    crow0 = e * p.cmat;
  }
  const int64_t ct0 = static_cast<int64_t>(bx) * 2;
  if constexpr (!COLS) {
    constexpr int N = 16 / static_cast<int>(sizeof(T));
    constexpr int P = 2 * kTileC / N;  // pieces of a row
    const uint8_t* tiles = p.rcodes + ((prow / kTileR + wave / 2) * p.rkt + ct0) * kTileBytes;
    const uint8_t* sc = p.rscales + ((prow / kPad) * p.rkt + ct0) * kScaleBytes + wave / 2;
    const int r0 = 16 * (wave & 1);
#pragma unroll 8
    for (int s = 0; s < 16 * P / 64; ++s) {
      const int r = r0 + (s * 64 + lane) / P, j = (s * 64 + lane) % P * N;  // row of the stripe, column
      const uint8_t* at = tiles + (j >> 5) * 512 + r * 16 + (j & 31) / 2;
      uint32_t w;
      if constexpr (N == 8) w = *reinterpret_cast<const uint32_t*>(at);
      else w = *reinterpret_cast<const uint16_t*>(at);
      struct alignas(16) { T e[N]; } y;
      decode<T, N>(w, scale_value(sc[(j >> 6) * kScaleBytes + ((j >> 5 & 1) * 32 + r) * 4]), y.e);
      const int64_t row = 32 * (wave / 2) + r, c = ct0 * kTileC + j;
      if (row >= left) continue;
      T* d = dst + (row0 + row) * p.ld + c;
      if (c + N <= p.cols) {
        if constexpr (ALIGNED) stream16(d, __builtin_bit_cast(i32x4, y));
        else store16(d, __builtin_bit_cast(i32x4, y));
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c + i < p.cols) d[i] = y.e[i];
      }
    }
  } else {
    const int r = lane & 31, half = lane >> 5, rw = wave & 3, t = wave >> 2;
    const int64_t stripe = (crow0 + (ct0 + t) * kTileC) / kTileR + half;
    const int64_t pr = pr0 + 32 * rw;
    const uint4 w = *reinterpret_cast<const uint4*>(p.ccodes + (stripe * p.ckt + pr / kTileC) * kTileBytes + ((pr / 32) & 1) * 512 + r * 16);
    const float scale = scale_value(p.cscales[((stripe / 4) * p.ckt + pr / kTileC) * kScaleBytes + (((pr / 32) & 1) * 32 + r) * 4 + (stripe & 3)]);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const int64_t c = (ct0 + t) * kTileC + 32 * half + r;
    if (c >= p.cols) return;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      T y[8];
      decode<T, 8>(ww[q], scale, y);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (32 * rw + 8 * q + i < left) dst[(row0 + 32 * rw + 8 * q + i) * p.ld + c] = y[i];
    }
  }
}

QuantParams make_params(const LinGeom& g, mx_role role, int64_t ld, const int32_t* offsets, const mx_linear_qtensor* q) {
  QuantParams p{};
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
  return p;
}

// Workgroups of 128 rows x `width` columns over the padded matrix (of all experts).
dim3 make_grid(const LinGeom& g, mx_role role, int width, QuantParams& p) {
  int64_t r, c;
  form_dims(g, role, MX_FORM_ROWS, r, c);
  p.ncb = static_cast<uint32_t>(c / width);
  return dim3(static_cast<unsigned>(p.ncb * (r * form_matrices(g, role) / kPad)));
}

template <class T>
void quantize_as(const QuantParams& p, dim3 grid, int block, bool sr, hipStream_t s) {
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(256 * tile_columns(sr)), 0, s, p); };
  auto with = [&](auto aligned) {
    constexpr bool A = decltype(aligned)::value;
    if (block == 32) sr ? go(k_lin_quantize<T, true, true, A>) : go(k_lin_quantize<T, true, false, A>);
    else sr ? go(k_lin_quantize<T, false, true, A>) : go(k_lin_quantize<T, false, false, A>);
  };
  const bool aligned = reinterpret_cast<uintptr_t>(p.src) % 16 == 0 && p.ld * static_cast<int64_t>(sizeof(T)) % 16 == 0;
  aligned ? with(std::true_type{}) : with(std::false_type{});
}

template <class T>
void dequantize_as(const QuantParams& p, dim3 grid, mx_form form, void* dst, bool aligned, hipStream_t s) {
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(512), 0, s, p, static_cast<T*>(dst)); };
  if (form == MX_FORM_COLS) go(k_lin_dequantize<T, true, false>);
  else aligned ? go(k_lin_dequantize<T, false, true>) : go(k_lin_dequantize<T, false, false>);
}

}  // namespace

hipError_t launch_lin_quantize(const LinGeom& g, mx_role role, int block, const void* src, mx_dtype dtype, int64_t ld,
                               const int32_t* offsets, const mx_linear_qtensor* dst, mx_round rounding, uint64_t seed,
                               hipStream_t s) {
  QuantParams p = make_params(g, role, ld, offsets, dst);
  p.src = src;
  p.seed = seed;
  const bool sr = rounding == MX_SR;
  const dim3 grid = make_grid(g, role, tile_columns(sr) * kTileC, p);
  if (grid.x == 0) return hipSuccess;
  switch (dtype) {
    case MX_BF16: quantize_as<bf16_t>(p, grid, block, sr, s); break;
    case MX_F16: quantize_as<f16_t>(p, grid, block, sr, s); break;
    default: quantize_as<float>(p, grid, block, sr, s); break;
  }
  return hipGetLastError();
}

bool lin_dequantize_streams(const void* dst, mx_dtype dtype, int64_t ld) { return whole_lines(dst, ld * (dtype == MX_F32 ? 4 : 2)); }

hipError_t launch_lin_dequantize(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                 mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t s) {
  QuantParams p = make_params(g, role, ld, offsets, q);
  const dim3 grid = make_grid(g, role, kPad, p);
  if (grid.x == 0) return hipSuccess;
  const bool aligned = lin_dequantize_streams(dst, dtype, ld);
  switch (dtype) {
    case MX_BF16: dequantize_as<bf16_t>(p, grid, form, dst, aligned, s); break;
    case MX_F16: dequantize_as<f16_t>(p, grid, form, dst, aligned, s); break;
    default: dequantize_as<float>(p, grid, form, dst, aligned, s); break;
  }
  return hipGetLastError();
}

}  // namespace mx
