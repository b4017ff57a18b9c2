// Quantizer and dequantizer of the microscaled linear layers (E2M1 elements,
// one E8M0 scale per 1x32 or 32x32 block; layout in mxlinear.h).
//
//   e = clamp(floor(log2 amax_block) - 2, -127, 127),  code = Round(|x| 2^-e)
//
// The multiplication by a power of two is exact, so the only rounding is the
// one onto the E2M1 grid.
//
// One workgroup takes 128 rows x 128 columns, a wave one tile of 32 x 64:
// wave w rows 32 (w%4) on, columns 64 (w/4) on.  Lane l holds row l%32 and 32 consecutive columns
// (l/32): a 1x32 block is one lane's, so its maximum needs no exchange, its
// 32 codes are one 16-byte store, and the wave's 64 stores are the 1 KiB tile
// in order.  A 32x32 block is half a wave's: five exchanges.  The column form
// needs the codes of a column: the wave writes its tile to LDS and reads it
// back through the transposing 4-bit LDS read.  Scale bytes are gathered in
// LDS, since 128 rows share a dword.
//
// Bound by memory traffic for RNE; SR adds a 64-bit multiplicative hash per
// two elements and is bound by those integer operations.
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
  uint32_t ncb;        // 128-column blocks: block b takes column block b % ncb of row block b / ncb
  uint64_t seed;
};

constexpr int kStageRow = kTileC + 1;  // elements between rows in LDS: a column's rows lie in different banks

// VEC: rows start at multiples of 16 bytes.
template <class T, bool SQUARE, bool SR, bool VEC>
__global__ __launch_bounds__(512) void k_lin_quantize(const QuantParams p) {
  __shared__ __attribute__((aligned(16))) uint8_t tiles[SQUARE ? 8 : 1][kTileBytes];
  __shared__ __attribute__((aligned(16))) uint8_t rsc[2][kScaleBytes], csc[2][kScaleBytes];
  __shared__ T stage[VEC ? 1 : 8][VEC ? 1 : 32 * kStageRow];
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
  const int64_t ct0 = static_cast<int64_t>(bx) * 2;  // first column tile
  const int64_t c = (ct0 + t) * kTileC + 32 * half;
  float x[32];
  if constexpr (VEC) {
    if (r < nr && c < p.cols) {
      load32(src + r * p.ld, c, p.cols, true, x);
    } else {
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] = 0.0f;
    }
  } else {
    // a lane of its own for each column, so that a load takes one piece of a
    // row; through LDS to the lane that encodes it
    T* ls = stage[4 * t + wave];
    const int64_t lc = (ct0 + t) * kTileC + lane;
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
    __builtin_amdgcn_wave_barrier();
  }
  uint32_t m = amax32(x);
  if constexpr (SQUARE) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), d)));
  }
  const uint32_t code = block_code(m);
  const uint4 w = encode32<SR>(x, code, p.seed, static_cast<uint64_t>(row) * static_cast<uint64_t>(p.cols) + c);
  if (p.rcodes) {
    reinterpret_cast<uint4*>(p.rcodes + ((prow / kTileR + wave) * p.rkt + ct0 + t) * kTileBytes)[lane] = w;
    rsc[t][lane * 4 + wave] = static_cast<uint8_t>(code);
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
      const int64_t stripe = (crow0 + (ct0 + t) * kTileC) / kTileR + half;
      const int64_t pr = pr0 + 32 * wave;
      uint8_t* dst = p.ccodes + (stripe * p.ckt + pr / kTileC) * kTileBytes + ((pr / 32) & 1) * 512 + r * 16;
      *reinterpret_cast<int4*>(dst) = make_int4(q0.x, q0.y, q1.x, q1.y);
      // its scale: row r of stripe 2t + half, column half wave%2 of tile wave/2
      csc[wave >> 1][((wave & 1) * 32 + r) * 4 + 2 * t + half] = static_cast<uint8_t>(code);
    }
  }
  __syncthreads();
  const int q = threadIdx.x;  // 128 dwords of each form's scales
  if (q < 128) {
    if (p.rcodes) {
      uint8_t* d = p.rscales + ((prow / kPad) * p.rkt + ct0) * kScaleBytes;
      reinterpret_cast<uint32_t*>(d)[q] = reinterpret_cast<const uint32_t*>(rsc)[q];
    }
  } else if (SQUARE && p.ccodes && q < 256) {
    const int i = q - 128;
    uint8_t* d = p.cscales + (((crow0 + ct0 * kTileC) / kPad) * p.ckt + pr0 / kTileC) * kScaleBytes;
    reinterpret_cast<uint32_t*>(d)[i] = reinterpret_cast<const uint32_t*>(csc)[i];
  }
}

// 2^(code - 127): 2^-127 is an fp32 subnormal, 0xFF is NaN
__device__ __forceinline__ float scale_value(uint32_t code) {
  return code == 0xFFu ? __uint_as_float(0x7FC00000u) : (code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23));
}

// Workgroups as in the quantizer.  COLS: from the column form, where a lane's
// 16 bytes are a column of the matrix.
template <class T, bool COLS, bool VEC>
__global__ __launch_bounds__(512) void k_lin_dequantize(const QuantParams p, T* __restrict__ dst) {
  using F = Fmt<FMT_E2M1>;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6 & 3, t = threadIdx.x >> 8;
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
  auto value = [](uint32_t c, float scale) {
    const float v = code_value<F>(c & 7u) * scale;
    return from_f32<T>((c & 8u) ? -v : v);
  };
  if constexpr (!COLS) {
    // N elements, 16 bytes where rows allow, per lane and pass, so that a
    // store takes whole pieces of rows
    constexpr int N = VEC ? 16 / static_cast<int>(sizeof(T)) : 1;
    constexpr int P = kTileC / N;
    const uint8_t* tile = p.rcodes + ((prow / kTileR + wave) * p.rkt + ct0 + t) * kTileBytes;
    const uint8_t* sc = p.rscales + ((prow / kPad) * p.rkt + ct0 + t) * kScaleBytes + wave;
#pragma unroll 8
    for (int s = 0; s < kTileR * P / 64; ++s) {
      const int r = (s * 64 + lane) / P, j = (s * 64 + lane) % P * N, half = j >> 5;
      const uint8_t* at = tile + half * 512 + r * 16 + (j & 31) / 2;
      uint32_t w;
      if constexpr (N == 8) w = *reinterpret_cast<const uint32_t*>(at);
      else if constexpr (N == 4) w = *reinterpret_cast<const uint16_t*>(at);
      else w = *at >> (4 * (j & 1));
      const float scale = scale_value(sc[(half * 32 + r) * 4]);
      struct alignas(N * sizeof(T)) { T e[N]; } y;
#pragma unroll
      for (int i = 0; i < N; ++i) y.e[i] = value(w >> (4 * i), scale);
      const int64_t c = (ct0 + t) * kTileC + j;
      if (32 * wave + r >= left) continue;
      T* d = dst + (row0 + 32 * wave + r) * p.ld + c;
      if (c + N <= p.cols) {
        *reinterpret_cast<decltype(y)*>(d) = y;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (c + i < p.cols) d[i] = y.e[i];
      }
    }
  } else {
    const int r = lane & 31, half = lane >> 5;
    const int64_t stripe = (crow0 + (ct0 + t) * kTileC) / kTileR + half;
    const int64_t pr = pr0 + 32 * wave;
    const uint4 w = *reinterpret_cast<const uint4*>(p.ccodes + (stripe * p.ckt + pr / kTileC) * kTileBytes + ((pr / 32) & 1) * 512 + r * 16);
    const float scale = scale_value(p.cscales[((stripe / 4) * p.ckt + pr / kTileC) * kScaleBytes + (((pr / 32) & 1) * 32 + r) * 4 + (stripe & 3)]);
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    const int64_t c = (ct0 + t) * kTileC + 32 * half + r;
    if (c >= p.cols) return;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (32 * wave + i < left) dst[(row0 + 32 * wave + i) * p.ld + c] = value(ww[i >> 3] >> (4 * (i & 7)), scale);
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
  p.ncb = static_cast<uint32_t>(c / kPad);
  return p;
}

// 128x128 blocks of the padded matrix (of all experts)
dim3 make_grid(const LinGeom& g, mx_role role) {
  int64_t r, c;
  form_dims(g, role, MX_FORM_ROWS, r, c);
  return dim3(static_cast<unsigned>((c / kPad) * (r * form_matrices(g, role) / kPad)));
}

// Whether rows start at multiples of 16 bytes.
template <class T> bool vec_rows(const void* p, int64_t ld) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * static_cast<int64_t>(sizeof(T)) % 16 == 0;
}

template <class T>
void quantize_as(const QuantParams& p, dim3 grid, int block, bool sr, hipStream_t s) {
  const bool vec = vec_rows<T>(p.src, p.ld);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(512), 0, s, p); };
  if (block == 32) {
    if (sr) vec ? go(k_lin_quantize<T, true, true, true>) : go(k_lin_quantize<T, true, true, false>);
    else vec ? go(k_lin_quantize<T, true, false, true>) : go(k_lin_quantize<T, true, false, false>);
  } else {
    if (sr) vec ? go(k_lin_quantize<T, false, true, true>) : go(k_lin_quantize<T, false, true, false>);
    else vec ? go(k_lin_quantize<T, false, false, true>) : go(k_lin_quantize<T, false, false, false>);
  }
}

template <class T>
void dequantize_as(const QuantParams& p, dim3 grid, mx_form form, void* dst, hipStream_t s) {
  const bool vec = vec_rows<T>(dst, p.ld);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, grid, dim3(512), 0, s, p, static_cast<T*>(dst)); };
  if (form == MX_FORM_COLS) go(k_lin_dequantize<T, true, false>);
  else vec ? go(k_lin_dequantize<T, false, true>) : go(k_lin_dequantize<T, false, false>);
}

}  // namespace

hipError_t launch_lin_quantize(const LinGeom& g, mx_role role, int block, const void* src, mx_dtype dtype, int64_t ld,
                               const int32_t* offsets, const mx_linear_qtensor* dst, mx_round rounding, uint64_t seed,
                               hipStream_t s) {
  QuantParams p = make_params(g, role, ld, offsets, dst);
  p.src = src;
  p.seed = seed;
  const dim3 grid = make_grid(g, role);
  if (grid.x == 0) return hipSuccess;
  const bool sr = rounding == MX_SR;
  switch (dtype) {
    case MX_BF16: quantize_as<bf16_t>(p, grid, block, sr, s); break;
    case MX_F16: quantize_as<f16_t>(p, grid, block, sr, s); break;
    default: quantize_as<float>(p, grid, block, sr, s); break;
  }
  return hipGetLastError();
}

hipError_t launch_lin_dequantize(const LinGeom& g, mx_role role, mx_form form, const mx_linear_qtensor* q, void* dst,
                                 mx_dtype dtype, int64_t ld, const int32_t* offsets, hipStream_t s) {
  const QuantParams p = make_params(g, role, ld, offsets, q);
  const dim3 grid = make_grid(g, role);
  if (grid.x == 0) return hipSuccess;
  switch (dtype) {
    case MX_BF16: dequantize_as<bf16_t>(p, grid, form, dst, s); break;
    case MX_F16: dequantize_as<f16_t>(p, grid, form, dst, s); break;
    default: dequantize_as<float>(p, grid, form, dst, s); break;
  }
  return hipGetLastError();
}

}  // namespace mx
