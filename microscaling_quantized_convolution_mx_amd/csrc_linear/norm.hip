// The root-mean-square norm with the residual's addition, and its gradients.
//
//   fwd   total = x + residual, rstd = (mean total^2 + eps)^(-1/2), y = total rstd weight
//   bwd   h = total rstd, g = dy weight,
//         dx = rstd (g - h mean(g h)) + dtotal,  dweight = sum over tokens of dy h
//
// Bound by memory traffic: everything is read and written once.  A row is held
// in the registers of a wave or a workgroup, CH pieces of 8 elements of each
// thread, between the sum over it and the results that need the sum.
// Workgroups take rows in turn and keep the weight, and in the backward pass
// the weight's gradient over their rows, in registers; those partial sums are
// added by a second kernel in a fixed order.  Rows too long for registers are
// read twice (4096x20480 bf16 forward 148 us, backward 272; 4096x16384 102 and 118).
//
// Measured: 16384x4096 bf16 forward 103 us (5.2 TB/s, a large copy's rate), to 8 bits
// 98 (4.8), backward 104 (5.2, the second kernel among it); 16384x5000, rows that share
// cache lines, forward 137 (4.8), to 8 bits 176 (3.3; why is open).  One row at a time
// fills the CUs better than several, whose registers leave room for fewer waves
// (8192x8192 forward 101 us, 116 with 2 rows at a time, 122 with 4).  So does keeping
// the row and the weight in fp32 between the arithmetic in fp64 (to 8 bits 98 us, 116
// with both in fp64 registers; 16384x5000 176 and 248).
#include <algorithm>
#include <type_traits>

#include "layer.h"
#include "linear8_codes.h"

namespace mx {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

struct FwdParams {
  NormFwd a;
  int tokens, features, padded_rows;  // padded_rows: with codes, those of the 8-bit form
  int chunks;                         // pieces of 8 of a row, with codes of the padded one
  int64_t kt;                         // column tiles of the 8-bit form
  float eps;
};
struct BwdParams {
  NormBwd a;
  int tokens, features;
  float* partial;
};

// 8 elements of a matrix of a type known at run time.
__device__ __forceinline__ void load_any(const void* p, mx_dtype t, int64_t row, int64_t c, int64_t cols, float* x) {
  if (t == MX_BF16) load_row8(static_cast<const bf16_t*>(p) + row, c, cols, x);
  else if (t == MX_F16) load_row8(static_cast<const f16_t*>(p) + row, c, cols, x);
  else load_row8(static_cast<const float*>(p) + row, c, cols, x);
}
__device__ __forceinline__ void store_any(void* p, mx_dtype t, int64_t row, int64_t c, int64_t cols, const float* x) {
  if (t == MX_BF16) store_row8(static_cast<bf16_t*>(p) + row, c, cols, x);
  else if (t == MX_F16) store_row8(static_cast<f16_t*>(p) + row, c, cols, x);
  else store_row8(static_cast<float*>(p) + row, c, cols, x);
}

// v of another lane of the row of 16 (DPP).
template <int CTRL>
__device__ __forceinline__ float dpp(float v) { return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true)); }
template <int CTRL>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(b), CTRL, 0xF, 0xF, true));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(b >> 32), CTRL, 0xF, 0xF, true));
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ float from_lane(float v, int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); }
__device__ __forceinline__ double from_lane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b), l));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), l));
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// The sum over a wave, in every lane: rows of 16 lanes (pairs, fours, mirrored
// halves), then the four rows.
template <class S>
__device__ __forceinline__ S wave_sum(S v) {
  v += dpp<0xB1>(v);
  v += dpp<0x4E>(v);
  v += dpp<0x141>(v);
  v += dpp<0x140>(v);
  return (from_lane(v, 0) + from_lane(v, 16)) + (from_lane(v, 32) + from_lane(v, 48));
}

// The sum over a row, a wave's (WAVE) or the workgroup's of at most MOST threads.
// `buf` is used in turn, so that one barrier is enough: a wave that writes half
// `turn` again has passed the barrier between, which all have reached after
// reading it.
template <bool WAVE, int MOST, class S>
__device__ __forceinline__ S row_sum(S v, S (*buf)[MOST / 64], int turn) {
  v = wave_sum(v);
  if constexpr (!WAVE) {
    const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[turn][wave] = v;
    __syncthreads();
    v = buf[turn][0];
    for (int w = 1; w < waves; ++w) v += buf[turn][w];
  }
  return v;
}

// 1 / sqrt(x): the hardware's value, good to some 23 bits, and two Newton steps.
__device__ __forceinline__ double inverse_root(double x) {
  const double r0 = __builtin_amdgcn_rsq(x);
  double r = r0;
#pragma unroll
  for (int i = 0; i < 2; ++i) r = __builtin_fma(0.5 * r, __builtin_fma(-(x * r), r, 1.0), r);
  return r0 > 0.0 && r0 < __builtin_inf() ? r : r0;
}

// q + x^2 of 8 elements.  fp64 has room for the square of every fp32: in fp32 the
// squares of elements over 2^64 would be Inf, or their sum by how many a thread
// has, and those under 2^-75 zero.
__device__ __forceinline__ double add_squares(const float* x, double q) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double v = x[i];
    q = __builtin_fma(v, v, q);
  }
  return q;
}

// y rounded to fp32, inexact values to the neighbour with an odd last bit: of the
// 24 bits the last then says whether there was more, so that rounding the result
// again, to E4M3's 4, gives what rounding y once would.
__device__ __forceinline__ float round_odd(double y) {
  const float f = static_cast<float>(y);
  const double d = y - static_cast<double>(f);  // what y has more than f, exactly
  // towards zero where the signs differ (f has y's), and then odd; an overflow stays as
  // it is, d being infinite then
  const int b = __float_as_int(f), up = static_cast<int>(__builtin_bit_cast(uint64_t, d) >> 32);
  constexpr int kFinite = 0x198;  // a normal or subnormal number of either sign, not zero
  return __int_as_float(__builtin_amdgcn_class(d, kFinite) ? (b + ((up ^ b) >> 31)) | 1 : b);
}

// What goes to 8 bits: t rstd w with rstd in fp64.  t w is exact there, the rest is
// off by (32 + features / 1024) 2^-53 at most: codes differ from those of the exact
// product only where it is nearer to a tie than that.
__device__ __forceinline__ float code_value(float t, double r, float w) {
  return round_odd(static_cast<double>(t) * static_cast<double>(w) * r);
}

__device__ __forceinline__ int64_t code_place(const FwdParams& p, int64_t row, int64_t c) {
  return ((row / kTileR) * p.kt + c / kTileC) * k8TileBytes + (c / 16 % 4) * 512 + (row % 32) * 16;
}
// 8 values as codes of the 8-bit row form: 16 lanes share a block of 128, whose
// scale is stored.
__device__ __forceinline__ uint2 encode_codes(const FwdParams& p, int64_t row, int64_t c, const float* y) {
  const uint32_t code = block8_code(row16_max(amax8(y)));
  if (c % kPad == 0)
    p.a.scales[(row / kPad * (p.kt / 2) + c / kPad) * k8ScaleBytes + (row % 32) * 4 + row / 32 % 4] = static_cast<uint8_t>(code);
  return encode8x8(y, code);
}

template <class T>
__device__ __forceinline__ void add_residual(Raw8<T>& v, const Raw8<T>& r, float* t) {
  float b[8];
  unpack8(v, t);
  unpack8(r, b);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] += b[i];
  v = pack8<T>(t);
}

// Rows are taken GROUP at a time, one after the other.  With GROUP = 4 the codes
// of 4 rows are written together, 64 consecutive bytes of 16 columns each: a
// wave keeps its columns' codes in LDS of its own until it has all four
// (16384x4096 bf16 98 us, 131 with 8 bytes written at a time; 16384x1024 27 and 26).
template <class T, bool WAVE, int MOST, int CH, bool CODES, int GROUP>
__global__ __launch_bounds__(MOST) void k_norm_fwd(const FwdParams p) {
  const int tpr = WAVE ? 64 : blockDim.x;     // threads of a row
  constexpr int RPW = WAVE ? MOST / 64 : 1;  // rows of a workgroup at a time
  __shared__ double buf[2][MOST / 64];
  extern __shared__ __attribute__((aligned(16))) uint8_t stage[];  // GROUP > 1: 512 * GROUP bytes of each wave and piece
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, t = WAVE ? lane : threadIdx.x;
  float w[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) load_any(p.a.weight, p.a.w_dtype, 0, (j * tpr + t) * 8, p.features, w[j]);
  const int rows = CODES ? p.padded_rows : p.tokens;
  int turn = 0;
  for (int64_t row0 = (static_cast<int64_t>(blockIdx.x) * RPW + (WAVE ? wave : 0)) * GROUP; row0 < rows;
       row0 += static_cast<int64_t>(gridDim.x) * RPW * GROUP) {
    for (int b = 0; b < GROUP; ++b, turn ^= 1) {
      const int64_t row = row0 + b;
      const bool in = row < p.tokens;
      Raw8<T> v[CH];
#pragma unroll
      for (int j = 0; j < CH; ++j) v[j] = load_raw8(static_cast<const T*>(p.a.x) + row * p.a.ldx, (j * tpr + t) * 8, in ? p.features : 0);
      if (p.a.residual) {
        Raw8<T> r[CH];
#pragma unroll
        for (int j = 0; j < CH; ++j)
          r[j] = load_raw8(static_cast<const T*>(p.a.residual) + row * p.a.ldr, (j * tpr + t) * 8, in ? p.features : 0);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          float sum[8];
          add_residual(v[j], r[j], sum);
        }
      }
      double q = 0.0;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        float x[8];
        unpack8(v[j], x);
        q = add_squares(x, q);
      }
      const double s = row_sum<WAVE, MOST>(q, buf, turn);
      const double r = inverse_root(s / p.features + static_cast<double>(p.eps));
      const float hi = static_cast<float>(r);
      if (p.a.rstd && t == 0 && in) p.a.rstd[row] = hi;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        const int c = (j * tpr + t) * 8;
        float x[8], y[8];
        unpack8(v[j], x);
        if (in && c < p.features) {
          if (p.a.total) store_raw8(static_cast<T*>(p.a.total) + row * p.a.ldt, c, p.features, v[j]);
          if (p.a.y) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = x[i] * hi * w[j][i];
            store_any(p.a.y, p.a.y_dtype, row * p.a.ldy, c, p.features, y);
          }
        }
        if constexpr (CODES) {
          if (c < 8 * p.chunks) {
            // (a row's padded columns are zeros of x and the weight; where rstd is not finite they share a block of NaNs)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // (the empty asm keeps the row and the weight in fp32 until here: in fp64 they would take twice the registers)
              asm("" : "+v"(x[i]), "+v"(w[j][i]));
              y[i] = in ? code_value(x[i], r, w[j][i]) : 0.0f;
            }
            const uint2 e = encode_codes(p, row, c, y);
            if constexpr (GROUP == 1) *reinterpret_cast<uint2*>(p.a.codes + code_place(p, row, c) + c % 16) = e;
            else *reinterpret_cast<uint2*>(stage + (wave * CH + j) * 512 * GROUP + ((lane / 2) * GROUP + b) * 16 + 8 * (lane % 2)) = e;
          }
        }
      }
    }
    if constexpr (CODES && GROUP > 1) {
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int k = 0; k < GROUP / 2; ++k) {
          const int piece = k * 64 + lane, c = (j * tpr + t - lane) * 8 + piece / GROUP * 16;
          if (c < 8 * p.chunks)
            *reinterpret_cast<i32x4*>(p.a.codes + code_place(p, row0 + piece % GROUP, c)) =
                *reinterpret_cast<const i32x4*>(stage + (wave * CH + j) * 512 * GROUP + piece * 16);
        }
      __builtin_amdgcn_wave_barrier();
    }
  }
}

template <class T>
__device__ __forceinline__ void load_total(const FwdParams& p, int64_t row, int64_t c, float* v) {
  Raw8<T> x = load_raw8(static_cast<const T*>(p.a.x) + row * p.a.ldx, c, p.features);
  if (p.a.residual) add_residual(x, load_raw8(static_cast<const T*>(p.a.residual) + row * p.a.ldr, c, p.features), v);
  unpack8(x, v);
}

// Rows of any length, read twice.
template <class T, bool CODES>
__global__ __launch_bounds__(1024) void k_norm_fwd_long(const FwdParams p) {
  constexpr int TPR = 1024;
  __shared__ double buf[2][TPR / 64];
  const int rows = CODES ? p.padded_rows : p.tokens;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    double s = 0.0;
    if (row < p.tokens) {
      for (int64_t c = 8 * threadIdx.x; c < p.features; c += 8 * TPR) {
        float v[8];
        load_total<T>(p, row, c, v);
        s = add_squares(v, s);
      }
    }
    s = row_sum<false, TPR>(s, buf, turn);
    const double r = inverse_root(s / p.features + static_cast<double>(p.eps));
    const float hi = static_cast<float>(r);
    if (p.a.rstd && threadIdx.x == 0 && row < p.tokens) p.a.rstd[row] = hi;
    for (int64_t c = 8 * threadIdx.x; c < 8 * static_cast<int64_t>(p.chunks); c += 8 * TPR) {
      float v[8] = {}, w[8] = {}, y[8];
      const bool in = row < p.tokens && c < p.features;
      if (in) {
        load_total<T>(p, row, c, v);
        load_any(p.a.weight, p.a.w_dtype, 0, c, p.features, w);
        if (p.a.total) store_row8(static_cast<T*>(p.a.total) + row * p.a.ldt, c, p.features, v);
      }
      if (in && p.a.y) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = v[i] * hi * w[i];
        store_any(p.a.y, p.a.y_dtype, row * p.a.ldy, c, p.features, y);
      }
      if constexpr (CODES) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = in && c + i < p.features ? code_value(v[i], r, w[i]) : 0.0f;
        *reinterpret_cast<uint2*>(p.a.codes + code_place(p, row, c) + c % 16) = encode_codes(p, row, c, y);
      }
    }
  }
}

// SAME: dy has total's type.
template <class T, bool SAME, bool WAVE, int MOST, int CH>
__global__ __launch_bounds__(MOST) void k_norm_bwd(const BwdParams p) {
  const int tpr = WAVE ? 64 : blockDim.x;
  constexpr int RPW = WAVE ? MOST / 64 : 1;
  __shared__ float buf[2][MOST / 64];
  const int t = WAVE ? threadIdx.x & 63 : threadIdx.x, group = WAVE ? threadIdx.x >> 6 : 0;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    load_any(p.a.weight, p.a.w_dtype, 0, (j * tpr + t) * 8, p.features, w[j]);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  }
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + group; row < p.tokens; row += static_cast<int64_t>(gridDim.x) * RPW, turn ^= 1) {
    Raw8<T> gr[CH], hr[CH], dr[CH];
    const float r = p.a.rstd[row];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * tpr + t) * 8;
      if constexpr (SAME) gr[j] = load_raw8(static_cast<const T*>(p.a.dy) + row * p.a.lddy, c, p.features);
      hr[j] = load_raw8(static_cast<const T*>(p.a.total) + row * p.a.ldt, c, p.features);
      dr[j] = {};
      if (p.a.dtotal) dr[j] = load_raw8(static_cast<const T*>(p.a.dtotal) + row * p.a.lddt, c, p.features);
    }
    float g[CH][8], h[CH][8], s = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if constexpr (SAME) unpack8(gr[j], g[j]);
      else load_any(p.a.dy, p.a.dy_dtype, row * p.a.lddy, (j * tpr + t) * 8, p.features, g[j]);
      unpack8(hr[j], h[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[j][i] *= r;
        dw[j][i] += g[j][i] * h[j][i];
        g[j][i] *= w[j][i];
        s += g[j][i] * h[j][i];
      }
    }
    if (!p.a.dx) continue;
    const float m = row_sum<WAVE, MOST>(s, buf, turn) / static_cast<float>(p.features);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * tpr + t) * 8;
      float d[8];
      unpack8(dr[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += r * (g[j][i] - h[j][i] * m);
      if (c < p.features) store_row8(static_cast<T*>(p.a.dx) + row * p.a.lddx, c, p.features, d);
    }
  }
  if (!p.partial) return;
  if constexpr (RPW > 1) {
    // the workgroup's waves in their order
    __shared__ float sum[RPW][64 * 8 + 8];
    const int rw = group;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[rw][8 * t + i] = dw[j][i];
      __syncthreads();
      if (rw == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          for (int q = 1; q < RPW; ++q) dw[j][i] += sum[q][8 * t + i];
      }
    }
    if (rw > 0) return;
  }
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (j * tpr + t) * 8;
    if (c < p.features) store_row8(p.partial + static_cast<int64_t>(blockIdx.x) * p.features, c, p.features, dw[j]);
  }
}

template <class T>
__global__ __launch_bounds__(1024) void k_norm_bwd_long(const BwdParams p) {
  constexpr int TPR = 1024;
  __shared__ float buf[2][TPR / 64];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.tokens; row += gridDim.x, turn ^= 1) {
    const float r = p.a.rstd[row];
    float m = 0.0f;
    for (int pass = 0; pass < 2; ++pass) {
      float s = 0.0f;
      for (int64_t c = 8 * threadIdx.x; c < p.features; c += 8 * TPR) {
        float g[8], h[8], w[8];
        load_any(p.a.dy, p.a.dy_dtype, row * p.a.lddy, c, p.features, g);
        load_row8(static_cast<const T*>(p.a.total) + row * p.a.ldt, c, p.features, h);
        load_any(p.a.weight, p.a.w_dtype, 0, c, p.features, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          h[i] *= r;
          g[i] *= w[i];
          s += g[i] * h[i];
        }
        if (pass == 0) continue;
        float d[8] = {};
        if (p.a.dtotal) load_row8(static_cast<const T*>(p.a.dtotal) + row * p.a.lddt, c, p.features, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] += r * (g[i] - h[i] * m);
        store_row8(static_cast<T*>(p.a.dx) + row * p.a.lddx, c, p.features, d);
      }
      if (pass == 0) m = row_sum<false, TPR>(s, buf, turn) / static_cast<float>(p.features);
    }
  }
}

// The weight's gradient over every gridDim.y-th row, where rows are long: a
// thread takes 8 columns.
template <class T>
__global__ __launch_bounds__(256) void k_norm_dweight(const BwdParams p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= p.features) return;
  float dw[8] = {};
  for (int64_t row = blockIdx.y; row < p.tokens; row += gridDim.y) {
    const float r = p.a.rstd[row];
    float g[8], h[8];
    load_any(p.a.dy, p.a.dy_dtype, row * p.a.lddy, c, p.features, g);
    load_row8(static_cast<const T*>(p.a.total) + row * p.a.ldt, c, p.features, h);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] += g[i] * (h[i] * r);
  }
  store_row8(p.partial + static_cast<int64_t>(blockIdx.y) * p.features, c, p.features, dw);
}

// Sums the workgroups' parts of the weight's gradient: 32 columns per
// workgroup, 32 threads each of every 32nd part, joined in their order.
__global__ __launch_bounds__(1024) void k_norm_reduce(const float* __restrict__ partial, int parts, int features, float* __restrict__ dw) {
  __shared__ float sum[32][32];
  const int l = threadIdx.x & 31, q = threadIdx.x >> 5;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 32 + l;
  float s = 0.0f;
  if (c < features) {
    for (int i = q; i < parts; i += 32 * 8) {
      float v[8];  // (loaded before the first is added, the last ones too)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = partial[static_cast<int64_t>(min(i + 32 * j, parts - 1)) * features + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) s += i + 32 * j < parts ? v[j] : 0.0f;
    }
  }
  sum[q][l] = s;
  __syncthreads();
  if (q == 0 && c < features) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sum[i][l];
    dw[c] = s;
  }
}

// How a row of `chunks` pieces is held in registers.
struct Layout {
  bool wave;    // by a wave, four rows of a workgroup; else by the workgroup
  int threads;  // of a workgroup; 0: it is not, and read twice
  int pieces;   // of a thread
  int most;     // threads that the kernel is made for
};
Layout layout(int64_t chunks) {
  if (chunks <= 128) return {true, 256, chunks <= 64 ? 1 : 2, 256};
  if (chunks > 2048) return {false, 0, 0, 0};
  const int pieces = chunks <= 256 ? 1 : 2;
  const int threads = static_cast<int>((chunks + 64 * pieces - 1) / (64 * pieces) * 64);
  return {false, threads, pieces, threads <= 512 ? 512 : 1024};
}

// Rows whose codes are written together: not of few rows, which are spread over
// the CUs.
int rows_together(int64_t tokens) { return tokens >= 1024 ? 4 : 1; }

// Workgroups: enough for all CUs to be full, then each takes more rows.  (Of the
// backward pass all write partial sums of the weight's gradient, which are read
// again.)
int norm_groups(int64_t rows, const Layout& l, int together, bool bwd) {
  const int64_t per = (l.wave ? 4 : 1) * together, n = (rows + per - 1) / per;
  return static_cast<int>(std::min<int64_t>(n, bwd || l.most == 1024 ? 512 : 2048));
}

// go(whether a wave has a row, threads, pieces) as compile-time constants
template <class F>
void by_layout(const Layout& l, F&& go) {
  auto with = [&](auto wave, auto most) {
    if (l.pieces == 1) go(wave, most, std::integral_constant<int, 1>{});
    else go(wave, most, std::integral_constant<int, 2>{});
  };
  if (l.wave) with(std::true_type{}, std::integral_constant<int, 256>{});
  else if (l.most == 512) with(std::false_type{}, std::integral_constant<int, 512>{});
  else go(std::false_type{}, std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <class F>
void by_type(mx_dtype t, F&& go) {
  if (t == MX_BF16) go(bf16_t{});
  else if (t == MX_F16) go(f16_t{});
  else go(float{});
}

// Workgroups of the backward pass, whose partial sums the workspace holds.
int bwd_groups(const mx_norm_desc& d) { return norm_groups(d.tokens, layout((static_cast<int64_t>(d.features) + 7) / 8), 1, true); }

}  // namespace

hipError_t launch_norm_fwd(const mx_norm_desc& d, const NormFwd& a, hipStream_t s) {
  FwdParams p{};
  p.a = a;
  p.tokens = d.tokens;
  p.features = d.features;
  p.eps = d.eps;
  p.padded_rows = static_cast<int>(pad128(d.tokens));
  p.kt = pad128(d.features) / kTileC;
  const bool codes = a.codes != nullptr;
  p.chunks = static_cast<int>(codes ? pad128(d.features) / 8 : (static_cast<int64_t>(d.features) + 7) / 8);
  const int64_t rows = codes ? p.padded_rows : p.tokens;
  if (rows == 0) return hipSuccess;
  const Layout l = layout(p.chunks);
  by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (l.threads == 0) {
      auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(norm_groups(rows, l, 1, false)), dim3(1024), 0, s, p); };
      codes ? go(k_norm_fwd_long<T, true>) : go(k_norm_fwd_long<T, false>);
    } else by_layout(l, [&](auto wave, auto most, auto pieces) {
      constexpr bool W = decltype(wave)::value;
      constexpr int M = decltype(most)::value, C = decltype(pieces)::value;
      auto go = [&](auto kern, int together) {
        const size_t lds = together > 1 ? static_cast<size_t>(l.threads / 64 * C * 512 * together) : 0;
        hipLaunchKernelGGL(kern, dim3(norm_groups(rows, l, together, false)), dim3(l.threads), lds, s, p);
      };
      if (!codes) go(k_norm_fwd<T, W, M, C, false, 1>, 1);
      else if (rows_together(d.tokens) == 4) go(k_norm_fwd<T, W, M, C, true, 4>, 4);
      else go(k_norm_fwd<T, W, M, C, true, 1>, 1);
    });
  });
  return hipGetLastError();
}

size_t norm_workspace(const mx_norm_desc& d) {
  return d.tokens == 0 ? 0 : sizeof(float) * static_cast<size_t>(bwd_groups(d)) * static_cast<size_t>(d.features);
}

hipError_t launch_norm_bwd(const mx_norm_desc& d, const NormBwd& a, void* workspace, hipStream_t s) {
  BwdParams p{};
  p.a = a;
  p.tokens = d.tokens;
  p.features = d.features;
  p.partial = a.dweight && d.tokens > 0 ? static_cast<float*>(workspace) : nullptr;
  const int64_t chunks = (static_cast<int64_t>(d.features) + 7) / 8;
  const Layout l = layout(chunks);
  const int groups = bwd_groups(d);
  if (d.tokens > 0) by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (l.threads == 0) {
      // (first, since dx may be in dy's place)
      if (p.partial) hipLaunchKernelGGL(k_norm_dweight<T>, dim3(static_cast<unsigned>((chunks + 255) / 256), groups), dim3(256), 0, s, p);
      if (a.dx) hipLaunchKernelGGL(k_norm_bwd_long<T>, dim3(groups), dim3(1024), 0, s, p);
    } else by_layout(l, [&](auto wave, auto most, auto pieces) {
      constexpr bool W = decltype(wave)::value;
      constexpr int M = decltype(most)::value, C = decltype(pieces)::value;
      auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(groups), dim3(l.threads), 0, s, p); };
      a.dy_dtype == a.dtype ? go(k_norm_bwd<T, true, W, M, C>) : go(k_norm_bwd<T, false, W, M, C>);
    });
  });
  if (a.dweight)
    hipLaunchKernelGGL(k_norm_reduce, dim3((d.features + 31u) / 32), dim3(1024), 0, s, p.partial, d.tokens > 0 ? groups : 0, d.features, a.dweight);
  return hipGetLastError();
}

}  // namespace mx
