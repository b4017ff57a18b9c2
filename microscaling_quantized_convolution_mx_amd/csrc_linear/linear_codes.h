// Device code that turns 32 consecutive elements into one block row of E2M1
// codes, shared by the quantizer and the fused serving kernel of the
// microscaled linear layers.
#pragma once

#include "linear.h"
#include "mx_formats.h"

namespace mx {

constexpr int kEmax = 2;  // exponent of the largest E2M1 value, 6 = 1.5 * 2^2

// E8M0 code of a block from the sign-cleared bits of its maximum (NaN orders
// above Inf above every finite value).
__device__ __forceinline__ uint32_t block_code(uint32_t amax) {
  if (amax >= NONFINITE_BITS) return 0xFFu;
  if (amax == 0u) return 0u;
  const int fl = amax >= 0x00800000u ? static_cast<int>(amax >> 23) - 127 : (31 - __builtin_clz(amax)) - 149;
  return static_cast<uint32_t>(max(fl - kEmax, -127) + 127);
}

// 8 consecutive elements as fp32
template <class T> __device__ __forceinline__ void load8(const T* p, float* x);
template <> __device__ __forceinline__ void load8<float>(const float* p, float* x) {
  const i32x4 a = load16(p), b = load16(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = __int_as_float(a[i]);
    x[4 + i] = __int_as_float(b[i]);
  }
}
template <> __device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float* x) {
  const i32x4 a = load16(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(static_cast<uint32_t>(a[i]) << 16);
    x[2 * i + 1] = __uint_as_float(static_cast<uint32_t>(a[i]) & 0xFFFF0000u);
  }
}
template <> __device__ __forceinline__ void load8<f16_t>(const f16_t* p, float* x) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  const h8 a = __builtin_bit_cast(h8, load16(p));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(a[i]);
}

// 32 consecutive elements of a row from column c on; zeros past the row's end.
template <class T>
__device__ __forceinline__ void load32(const T* row, int64_t c, int64_t cols, float* x) {
  if (c + 32 <= cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(row + c + 8 * i, x + 8 * i);
    return;
  }
  // the row's end: its last element where there is none, so that no load waits for a comparison
  const int n = c < cols ? static_cast<int>(cols - c) : 0;
  const T* p = n > 0 ? row + c : row;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const T v = p[max(min(i, n - 1), 0)];
    x[i] = i < n ? to_f32(v) : 0.0f;
  }
}

__device__ __forceinline__ uint32_t amax32(const float* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// Stochastic rounding of x / 2^(code - 127), below 8 in magnitude, onto E2M1
// with its sign: sr_code's rule (ub: the complemented uniform) on the bits of
// x itself.  With b the binades of the quotient above [1, 2), none below it,
// Q = |x| 2^(152 - code - b) is the quotient over the grid step times 2^24, and
// the index on the grid is (ceil(Q) + ub) >> 24, plus 2 for each binade.
__device__ __forceinline__ uint32_t sr_e2m1(float x, uint32_t code, uint32_t ub) {
  const uint32_t e = __builtin_amdgcn_ubfe(__float_as_uint(x), 23, 8);
  const uint32_t b = e > code ? e - code : 0u;
  const float q = __builtin_amdgcn_ldexpf(fabsf(x), 152 - static_cast<int>(code) - static_cast<int>(b));
  int m;  // -ceil(Q) = floor(-Q)
  asm("v_cvt_flr_i32_f32 %0, -%1" : "=v"(m) : "v"(q));
  const uint32_t c = min((b << 1) + ((ub - static_cast<uint32_t>(m)) >> 24), 7u);
  return c | (__float_as_uint(x) >> 28 & 8u);
}

// One draw serves elements 2i and 2i+1.  ODD: idx may be odd, and the row then
// begins with the second half of a draw.
template <bool ODD>
__device__ __forceinline__ void sr_codes(const float* x, uint32_t code, uint64_t seed, uint64_t idx, uint32_t* w) {
  const bool odd = ODD && (idx & 1) != 0;
  uint64_t gk = kGolden64 * ((idx >> 1) + 1ull);
  uint32_t even_u, odd_u;
  sr_ubar_pair(seed, gk, even_u, odd_u);
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    gk += kGolden64;
    uint32_t next_even = 0, next_odd = 0;
    if (j < 15 || ODD) sr_ubar_pair(seed, gk, next_even, next_odd);
    const uint32_t c0 = sr_e2m1(x[2 * j], code, odd ? odd_u : even_u), c1 = sr_e2m1(x[2 * j + 1], code, odd ? next_even : odd_u);
    w[j >> 2] |= (c0 | c1 << 4) << (8 * (j & 3));
    even_u = next_even;
    odd_u = next_odd;
  }
}

// 32 elements as codes of the block whose scale code is `code`.
// For the stochastic rounding, idx: index of the first one; odd_rows: whether
// it may be odd (the same for all lanes).
template <bool SR>
__device__ __forceinline__ uint4 encode32(const float* x, uint32_t code, uint64_t seed, uint64_t idx, bool odd_rows) {
  using F = Fmt<FMT_E2M1>;
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  if (code == 0xFFu) return make_uint4(0, 0, 0, 0);
  const float inv = __uint_as_float((254u - code) << 23);  // 2^-e, a normal fp32 for the codes 0..252 of finite blocks
  if constexpr (!SR) {
    // the hardware conversion rounds to nearest even; magnitudes are clamped
    // to the format's largest first
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __builtin_amdgcn_fmed3f(x[8 * i + j] * inv, -F::MAXV, F::MAXV);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[0], v[1], 1.0f, 0);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[2], v[3], 1.0f, 1);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[4], v[5], 1.0f, 2);
      w[i] = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w[i], v[6], v[7], 1.0f, 3);
    }
  } else {
    if (odd_rows) sr_codes<true>(x, code, seed, idx, w);
    else sr_codes<false>(x, code, seed, idx, w);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace mx
