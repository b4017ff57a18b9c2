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
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <> __device__ __forceinline__ void load8<bf16_t>(const bf16_t* p, float* x) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
template <> __device__ __forceinline__ void load8<f16_t>(const f16_t* p, float* x) {
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  const h8 a = *reinterpret_cast<const h8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = static_cast<float>(a[i]);
}

// 32 consecutive elements of a row from column c on; zeros past the row's end.
// vec: the row starts at a multiple of 16 bytes.
template <class T>
__device__ __forceinline__ void load32(const T* row, int64_t c, int64_t cols, bool vec, float* x) {
  if (vec && c + 32 <= cols) {
#pragma unroll
    for (int i = 0; i < 4; ++i) load8(row + c + 8 * i, x + 8 * i);
    return;
  }
  const T* p = row + c;
  if (c + 32 <= cols) {
    T v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = p[i];
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = to_f32(v[i]);
    return;
  }
  // the row's end: its last element where there is none, so that no load waits for a comparison
  const int n = c < cols ? static_cast<int>(cols - c) : 0;
  if (n == 0) p = row;
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

// 32 elements as codes of the block whose scale code is `code`.
// idx: index of the first one, for the stochastic rounding.
template <bool SR>
__device__ __forceinline__ uint4 encode32(const float* x, uint32_t code, uint64_t seed, uint64_t idx) {
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
    uint32_t ub[32];
    if ((idx & 1) == 0) {
      uint64_t gk = kGolden64 * ((idx >> 1) + 1ull);
#pragma unroll
      for (int j = 0; j < 16; ++j, gk += kGolden64) sr_ubar_pair(seed, gk, ub[2 * j], ub[2 * j + 1]);
    } else {
#pragma unroll
      for (int j = 0; j < 32; ++j) ub[j] = sr_ubar(seed, idx + j);
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const uint32_t c = sr_code<F>(fabsf(x[j]) * inv, ub[j]) | ((__float_as_uint(x[j]) >> 31) << F::SIGN);
      w[j >> 3] |= c << (4 * (j & 7));
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace mx
