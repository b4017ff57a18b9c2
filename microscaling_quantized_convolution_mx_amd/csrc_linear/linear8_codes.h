// Device code that turns elements into E4M3 codes and back, shared by the
// quantizer, the norm and the fused serving kernel of the layers in 8 bits.
#pragma once

#include "linear8.h"
#include "linear_codes.h"

namespace mx {

// E8M0 code of a block from the sign-cleared bits of its maximum: the smallest
// e >= -127 with amax <= 448 * 2^e = 1.75 * 2^(e + 8), plus 127.  The addition
// carries into the exponent exactly where the significand is over 1.75.
__device__ __forceinline__ uint32_t block8_code(uint32_t amax) {
  if (amax >= NONFINITE_BITS) return 0xFFu;
  return static_cast<uint32_t>(max(static_cast<int>((amax + 0x1FFFFFu) >> 23) - 8, 0));
}

// What a block's elements are multiplied with: 2^-e, a normal fp32 for the
// codes 0..247 of finite blocks.
__device__ __forceinline__ float block8_inverse(uint32_t code) { return __uint_as_float((254u - code) << 23); }

// 4 elements as codes of the block whose scale code is `code`.  The product
// with a power of two is exact (or, below E4M3's range, rounds to zero all the
// same); the hardware conversion rounds to nearest even.
__device__ __forceinline__ uint32_t encode8x4(float a, float b, float c, float d, float inv) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
  return static_cast<uint32_t>(w);
}
__device__ __forceinline__ uint2 encode8x8(const float* x, uint32_t code) {
  if (code == 0xFFu) return make_uint2(0, 0);
  const float inv = block8_inverse(code);
  return make_uint2(encode8x4(x[0], x[1], x[2], x[3], inv), encode8x4(x[4], x[5], x[6], x[7], inv));
}

// 8 codes as bf16 values, which hold every E4M3 value times every scale exactly
// (a result below 2^-126 is a bf16 subnormal).  The conversion takes the
// scale's exponent field, which is its E8M0 code: 0 stands for 2^-127, 0xFF for
// NaN.
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
// An operand's 32 codes of a lane for the exact product: 4 steps of the bf16
// MFMA.  `scales`: the dword of four stripes' scales, of which `byte` is meant.
struct Wide { bf16x8 k[4]; };
__device__ __forceinline__ Wide widen(i32x8 v, uint32_t scales, int byte) {
  const float s = __uint_as_float((scales >> (8 * byte) & 0xFFu) << 23);
  return {{widen8(v[0], v[1], s), widen8(v[2], v[3], s), widen8(v[4], v[5], s), widen8(v[6], v[7], s)}};
}

// 2^(code - 127): 2^-127 is an fp32 subnormal, 0xFF is NaN
__device__ __forceinline__ float scale_value8(uint32_t code) {
  return code == 0xFFu ? __uint_as_float(0x7FC00000u) : (code == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(code << 23));
}

__device__ __forceinline__ uint32_t amax8(const float* x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// The maximum over a row of 16 lanes, in each of them: pairs, fours, eights by
// mirrored halves, all.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xF, 0xF, true)));
}
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = dpp_max<0xB1>(v);
  v = dpp_max<0x4E>(v);
  v = dpp_max<0x141>(v);
  return dpp_max<0x140>(v);
}

// 8 consecutive elements as they are in memory.  Loading them apart from their
// conversion keeps the loads of many pieces on their way together: a
// conversion next to its load, in the branch for the row's end, would wait for
// that load before the next one is issued.
template <class T>
struct Raw8 { i32x4 v[sizeof(T) / 2]; };

// ... of a row from column c on; zeros past the row's end.
template <class T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* row, int64_t c, int64_t cols) {
  Raw8<T> r{};
  if (c + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.v[i] = load16(reinterpret_cast<const uint8_t*>(row + c) + 16 * i);
  } else if (c < cols) {
    T e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = c + i < cols ? row[c + i] : T{};
    __builtin_memcpy(&r, e, sizeof(r));
  }
  return r;
}
template <class T>
__device__ __forceinline__ void unpack8(const Raw8<T>& r, float* x) {
  T e[8];
  __builtin_memcpy(e, &r, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = to_f32(e[i]);
}
template <class T>
__device__ __forceinline__ Raw8<T> pack8(const float* x) {
  T e[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) e[i] = from_f32<T>(x[i]);
  Raw8<T> r;
  __builtin_memcpy(&r, e, sizeof(r));
  return r;
}
template <class T>
__device__ __forceinline__ void load_row8(const T* row, int64_t c, int64_t cols, float* x) { unpack8(load_raw8(row, c, cols), x); }

// ... to column c on of a row of `cols`.  STREAM: past the caches.
template <bool STREAM = false, class T>
__device__ __forceinline__ void store_raw8(T* row, int64_t c, int64_t cols, const Raw8<T>& r) {
  if (c + 8 <= cols) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
      uint8_t* at = reinterpret_cast<uint8_t*>(row + c) + 16 * i;
      if constexpr (STREAM) stream16(at, r.v[i]);
      else store16(at, r.v[i]);
    }
    return;
  }
  T e[8];
  __builtin_memcpy(e, &r, sizeof(e));
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < cols) row[c + i] = e[i];
}
template <bool STREAM = false, class T>
__device__ __forceinline__ void store_row8(T* row, int64_t c, int64_t cols, const float* x) { store_raw8<STREAM>(row, c, cols, pack8<T>(x)); }

}  // namespace mx
