// The root-mean-square norm with the residual's addition, and its gradients.
//
//   fwd   total = x + residual, rstd = (mean total^2 + eps)^(-1/2), y = total rstd weight
//   bwd   h = total rstd, g = dy weight,
//         dx = rstd (g - h mean(g h)) + dtotal,  dweight = sum over tokens of dy h
//
// Bound by memory traffic: everything is read and written once.  A row is held
// in the registers of one wave, of 4 or of 16 (TPR threads), CH pieces of 8
// elements each, between the sum over it and the results that need the sum.
// Workgroups take rows in turn and keep the weight, and in the backward pass
// the weight's gradient over their rows, in registers; those partial sums are
// added by a second kernel in a fixed order.  Rows too long for registers are
// read twice.
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

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), CTRL, 0xF, 0xF, true));
}
// The sum over a wave, in every lane: rows of 16 lanes, then the four rows.
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(v))));
  const int b = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

// The sum over a row's TPR threads.  `buf` is used in turn, so that one barrier
// per row is enough: a wave that writes half `turn` again has passed the
// barrier of the row between, which all have reached after reading it.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float (*buf)[TPR / 64], int turn) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[turn][wave] = v;
    __syncthreads();
    v = buf[turn][0];
#pragma unroll
    for (int w = 1; w < TPR / 64; ++w) v += buf[turn][w];
  }
  return v;
}

// 8 values as codes of the 8-bit row form: 16 lanes share a block of 128.
__device__ __forceinline__ void store_codes(const FwdParams& p, int64_t row, int64_t c, const float* y) {
  const uint32_t code = block8_code(row16_max(amax8(y)));
  const uint2 w = encode8x8(y, code);
  uint8_t* at = p.a.codes + ((row / kTileR) * p.kt + c / kTileC) * k8TileBytes + (c / 16 % 4) * 512 + (row % 32) * 16 + c % 16;
  *reinterpret_cast<uint2*>(at) = w;
  if (c % kPad == 0)
    p.a.scales[(row / kPad * (p.kt / 2) + c / kPad) * k8ScaleBytes + (row % 32) * 4 + row / 32 % 4] = static_cast<uint8_t>(code);
}

template <class T>
__device__ __forceinline__ void load_total(const FwdParams& p, int64_t row, int64_t c, float* v) {
  load_row8(static_cast<const T*>(p.a.x) + row * p.a.ldx, c, p.features, v);
  if (p.a.residual) {
    float r[8];
    load_row8(static_cast<const T*>(p.a.residual) + row * p.a.ldr, c, p.features, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = to_f32(from_f32<T>(v[i] + r[i]));
  }
}

template <class T, int TPR, int CH, bool CODES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_fwd(const FwdParams p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;  // rows of a workgroup
  __shared__ float buf[2][TPR / 64];
  const int t = threadIdx.x % TPR;
  float w[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (j * TPR + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] = 0.0f;
    if (c < p.features) load_any(p.a.weight, p.a.w_dtype, 0, c, p.features, w[j]);
  }
  const int rows = CODES ? p.padded_rows : p.tokens;
  int turn = 0;
  for (int row = blockIdx.x * RPW + threadIdx.x / TPR; row < rows; row += gridDim.x * RPW, turn ^= 1) {
    float v[CH][8];
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.0f;
      if (row < p.tokens && c < p.features) load_total<T>(p, row, c, v[j]);
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[j][i] * v[j][i];
    s = row_sum<TPR>(s, buf, turn);
    const float r = 1.0f / __builtin_sqrtf(s / static_cast<float>(p.features) + p.eps);
    if (p.a.rstd && t == 0 && row < p.tokens) p.a.rstd[row] = r;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * TPR + t) * 8;
      const bool in = row < p.tokens && c < p.features;
      if (in && p.a.total) store_row8(static_cast<T*>(p.a.total) + row * p.a.ldt, c, p.features, v[j]);
      float y[8];
      // (padding is zero also where rstd is not finite)
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = in && c + i < p.features ? v[j][i] * r * w[j][i] : 0.0f;
      if (in && p.a.y) store_any(p.a.y, p.a.y_dtype, row * p.a.ldy, c, p.features, y);
      if constexpr (CODES) {
        if (c < 8 * p.chunks) store_codes(p, row, c, y);
      }
    }
  }
}

// Rows of any length, read twice.
template <class T, bool CODES>
__global__ __launch_bounds__(1024) void k_norm_fwd_long(const FwdParams p) {
  constexpr int TPR = 1024;
  __shared__ float buf[2][TPR / 64];
  const int rows = CODES ? p.padded_rows : p.tokens;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
    float s = 0.0f;
    if (row < p.tokens) {
      for (int64_t c = 8 * threadIdx.x; c < p.features; c += 8 * TPR) {
        float v[8];
        load_total<T>(p, row, c, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i] * v[i];
      }
    }
    s = row_sum<TPR>(s, buf, turn);
    const float r = 1.0f / __builtin_sqrtf(s / static_cast<float>(p.features) + p.eps);
    if (p.a.rstd && threadIdx.x == 0 && row < p.tokens) p.a.rstd[row] = r;
    for (int64_t c = 8 * threadIdx.x; c < 8 * static_cast<int64_t>(p.chunks); c += 8 * TPR) {
      float v[8] = {}, w[8] = {}, y[8];
      const bool in = row < p.tokens && c < p.features;
      if (in) {
        load_total<T>(p, row, c, v);
        load_any(p.a.weight, p.a.w_dtype, 0, c, p.features, w);
        if (p.a.total) store_row8(static_cast<T*>(p.a.total) + row * p.a.ldt, c, p.features, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = in && c + i < p.features ? v[i] * r * w[i] : 0.0f;
      if (in && p.a.y) store_any(p.a.y, p.a.y_dtype, row * p.a.ldy, c, p.features, y);
      if constexpr (CODES) store_codes(p, row, c, y);
    }
  }
}

template <class T, int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_norm_bwd(const BwdParams p) {
  constexpr int RPW = TPR < 256 ? 256 / TPR : 1;
  __shared__ float buf[2][TPR / 64];
  const int t = threadIdx.x % TPR;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = (j * TPR + t) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[j][i] = dw[j][i] = 0.0f;
    if (c < p.features) load_any(p.a.weight, p.a.w_dtype, 0, c, p.features, w[j]);
  }
  int turn = 0;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * RPW + threadIdx.x / TPR; row < p.tokens; row += gridDim.x * RPW, turn ^= 1) {
    const float r = p.a.rstd[row];
    float g[CH][8], h[CH][8];
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * TPR + t) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) g[j][i] = h[j][i] = 0.0f;
      if (c < p.features) {
        load_any(p.a.dy, p.a.dy_dtype, row * p.a.lddy, c, p.features, g[j]);
        load_row8(static_cast<const T*>(p.a.total) + row * p.a.ldt, c, p.features, h[j]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        h[j][i] *= r;
        dw[j][i] += g[j][i] * h[j][i];
        g[j][i] *= w[j][i];
        s += g[j][i] * h[j][i];
      }
    }
    if (!p.a.dx) continue;
    const float m = row_sum<TPR>(s, buf, turn) / static_cast<float>(p.features);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int c = (j * TPR + t) * 8;
      if (c >= p.features) continue;
      float d[8] = {};
      if (p.a.dtotal) load_row8(static_cast<const T*>(p.a.dtotal) + row * p.a.lddt, c, p.features, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += r * (g[j][i] - h[j][i] * m);
      store_row8(static_cast<T*>(p.a.dx) + row * p.a.lddx, c, p.features, d);
    }
  }
  if (!p.partial) return;
  if constexpr (RPW > 1) {
    // the rows' waves in their order
    __shared__ float sum[RPW][TPR * 8 + 8];
    const int rw = threadIdx.x / TPR;
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
    const int c = (j * TPR + t) * 8;
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
      if (pass == 0) m = row_sum<TPR>(s, buf, turn) / static_cast<float>(p.features);
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

// Sums the workgroups' parts of the weight's gradient: 64 columns per
// workgroup, 16 threads each of every 16th part, joined in their order.
__global__ __launch_bounds__(1024) void k_norm_reduce(const float* __restrict__ partial, int parts, int features, float* __restrict__ dw) {
  __shared__ float sum[16][64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + l;
  float s = 0.0f;
  if (c < features) {
#pragma unroll 8
    for (int i = q; i < parts; i += 16) s += partial[static_cast<int64_t>(i) * features + c];
  }
  sum[q][l] = s;
  __syncthreads();
  if (q == 0 && c < features) {
    for (int i = 1; i < 16; ++i) s += sum[i][l];
    dw[c] = s;
  }
}

// Threads of a row of `chunks` pieces, which they hold in registers (1 or 2
// each, or 4 of 256 threads), or 0 where that is too much.
int threads_per_row(int64_t chunks) { return chunks <= 128 ? 64 : chunks <= 1024 ? 256 : chunks <= 2048 ? 1024 : 0; }
int rows_per_group(int tpr) { return tpr == 64 ? 4 : 1; }

// Workgroups: enough for all CUs to be full, then each takes more rows.
int fwd_groups(int64_t rows, int tpr) {
  const int64_t n = (rows + rows_per_group(tpr) - 1) / rows_per_group(tpr);
  return static_cast<int>(std::min<int64_t>(n, tpr == 1024 ? 512 : 2048));
}
// (of whose partial sums of the weight's gradient all are read again)
int bwd_groups(int64_t rows, int tpr) {
  const int64_t n = (rows + rows_per_group(tpr) - 1) / rows_per_group(tpr);
  return static_cast<int>(std::min<int64_t>(n, 512));
}

// go(threads per row, pieces of a thread) as compile-time constants
template <class F>
void by_size(int64_t chunks, F&& go) {
  const int tpr = threads_per_row(chunks);
  auto with = [&](auto t) {
    const int64_t n = (chunks + decltype(t)::value - 1) / decltype(t)::value;
    if (n <= 1) go(t, std::integral_constant<int, 1>{});
    else if (n <= 2) go(t, std::integral_constant<int, 2>{});
    else if constexpr (decltype(t)::value == 256) go(t, std::integral_constant<int, 4>{});
  };
  if (tpr == 64) with(std::integral_constant<int, 64>{});
  else if (tpr == 256) with(std::integral_constant<int, 256>{});
  else with(std::integral_constant<int, 1024>{});
}

template <class F>
void by_type(mx_dtype t, F&& go) {
  if (t == MX_BF16) go(bf16_t{});
  else if (t == MX_F16) go(f16_t{});
  else go(float{});
}

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
  const int tpr = threads_per_row(p.chunks);
  by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern, int threads) { hipLaunchKernelGGL(kern, dim3(fwd_groups(rows, tpr ? tpr : 1024)), dim3(threads), 0, s, p); };
    if (tpr == 0) codes ? go(k_norm_fwd_long<T, true>, 1024) : go(k_norm_fwd_long<T, false>, 1024);
    else by_size(p.chunks, [&](auto n, auto ch) {
      constexpr int N = decltype(n)::value, C = decltype(ch)::value;
      codes ? go(k_norm_fwd<T, N, C, true>, N < 256 ? 256 : N) : go(k_norm_fwd<T, N, C, false>, N < 256 ? 256 : N);
    });
  });
  return hipGetLastError();
}

size_t norm_workspace(const mx_norm_desc& d) {
  const int tpr = threads_per_row((static_cast<int64_t>(d.features) + 7) / 8);
  return d.tokens == 0 ? 0 : sizeof(float) * static_cast<size_t>(bwd_groups(d.tokens, tpr ? tpr : 1024)) * static_cast<size_t>(d.features);
}

hipError_t launch_norm_bwd(const mx_norm_desc& d, const NormBwd& a, void* workspace, hipStream_t s) {
  BwdParams p{};
  p.a = a;
  p.tokens = d.tokens;
  p.features = d.features;
  p.partial = a.dweight && d.tokens > 0 ? static_cast<float*>(workspace) : nullptr;
  const int64_t chunks = (static_cast<int64_t>(d.features) + 7) / 8;
  const int tpr = threads_per_row(chunks), groups = bwd_groups(d.tokens, tpr ? tpr : 1024);
  if (d.tokens > 0) by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (tpr == 0) {
      // (first, since dx may be in dy's place)
      if (p.partial) hipLaunchKernelGGL(k_norm_dweight<T>, dim3(static_cast<unsigned>((chunks + 255) / 256), groups), dim3(256), 0, s, p);
      if (a.dx) hipLaunchKernelGGL(k_norm_bwd_long<T>, dim3(groups), dim3(1024), 0, s, p);
    } else by_size(chunks, [&](auto n, auto ch) {
      constexpr int N = decltype(n)::value, C = decltype(ch)::value;
      hipLaunchKernelGGL((k_norm_bwd<T, N, C>), dim3(groups), dim3(N < 256 ? 256 : N), 0, s, p);
    });
  });
  if (a.dweight)
    hipLaunchKernelGGL(k_norm_reduce, dim3((d.features + 63u) / 64), dim3(1024), 0, s, p.partial, d.tokens > 0 ? groups : 0, d.features, a.dweight);
  return hipGetLastError();
}

}  // namespace mx
