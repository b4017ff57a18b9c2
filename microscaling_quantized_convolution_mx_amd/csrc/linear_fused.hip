// Serving form of the microscaled linear layers for few tokens: one launch
// quantizes the tokens (1x32 blocks) and multiplies them by the row form of
// the weight,  y[t][i] = sum_c xq[t][c] w[i][c].
//
// Bound by the weight's bytes (17/32 of a byte per element), or by the launch
// where there are few of them.  A workgroup takes 32 output features, one
// stripe of W, which is contiguous in memory: its waves take the stripe's
// tiles in turn, straight from memory into the MFMA's operand registers, and
// their sums are joined in LDS.  Meanwhile the tokens, 32 at a time at most,
// are quantized into LDS in the operand's order; every workgroup does that
// for itself, which is cheaper than a launch of its own as long as the
// tokens are few.
#include "linear.h"
#include "linear_codes.h"

namespace mx {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;
constexpr int kAhead = 8;                    // weight tiles of a wave in flight
constexpr int kMaxTokens = 32;               // per pass
constexpr size_t kTokenLds = size_t{64} << 10;  // for the pass' codes and scales
constexpr int kSumStride = 33;               // words per token of a wave's sums: no bank conflicts

struct FusedParams {
  const uint8_t *w, *ws;
  int64_t kt;              // column tiles of a stripe
  const void* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int tokens, n, k;
  int stripes;             // of one expert's matrix that hold outputs
  int mat_stripes;         // of one expert's matrix
  const int32_t* offsets;
  int experts;
  int per_pass;            // tokens of a pass, kMaxTokens at most
  int units;               // workgroups with work
  int per_xcd;
};

template <class TX, class TY, bool VEC>
__global__ __launch_bounds__(kThreads) void k_lin_fused(const FusedParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // blocks go to the 8 XCDs in turn: XCD x takes the x-th part of the stripes,
  // so that the 4 stripes that share scale words share an L2
  const int u = static_cast<int>(blockIdx.x & 7) * p.per_xcd + static_cast<int>(blockIdx.x >> 3);
  if (static_cast<int>(blockIdx.x >> 3) >= p.per_xcd || u >= p.units) return;
  const int e = u / p.stripes, st = u - e * p.stripes;
  int len = p.tokens;
  int64_t row0 = 0;
  if (p.experts > 0) {
    Segment s;
    find_segment(p.offsets, p.experts, p.tokens, e, 0, s);
    len = s.len;
    row0 = s.row0;
  }
  if (len == 0) return;
  const int kt = static_cast<int>(p.kt);
  const int64_t stripe = static_cast<int64_t>(e) * p.mat_stripes + st;
  const uint4* wsrc = reinterpret_cast<const uint4*>(p.w + stripe * p.kt * kTileBytes) + lane;
  const uint8_t* ssrc = p.ws + (stripe / 4) * p.kt * kScaleBytes + lane * 4 + (stripe & 3);
  const int half = lane >> 5, l32 = lane & 31;

  for (int t0 = 0; t0 < len; t0 += p.per_pass) {
    const int nt = min(p.per_pass, len - t0);
    // the wave's first tiles
    uint4 w[kAhead];
    uint32_t sc[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int t = min(wave + i * kWaves, kt - 1);
      w[i] = wsrc[static_cast<int64_t>(t) * 64];
      sc[i] = ssrc[static_cast<int64_t>(t) * kScaleBytes];
    }
    // quantize: a thread takes a token's 32 columns at a time; block b of
    // token r has its codes at (b * nt + r) * 16, all scales follow
    const int nb = kt * 2;
    uint8_t* lsc = lds + static_cast<size_t>(nb) * nt * 16;
    for (int i = tid; i < nb * nt; i += kThreads) {
      const int r = i / nb, b = i - r * nb;
      const TX* src = static_cast<const TX*>(p.x) + (row0 + t0 + r) * p.ldx;
      float v[32];
      load32<TX, VEC>(src, static_cast<int64_t>(b) * 32, p.k, true, v);
      const uint32_t code = block_code(amax32(v));
      reinterpret_cast<uint4*>(lds)[b * nt + r] = encode32<false>(v, code, 0, 0);
      lsc[b * nt + r] = static_cast<uint8_t>(code);
    }
    __syncthreads();
    f32x16 acc;
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[v] = 0.0f;
    // lanes past the pass' tokens repeat the last one: their sums are not used
    const int r = min(l32, nt - 1);
    for (int base = wave; base < kt; base += kWaves * kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int t = base + i * kWaves;
        if (t < kt) {
          const int b = (2 * t + half) * nt + r;
          const uint4 x = reinterpret_cast<const uint4*>(lds)[b];
          const i32x8 fa{static_cast<int>(w[i].x), static_cast<int>(w[i].y), static_cast<int>(w[i].z), static_cast<int>(w[i].w), 0, 0, 0, 0};
          const i32x8 fb{static_cast<int>(x.x), static_cast<int>(x.y), static_cast<int>(x.z), static_cast<int>(x.w), 0, 0, 0, 0};
          acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fa, fb, acc, 4, 4, 0, static_cast<int>(sc[i]), 0, static_cast<int>(lsc[b]));
        }
        const int tn = min(t + kWaves * kAhead, kt - 1);
        w[i] = wsrc[static_cast<int64_t>(tn) * 64];
        sc[i] = ssrc[static_cast<int64_t>(tn) * kScaleBytes];
      }
    }
    __syncthreads();
    // join the waves' sums in their order: lane holds token l32, features
    // 8(v/4) + 4 half + v%4
    float* sums = reinterpret_cast<float*>(lds);
    if (l32 < nt) {
      float* d = sums + (wave * nt + l32) * kSumStride + 4 * half;
#pragma unroll
      for (int v = 0; v < 16; ++v) d[8 * (v / 4) + v % 4] = acc[v];
    }
    __syncthreads();
    for (int i = tid; i < nt * 32; i += kThreads) {
      const int t = i >> 5, f = i & 31;
      float s = 0.0f;
#pragma unroll
      for (int q = 0; q < kWaves; ++q) s += sums[(q * nt + t) * kSumStride + f];
      const int col = st * 32 + f;
      if (col < p.n) static_cast<TY*>(p.y)[(row0 + t0 + t) * p.ldy + col] = from_f32<TY>(s);
    }
    __syncthreads();
  }
}

// LDS of a pass: codes and scales of the tokens, then the waves' sums in
// their place.
size_t fused_lds(int64_t kp, int tokens) {
  const size_t x = static_cast<size_t>(kp / 32) * tokens * 17, s = static_cast<size_t>(kWaves) * tokens * kSumStride * 4;
  return ((x > s ? x : s) + 15) / 16 * 16;
}

int tokens_per_pass(const LinGeom& g) {
  int t = kMaxTokens;
  while (t > 0 && fused_lds(g.kp, t) > kTokenLds) --t;
  return t;
}

}  // namespace

bool lin_fused(const LinGeom& g) {
  const int t = tokens_per_pass(g);
  if (g.e == 0) return g.m <= t;
  return t > 0 && g.m <= 8ll * g.e;
}

hipError_t launch_lin_fused(const LinGeom& g, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                            void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s) {
  FusedParams p{};
  p.w = static_cast<const uint8_t*>(wq->rows);
  p.ws = wq->row_scales;
  p.kt = g.kp / kTileC;
  p.x = x;
  p.ldx = ldx;
  p.y = y;
  p.ldy = ldy;
  p.tokens = static_cast<int>(g.m);
  p.n = static_cast<int>(g.n);
  p.k = static_cast<int>(g.k);
  p.stripes = static_cast<int>((g.n + kTileR - 1) / kTileR);
  p.mat_stripes = static_cast<int>(g.np / kTileR);
  p.offsets = offsets;
  p.experts = g.e;
  const int most = tokens_per_pass(g);
  p.per_pass = g.m < most ? static_cast<int>(g.m) : most;
  p.units = p.stripes * g.ew;
  p.per_xcd = ((p.units + 7) / 8 + 3) / 4 * 4;
  const size_t lds = fused_lds(g.kp, p.per_pass);
  const unsigned grid = static_cast<unsigned>(p.per_xcd) * 8;
  auto go = [&](auto tx, auto ty) {
    using TX = decltype(tx);
    using TY = decltype(ty);
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && ldx * static_cast<int64_t>(sizeof(TX)) % 16 == 0;
    if (vec) hipLaunchKernelGGL((k_lin_fused<TX, TY, true>), dim3(grid), dim3(kThreads), lds, s, p);
    else hipLaunchKernelGGL((k_lin_fused<TX, TY, false>), dim3(grid), dim3(kThreads), lds, s, p);
  };
  auto with_x = [&](auto tx) {
    switch (y_dtype) {
      case MX_BF16: go(tx, bf16_t{}); break;
      case MX_F16: go(tx, f16_t{}); break;
      default: go(tx, float{}); break;
    }
  };
  switch (x_dtype) {
    case MX_BF16: with_x(bf16_t{}); break;
    case MX_F16: with_x(f16_t{}); break;
    default: with_x(float{}); break;
  }
  return hipGetLastError();
}

}  // namespace mx
