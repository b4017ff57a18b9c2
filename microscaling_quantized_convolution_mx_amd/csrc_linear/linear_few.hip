// Products of the microscaled linear layers with few tokens:
//   y[t][i] = sum_c x[t][c] w[i][c]
// with the lines of w in a form whose columns are c (fwd: W's row form, dgrad:
// W's column form), and x either in its row form or, for serving, unquantized
// and quantized here (1x32 blocks), in one launch.
//
// Bound by w's bytes (17/32 of a byte per element), or by the launch where
// there are few of them.  A workgroup takes SN stripes of 32 lines of w; its
// waves take the stripes' column tiles in turn, straight from memory into the
// MFMA's operand registers, several of them on their way, and their sums are
// joined in LDS.  Its tokens, 32 at most, come from memory (L2) in the same way,
// or quantized into LDS by the whole workgroup while the first tiles of w are
// on their way.  Every workgroup quantizes for itself, which is cheaper
// than a launch of its own while the tokens are few (lin_fused()).
//
// Measured in graphs of such calls, which leave the weight in the last-level
// cache: 1x16384x8192 13.2 us (5.4 TB/s of weight), 1x4096x4096 3.5 or, quantizing,
// 3.9, 256 tokens of 64 experts, 2048x2048, 25 (5.8 TB/s).  Eight tiles on their
// way for each wave are enough: with 12, in more registers, 1x4096x4096 takes 7.5
// us and 256 tokens of 64 experts 42.
#include <type_traits>

#include "linear_codes.h"
#include "linear_few.h"

namespace mx {
namespace {

constexpr size_t kTokenLds = size_t{48} << 10;  // for a pass' codes and scales: three workgroups share a CU where there are that many

// TX: type of the unquantized tokens, void for codes.
template <class TX, int SN>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void k_lin_few(const FewParams p) {
  constexpr bool kFused = !std::is_void_v<TX>;
  constexpr int kAhead = 8 / SN;  // column tiles of a wave on their way
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
  FewWork w0;
  if (!find_pass(p, SN, kFused ? p.per_pass : 32, w0)) return;
  const int st = w0.st, e = w0.e, nt = w0.nt;
  const int64_t row0 = w0.row0, prow = w0.prow;
  const int kt = static_cast<int>(p.kt);
  const int64_t stripe = static_cast<int64_t>(e) * p.mat_stripes + st;
  const uint8_t* wsrc = p.w + stripe * p.kt * kTileBytes;
  const uint8_t* ssrc = p.ws + (stripe / 4) * p.kt * kScaleBytes;
  const int sshift = 8 * static_cast<int>(stripe & 3);  // SN stripes lie in one group of four
  const int half = lane >> 5, l32 = lane & 31;
  i32x4 w[kAhead][SN], xv[kAhead];
  int ws[kAhead], xs[kAhead];
  // the wave's column tiles; a fetch past them takes the last one again
  const int chunk = (kt + waves - 1) / waves, begin = min(wave * chunk, kt), end = min(begin + chunk, kt);
  auto fetch = [&](int q, int t) {
    t = max(min(t, end - 1), 0);
#pragma unroll
    for (int j = 0; j < SN; ++j) w[q][j] = lane_load<i32x4>(wsrc + (j * p.kt + t) * kTileBytes, lane);
    ws[q] = lane_load<int>(ssrc + static_cast<int64_t>(t) * kScaleBytes, lane);
    if constexpr (!kFused) {
      xv[q] = lane_load<i32x4>(static_cast<const uint8_t*>(p.x) + ((prow / kTileR) * p.kt + t) * kTileBytes, lane);
      xs[q] = lane_load<int>(p.xs + ((prow / kPad) * p.kt + t) * kScaleBytes, lane);
    }
  };
#pragma unroll
  for (int q = 0; q < kAhead; ++q) fetch(q, begin + q);

  const uint8_t* lsc = nullptr;
  if constexpr (kFused) {
    // a thread takes a token's 32 columns at a time; block b of token r has
    // its codes at (b * nt + r) * 16, all scales follow
    const int nb = kt * 2;
    uint8_t* sc = lds + static_cast<size_t>(nb) * nt * 16;
    lsc = sc;
    for (int b = tid; b < nb * nt; b += threads) {
      const int r = b / nb, c = b - r * nb;
      const TX* src = static_cast<const TX*>(p.x) + (row0 + r) * p.ldx;
      float v[32];
      load32<TX>(src, static_cast<int64_t>(c) * 32, p.k, v);
      const uint32_t code = block_code(amax32(v));
      reinterpret_cast<uint4*>(lds)[c * nt + r] = encode32<false>(v, code, 0, 0, false);
      sc[c * nt + r] = static_cast<uint8_t>(code);
    }
    __syncthreads();
  }
  f32x16 acc[SN];
#pragma unroll
  for (int j = 0; j < SN; ++j)
#pragma unroll
    for (int v = 0; v < 16; ++v) acc[j][v] = 0.0f;
  // lanes past the pass' tokens repeat the last one: their sums are not used
  const int r = min(l32, nt - 1);
  const int xshift = kFused ? 0 : 8 * static_cast<int>(prow / kTileR & 3);
  auto multiply = [&](int q, int t, bool in) {
    int xsc;
    if constexpr (kFused) {
      const int b = (2 * t + half) * nt + r;
      xv[q] = reinterpret_cast<const i32x4*>(lds)[b];
      xsc = lsc[b];
    } else {
      xsc = static_cast<int>(static_cast<uint32_t>(xs[q]) >> xshift);
    }
    const int wsc = static_cast<int>(static_cast<uint32_t>(ws[q]) >> sshift);
    const int m = in ? -1 : 0;
    auto mul = [&](auto jc) {
      constexpr int J = decltype(jc)::value;
      if constexpr (J < SN)
        acc[J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(w[q][J]), operand(xv[q] & m), acc[J], 4, 4, J, wsc, 0, xsc);
    };
    mul(std::integral_constant<int, 0>{});
    mul(std::integral_constant<int, 1>{});
    mul(std::integral_constant<int, 2>{});
    mul(std::integral_constant<int, 3>{});
  };
  int t = begin;
  for (; t + kAhead < end; t += kAhead) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      multiply(q, t + q, true);
      fetch(q, t + kAhead + q);
    }
  }
  // the last ones, some of them repeated with x as zeros.  (A scale that is
  // NaN has already made those sums NaN.)
  if (t < end) {
#pragma unroll
    for (int q = 0; q < kAhead; ++q) multiply(q, min(t + q, end - 1), t + q < end);
  }
  join_sums<SN>(p, acc, reinterpret_cast<float*>(lds), nt, row0, st);
}

// LDS of a pass: codes and scales of the tokens, and then the waves' sums in
// their place.
size_t fused_lds(int64_t kt, int waves, int tokens) {
  const size_t x = static_cast<size_t>(2 * kt) * tokens * 17, s = static_cast<size_t>(waves) * tokens * kSumStride * 4;
  return ((x > s ? x : s) + 15) / 16 * 16;
}

int tokens_per_pass(int64_t kt) {
  int t = 32;
  while (t > 0 && fused_lds(kt, waves_of(kt), t) > kTokenLds) --t;
  return t;
}

FewParams make_few(const LinGeom& g, bool dgrad, bool fused, const mx_linear_qtensor* wq, void* y, mx_dtype y_dtype, int64_t ldy,
                   const int32_t* offsets, int& sn) {
  FewParams p{};
  int64_t lines, cols;
  const mx_form form = dgrad ? MX_FORM_COLS : MX_FORM_ROWS;
  form_dims(g, MX_ROLE_WEIGHT, form, lines, cols);
  p.w = static_cast<const uint8_t*>(dgrad ? wq->cols : wq->rows);
  p.ws = dgrad ? wq->col_scales : wq->row_scales;
  p.kt = cols / kTileC;
  p.mat_stripes = lines / kTileR;
  p.y = y;
  p.ldy = ldy;
  p.y_dtype = y_dtype;
  p.tokens = static_cast<int>(g.m);
  p.n = static_cast<int>(dgrad ? g.k : g.n);
  p.k = static_cast<int>(dgrad ? g.n : g.k);
  p.offsets = offsets;
  p.experts = g.e;
  const int64_t stripes = (p.n + kTileR - 1) / kTileR;
  sn = stripes_per_group(stripes * g.ew);
  const int64_t most = fused ? tokens_per_pass(p.kt) : 32;
  p.per_pass = static_cast<int>(g.m < most ? g.m : most);
  // an expert with tokens has one pass, and one more for every per_pass tokens past its first
  const int64_t used = g.m < g.ew ? g.m : g.ew;
  p.passes = g.e > 0 ? static_cast<int>(used + (g.m - used) / p.per_pass) : 1;
  // An XCD takes an eighth of each pass' stripes: the same work for all of them,
  // and consecutive memory.  Of 64 passes and more it takes whole ones, longer
  // pieces of memory, one in eight (4 tokens each of 64 experts, 2048x2048, 25 us
  // and 30 in eighths; 16 each of 1024 experts, 512x512, 39 and 68).  Whole groups
  // of four stripes, which share scale words.
  p.whole = p.passes >= 64 ? 1 : 0;
  const int64_t quads = (stripes + 3) / 4;
  p.part = static_cast<int>(p.whole ? quads : (quads + 7) / 8) * (4 / sn);
  return p;
}

LinVariant variant(const FewParams& p, int sn, bool fused) {
  const int64_t rounds = p.whole ? (p.passes + 7) / 8 : p.passes;
  return {fused ? 2 : 1, sn, 1, 64 * waves_of(p.kt), rounds * 8 * p.part};
}

}  // namespace

LinVariant lin_few_variant(const LinGeom& g, bool dgrad, bool fused) {
  const mx_linear_qtensor none{};
  int sn;
  const FewParams p = make_few(g, dgrad, fused, &none, nullptr, MX_F32, 0, nullptr, sn);
  return variant(p, sn, fused);
}

// Quantizing M tokens in every group of an expert's stripes takes about
// M * columns * groups / 2e12 s over the whole GPU, much of it while the weight
// is on its way; a launch of its own takes about 4 us and an L2 read of the
// codes.  (In graphs: 256 tokens of 64 experts, 2048x2048, 8.4M elements, 24 us here
// and 31 in two launches; 16x8192x2048, 8.4M, 5.7 and 6.5; 32x8192x2048, 16.8M, 7.9
// and 6.9.)
bool lin_fused(const LinGeom& g) {
  const int64_t kt = g.kp / kTileC, stripes = (g.n + kTileR - 1) / kTileR;
  const int t = tokens_per_pass(kt), sn = stripes_per_group(stripes * g.ew);
  const int64_t groups = (stripes + sn - 1) / sn;
  if (t == 0 || g.m * g.kp * groups >= (int64_t{1} << 24)) return false;
  return g.e == 0 ? g.m <= t : lin_few(g);
}

// One pass of tokens, or experts with few tokens each.  (32x4096x4096 takes 4.0
// us here and 7.7 in 64x64 tiles, 32x1024x1024 4.0 and 3.9; 16 tokens each of 64
// experts, 2048x2048, 25.8 and 26.2, of 1024 experts, 512x512, 39 and 126.  Where
// all of these tokens choose one expert, 12 and 8, and 30 and 57.)
bool lin_few(const LinGeom& g) { return g.e == 0 ? g.m <= 32 : g.m <= 16 * static_cast<int64_t>(g.e); }

hipError_t launch_lin_fused(const LinGeom& g, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
                            void* y, mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s) {
  int sn;
  FewParams p = make_few(g, false, true, wq, y, y_dtype, ldy, offsets, sn);
  p.x = x;
  p.ldx = ldx;
  const size_t lds = fused_lds(p.kt, waves_of(p.kt), p.per_pass);
  const LinVariant v = variant(p, sn, true);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(v.workgroups)), dim3(v.threads), lds, s, p); };
  auto with = [&](auto t) {
    using T = decltype(t);
    sn == 4 ? go(k_lin_few<T, 4>) : sn == 2 ? go(k_lin_few<T, 2>) : go(k_lin_few<T, 1>);
  };
  switch (x_dtype) {
    case MX_BF16: with(bf16_t{}); break;
    case MX_F16: with(f16_t{}); break;
    default: with(float{}); break;
  }
  return hipGetLastError();
}

hipError_t launch_lin_few(const LinGeom& g, bool dgrad, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                          mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s) {
  int sn;
  FewParams p = make_few(g, dgrad, false, wq, y, y_dtype, ldy, offsets, sn);
  p.x = xq->rows;
  p.xs = xq->row_scales;
  const size_t lds = static_cast<size_t>(waves_of(p.kt)) * p.per_pass * kSumStride * 4;
  const LinVariant v = variant(p, sn, false);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(v.workgroups)), dim3(v.threads), lds, s, p); };
  sn == 4 ? go(k_lin_few<void, 4>) : sn == 2 ? go(k_lin_few<void, 2>) : go(k_lin_few<void, 1>);
  return hipGetLastError();
}

}  // namespace mx
