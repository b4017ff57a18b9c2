// Products of the linear layers in 8 bits with few tokens:
//   y[t][i] = sum_c x[t][c] w[i][c]
// with the lines of w in a form whose columns are c (fwd: W's row form, dgrad:
// W's column form), and x either in its row form or, for serving, unquantized
// and quantized here (1x128 blocks), in one launch.
//
// Bound by w's bytes, or by the launch where there are few of them.  Work is
// dealt out as in 4 bits: a workgroup takes SN stripes of 32 lines of w, whose
// column tiles its waves take in turn, straight from memory into registers,
// several of them on their way, and their sums are joined in LDS.  Its tokens,
// 32 at most, come from memory (L2) in the same way, or are quantized into LDS
// while the first tiles of w are on their way.
//
// The codes are widened to bf16 with their scales, and the products are exact
// whatever the output's type: the matrix units have time for that while w
// arrives.  Tokens quantized here are kept in LDS as bf16.
//
// Measured in graphs of such calls, which leave the weight in the last-level
// cache: 1x16384x8192 22.8 us (5.9 TB/s of weight) or, quantizing, 23.9,
// 1x4096x4096 5.7 and 5.4 (128 workgroups: half of the CUs have none, which stripes of
// 16 lines would change; not tried), 256 tokens of 64 experts, 2048x2048, 42 (6.4 TB/s).
#include <algorithm>
#include <type_traits>

#include "linear8_codes.h"
#include "linear_few.h"

namespace mx {
namespace {

// Stripes of a workgroup.  (Four, as in 4 bits, would take more registers than
// half of a SIMD's, which two workgroups share.)
int stripes8_per_group(int64_t stripes) { return std::min(stripes_per_group(stripes), 2); }

// TX: type of the unquantized tokens, void for codes.
template <class TX, int SN>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void k_lin8_few(const FewParams p) {
  constexpr bool kFused = !std::is_void_v<TX>;
  // column tiles of a wave on their way, in half of the registers (1x4096x4096
  // quantizing 5.4 us, 7.6 with 6 of them, 5.8 with 8 in all registers; not
  // quantizing 5.7, 7.3 with 4, which spill)
  constexpr int kAhead = SN == 1 ? kFused ? 4 : 3 : 2;
  // loads of the tokens at once (20x4096x1024 7.4 us, 8.0 with one; 31x1024x1024 9.5 and 10.4)
  constexpr int kLoads = sizeof(std::conditional_t<kFused, TX, float>) == 2 ? 4 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
  FewWork w0;
  if (!find_pass(p, SN, kFused ? p.per_pass : 32, w0)) return;
  const int st = w0.st, nt = w0.nt;
  const int64_t row0 = w0.row0, prow = w0.prow;
  const int kt = static_cast<int>(p.kt);
  const int64_t stripe = static_cast<int64_t>(w0.e) * p.mat_stripes + st;
  const uint8_t* wsrc = p.w + stripe * p.kt * k8TileBytes;
  const uint8_t* ssrc = p.ws + (stripe / 4) * (p.kt / 2) * k8ScaleBytes;
  const int sbyte = static_cast<int>(stripe & 3);  // SN stripes lie in one group of four
  const int half = lane >> 5, l32 = lane & 31;
  struct Tile { i32x4 lo, hi; };
  Tile w[kAhead][SN], xv[kFused ? 1 : kAhead];
  int ws[kAhead], xs[kFused ? 1 : kAhead];
  // the wave's column tiles; a fetch past them takes the last one again
  const int chunk = (kt + waves - 1) / waves, begin = min(wave * chunk, kt), end = min(begin + chunk, kt);
  auto tile = [&](const uint8_t* at) { return Tile{lane_load<i32x4>(at, lane), lane_load<i32x4>(at + 1024, lane)}; };
  auto fetch = [&](int q, int t) {
    t = max(min(t, end - 1), 0);
#pragma unroll
    for (int j = 0; j < SN; ++j) w[q][j] = tile(wsrc + (j * p.kt + t) * k8TileBytes);
    ws[q] = lane_load<int>(ssrc + static_cast<int64_t>(t / 2) * k8ScaleBytes, l32);
    if constexpr (!kFused) {
      xv[q] = tile(static_cast<const uint8_t*>(p.x) + ((prow / kTileR) * p.kt + t) * k8TileBytes);
      xs[q] = lane_load<int>(p.xs + ((prow / kPad) * (p.kt / 2) + t / 2) * k8ScaleBytes, l32);
    }
  };
#pragma unroll
  for (int q = 0; q < kAhead; ++q) fetch(q, begin + q);

  if constexpr (kFused) {
    // a thread takes a token's 8 columns at a time, 16 of them a block; 8
    // columns c/8 of token r are at (c/8 * nt + r) * 16.  (An odd stride between
    // columns, free of bank conflicts, changes nothing.)
    const int nc = kt * (kTileC / 8), all = nc * nt;
    for (int b0 = tid; b0 < all; b0 += kLoads * threads) {
      Raw8<TX> raw[kLoads];
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int b = b0 + i * threads, r = b / nc, c = b - r * nc;
        if (b < all) raw[i] = load_raw8(static_cast<const TX*>(p.x) + (row0 + r) * p.ldx, static_cast<int64_t>(c) * 8, p.k);
      }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int b = b0 + i * threads, r = b / nc, c = b - r * nc;
        if (b >= all) break;  // (blocks are whole: 16 lanes)
        float v[8];
        unpack8(raw[i], v);
        const uint32_t code = block8_code(row16_max(amax8(v)));
        const uint2 e = encode8x8(v, code);
        reinterpret_cast<bf16x8*>(lds)[c * nt + r] = widen8(static_cast<int>(e.x), static_cast<int>(e.y), __uint_as_float(code << 23));
      }
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
  const int xbyte = kFused ? 0 : static_cast<int>(prow / kTileR & 3);
  auto both = [](const Tile& t) { return i32x8{t.lo.x, t.lo.y, t.lo.z, t.lo.w, t.hi.x, t.hi.y, t.hi.z, t.hi.w}; };
  auto multiply = [&](int q, int t, bool in) {
    Wide x;
    if constexpr (kFused) {
#pragma unroll
      for (int i = 0; i < 4; ++i) x.k[i] = reinterpret_cast<const bf16x8*>(lds)[(8 * t + 4 * (i / 2) + 2 * half + i % 2) * nt + r];
    } else {
      x = widen(both(xv[q]), static_cast<uint32_t>(xs[q]), xbyte);
    }
    const int m = in ? -1 : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) x.k[i] = __builtin_bit_cast(bf16x8, __builtin_bit_cast(i32x4, x.k[i]) & m);
#pragma unroll
    for (int j = 0; j < SN; ++j) {
      const Wide a = widen(both(w[q][j]), static_cast<uint32_t>(ws[q]), sbyte + j);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a.k[i], x.k[i], acc[j], 0, 0, 0);
    }
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

// LDS of a pass: the tokens, and then the waves' sums in their place.
size_t fused_lds(int64_t kt, int waves, int tokens) {
  const size_t x = static_cast<size_t>(kt) * kTileC * 2 * tokens, s = static_cast<size_t>(waves) * tokens * kSumStride * 4;
  return ((x > s ? x : s) + 15) / 16 * 16;
}

// Tokens of a pass, whose LDS is the most that any workgroup may need.  Without
// experts a pass has all tokens, and two workgroups share a CU.  With experts,
// most of which have few, as many share it as its registers hold, 16 waves, and
// an expert with more tokens takes more passes: 64 tokens of 64 experts,
// 2048x1024, 23.5 us evenly spread (5.7 TB/s of weight), 16.4 at random, 9.9 all on
// one expert; with 64 KiB for every workgroup 27.4, 19.6 and 12.8 (1024x512,
// 256 tokens at random, 9.1 and 8.9).
int tokens_per_pass(int64_t kt, bool experts) {
  const size_t most = experts ? std::min<size_t>(64, 10 * waves_of(kt)) << 10 : size_t{64} << 10;
  int t = 32;
  while (t > 0 && fused_lds(kt, waves_of(kt), t) > most) --t;
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
  sn = stripes8_per_group(stripes * g.ew);
  const int64_t most = fused ? tokens_per_pass(p.kt, g.e > 0) : 32;
  p.per_pass = static_cast<int>(g.m < most ? g.m : most);
  // an expert with tokens has one pass, and one more for every per_pass tokens past its first
  const int64_t used = g.m < g.ew ? g.m : g.ew;
  p.passes = g.e > 0 ? static_cast<int>(used + (g.m - used) / p.per_pass) : 1;
  // An XCD takes an eighth of each pass' stripes, or of 64 passes and more whole
  // ones, one in eight, as in 4 bits.  Whole groups of four stripes, which share
  // scale words.
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

LinVariant lin8_few_variant(const LinGeom& g, bool dgrad, bool fused) {
  const mx_linear_qtensor none{};
  int sn;
  const FewParams p = make_few(g, dgrad, fused, &none, nullptr, MX_F32, 0, nullptr, sn);
  return variant(p, sn, fused);
}

// Whether every group of an expert's stripes quantizes the tokens for itself,
// which is cheaper than a launch of its own while they are few: the rule of
// the 4-bit kernel.
bool lin8_fused(const LinGeom& g) {
  const int64_t kt = g.kp / kTileC, stripes = (g.n + kTileR - 1) / kTileR;
  const int t = tokens_per_pass(kt, g.e > 0), sn = stripes8_per_group(stripes * g.ew);
  const int64_t groups = (stripes + sn - 1) / sn;
  if (t == 0 || g.m * g.kp * groups >= (int64_t{1} << 24)) return false;
  return g.e == 0 ? g.m <= t : lin8_few(g);
}

// One pass of tokens, or experts with few tokens each.
bool lin8_few(const LinGeom& g) { return g.e == 0 ? g.m <= 32 : g.m <= 16 * static_cast<int64_t>(g.e); }

hipError_t launch_lin8_fused(const LinGeom& g, const mx_linear_qtensor* wq, const void* x, mx_dtype x_dtype, int64_t ldx,
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
    sn == 2 ? go(k_lin8_few<T, 2>) : go(k_lin8_few<T, 1>);
  };
  switch (x_dtype) {
    case MX_BF16: with(bf16_t{}); break;
    case MX_F16: with(f16_t{}); break;
    default: with(float{}); break;
  }
  return hipGetLastError();
}

hipError_t launch_lin8_few(const LinGeom& g, bool dgrad, const mx_linear_qtensor* wq, const mx_linear_qtensor* xq, void* y,
                           mx_dtype y_dtype, int64_t ldy, const int32_t* offsets, hipStream_t s) {
  int sn;
  FewParams p = make_few(g, dgrad, false, wq, y, y_dtype, ldy, offsets, sn);
  p.x = xq->rows;
  p.xs = xq->row_scales;
  const size_t lds = static_cast<size_t>(waves_of(p.kt)) * p.per_pass * kSumStride * 4;
  const LinVariant v = variant(p, sn, false);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(v.workgroups)), dim3(v.threads), lds, s, p); };
  sn == 2 ? go(k_lin8_few<void, 2>) : go(k_lin8_few<void, 1>);
  return hipGetLastError();
}

}  // namespace mx
