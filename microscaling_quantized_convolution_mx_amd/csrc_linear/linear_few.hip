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

#include "linear.h"
#include "linear_codes.h"

namespace mx {
namespace {

constexpr int kMaxWaves = 8;
constexpr size_t kTokenLds = size_t{48} << 10;  // for a pass' codes and scales: three workgroups share a CU where there are that many
constexpr int kSumStride = 33;                  // words per token of a wave's sums: no bank conflicts

struct FewParams {
  const uint8_t *w, *ws;
  int64_t kt;              // column tiles of a stripe
  int64_t mat_stripes;     // of one expert's matrix
  const void* x;           // unquantized tokens, or their codes
  const uint8_t* xs;       // the codes' scales
  int64_t ldx;
  void* y;
  int64_t ldy;
  int y_dtype;
  int tokens, n, k;
  const int32_t* offsets;
  int experts;
  int per_pass;            // tokens of a pass, 32 at most
  int passes;              // of all experts, at most
  int whole;               // whether an XCD takes all stripes of a pass, else an eighth
  int part;                // groups of SN stripes that it takes
};

// The lane's piece of what starts at p, an address that the wave has in common.
// (The empty asm keeps the compiler from adding the lane's part first, which
// would cost a pair of vector registers for each of these loads.)
template <class T>
__device__ __forceinline__ T lane_load(const uint8_t* p, int lane) {
  asm("" : "+s"(p));
  return ((const __attribute__((address_space(1))) T*)p)[static_cast<uint32_t>(lane)];
}

__device__ __forceinline__ void store(void* y, int dtype, int64_t i, float v) {
  if (dtype == MX_BF16) static_cast<bf16_t*>(y)[i] = from_f32<bf16_t>(v);
  else if (dtype == MX_F16) static_cast<f16_t*>(y)[i] = from_f32<f16_t>(v);
  else static_cast<float*>(y)[i] = v;
}

// TX: type of the unquantized tokens, void for codes.
template <class TX, int SN>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void k_lin_few(const FewParams p) {
  constexpr bool kFused = !std::is_void_v<TX>;
  constexpr int kAhead = 8 / SN;  // column tiles of a wave on their way
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, threads = blockDim.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), waves = threads >> 6;
  // Work: (pass of tokens, SN stripes).  An expert with many tokens has many
  // passes, each of them workgroups of its own.  Blocks go to the 8 XCDs in turn:
  // an XCD takes the x-th part of every pass' stripes, or, of many passes, every
  // eighth one (make_few).
  const int x = static_cast<int>(blockIdx.x & 7), i = static_cast<int>(blockIdx.x >> 3), d = i / p.part;
  const int u = p.whole ? d * 8 + x : d, st = (i - d * p.part + (p.whole ? 0 : x * p.part)) * SN;
  if (u >= p.passes || st * kTileR >= p.n) return;
  int e = 0, nt = p.tokens;  // without experts there is one pass
  int64_t row0 = 0, prow = 0;
  if (p.experts > 0) {
    const int pass = kFused ? p.per_pass : 32;
    Segment s;
    if (!find_segment(p.offsets, p.experts, p.tokens, u, pass, s)) return;
    const int t0 = __builtin_amdgcn_readfirstlane(s.unit) * pass;
    e = __builtin_amdgcn_readfirstlane(s.e);
    nt = min(pass, __builtin_amdgcn_readfirstlane(s.len) - t0);
    row0 = s.row0 + t0;
    prow = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(s.prow))) + t0;
  }
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
  // join the waves' sums in their order, 32 tokens x 32 lines at a time: a
  // lane holds token l32, lines 8(v/4) + 4 half + v%4
  float* sums = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int j = 0; j < SN; ++j) {
    __syncthreads();
    if (l32 < nt) {
      float* d = sums + (wave * nt + l32) * kSumStride + 4 * half;
#pragma unroll
      for (int v = 0; v < 16; ++v) d[8 * (v / 4) + v % 4] = acc[j][v];
    }
    __syncthreads();
    for (int i = tid; i < nt * 32; i += threads) {
      const int t = i >> 5, f = i & 31;
      float s = 0.0f;
      for (int q = 0; q < waves; ++q) s += sums[(q * nt + t) * kSumStride + f];
      const int col = (st + j) * 32 + f;
      if (col < p.n) store(p.y, p.y_dtype, (row0 + t) * p.ldy + col, s);
    }
  }
}

// Stripes of a workgroup: enough workgroups to fill the CUs first, then fewer
// and longer ones, which share the tokens and the search for the expert.
int stripes_per_group(int64_t stripes) { return stripes >= 2048 ? 4 : stripes >= 512 ? 2 : 1; }

// Waves of a workgroup: each takes 4 column tiles at least.
int waves_of(int64_t kt) {
  int w = kMaxWaves;
  while (w > 1 && kt < 4 * w) w /= 2;
  return w;
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
