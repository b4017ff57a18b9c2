// The products of the microscaled linear layers on the scaled FP4 MFMA.
//
// out[i][j] = sum_c a[i][c] b[j][c] with both operands in a form whose
// columns are c (mxlinear.h):
//   fwd    a = X rows,   b = W rows,   c = in features
//   dgrad  a = dY rows,  b = W cols,   c = out features
//   wgrad  a = dY cols,  b = X cols,   c = tokens
// so one kernel serves all three.  With experts, fwd and dgrad take the rows
// of `a` in segments with a weight matrix each (ROWS), wgrad the columns in
// segments with an output matrix each (CONTRACT).
//
// Measured (bf16 outputs, fp32 for wgrad): 8192x8192x8192 238 to 278 us, 4.0 to
// 4.6 PFLOP/s; 16384x4096x4096 forward 131 to 146, weight gradient 115 to 120;
// 4096^3 36.  In 8192^3 the MFMA is busy 61% of the time at 1.74 GHz of 2.4, in
// the 16384x4096x4096 forward 47% at 1.92: power sets the clock, and a part of
// the rest (of 76 us in the latter about 36) is the start and the end of each
// round of 256 tiles, whose first operands and stores take about 9 us without
// MFMAs by the fit of make_plan.  Experts' products run
// at the full clock: 16 experts of 2048x2048 with 16384 uneven tokens 61 us
// forward, 23% busy, and 118 for the weight gradient, 12%, which waits for the
// XCDs with the most tokens (70 with even ones; its stores take 52).
#include "linear_product.h"

#include <limits>
#include <type_traits>

namespace mx {
namespace {

// Big for the MFMA's rate, Tiny for short latency (make_plan).
using Big = Shape<256, 256, 2, 2, 4>;
using Small = Shape<128, 128, 2, 2, 4>;
using Tiny = Shape<64, 64, 2, 2, 4>;

// Copies BYTES per lane from src + lane * BYTES to the LDS address dst + lane *
// BYTES without passing registers.  src and dst are the wave's.  The compiler
// does not know of the copy (told of it, it would wait for all copies on
// their way before any LDS read), so whoever reads the data waits for it with
// wait_barrier.  There is no output register, and the address registers are
// read when the instruction issues.  The LDS address goes in m0, which is an
// operand, so that the compiler writes it and knows of it (and an instruction
// has to pass between that write and the copy).
template <int BYTES>
__device__ __forceinline__ void copy_lds(const uint8_t* src, uint32_t dst, int lane) {
  const uint32_t off = static_cast<uint32_t>(lane) * BYTES;
  if constexpr (BYTES == 16)
    asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" : : "{m0}"(dst), "v"(off), "s"(src) : "memory");
  else
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %1, %2" : : "{m0}"(dst), "v"(off), "s"(src) : "memory");
}

// TM x TN outputs per workgroup, by WM x WN waves in MFMAs of 32x32x64.  One
// step contracts 128 columns: two MFMA slices.  A tile in LDS is read as it
// is, 64 lanes x 16 consecutive bytes, which is free of bank conflicts.
template <class T, class Shape, bool CONTRACT>
__global__ __launch_bounds__(64 * Shape::WM * Shape::WN) void k_lin_product(const ProductParams p) {
  constexpr int TM = Shape::TM, TN = Shape::TN, WM = Shape::WM, WN = Shape::WN, kStages = Shape::kStages;
  constexpr int RM = TM / WM / 32, RN = TN / WN / 32;  // MFMA rows and columns of a wave
  constexpr int kWaves = WM * WN;
  constexpr int kOpndA = TM / 32 * kStepTiles * kTileBytes, kOpndB = TN / 32 * kStepTiles * kTileBytes;
  // 256-byte groups of scales, of 128 rows each (of which a tile of 64 uses half)
  constexpr int kGroupsA = (TM + kPad - 1) / kPad * kStepTiles, kGroups = kGroupsA + (TN + kPad - 1) / kPad * kStepTiles;
  constexpr int kScales = kOpndA + kOpndB;  // their place in a stage
  constexpr int kStage = kScales + kGroups * kScaleBytes;
  constexpr int kStoreBytes = kWaves * store_bytes<T, RN>();
  __shared__ __attribute__((aligned(16))) uint8_t lds[kStages * kStage > kStoreBytes ? kStages * kStage : kStoreBytes];

  const int tid = threadIdx.x;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave % WM, wn = wave / WM;

  // Work: (expert, row tile, column tile, split).
  Work w;
  if (!find_work<TM, TN, CONTRACT>(p, w)) return;
  const int64_t arow = w.arow, brow = w.brow, orow = w.orow, rleft = w.rleft, cleft = w.cleft, k0 = w.k0;
  const int tj = w.tj, nsteps = w.nsteps;
  T* out = static_cast<T*>(p.out) + w.out;

  // Copies.  A step's tiles go from memory to LDS as they are stored, without
  // passing registers: copy l of wave w takes tile l * kWaves + w of a's, then
  // b's tiles (two columns of them, 64 lanes x 16 bytes each) and then groups
  // of scales.  A stripe past the operand's end is read as its last one:
  // those outputs are not stored.
  constexpr int kTilesA = TM / 16 / kWaves, kTiles = (TM + TN) / 16 / kWaves;
  constexpr int kScaleCopies = (kGroups + kWaves - 1) / kWaves, kCopies = kTiles + kScaleCopies;
  static_assert(TM / 16 % kWaves == 0 && TN / 16 % kWaves == 0);
  const uint8_t *src[kTiles], *ssrc[kScaleCopies];
  uint32_t sdst[kScaleCopies];
  static_for<kTiles>([&](auto lc) {
    constexpr int L = decltype(lc)::value;
    constexpr bool of_b = L >= kTilesA;
    const int i = (of_b ? L - kTilesA : L) * kWaves + wave;
    const int64_t st = min((of_b ? brow : arow) / kTileR + i / kStepTiles, (of_b ? p.b_rows : p.a_rows) / kTileR - 1);
    src[L] = (of_b ? p.b : p.a) + (st * (of_b ? p.bkt : p.akt) + k0 + i % kStepTiles) * kTileBytes;
  });
  static_for<kScaleCopies>([&](auto lc) {
    constexpr int L = decltype(lc)::value;
    const int i = min(L * kWaves + wave, kGroups - 1);  // (the last group may be copied twice)
    const bool of_b = i >= kGroupsA;
    const int j = of_b ? i - kGroupsA : i;
    const int64_t g = min((of_b ? brow : arow) / kPad + j / kStepTiles, (of_b ? p.b_rows : p.a_rows) / kPad - 1);
    ssrc[L] = (of_b ? p.bs : p.as) + (g * (of_b ? p.bkt : p.akt) + k0 + j % kStepTiles) * kScaleBytes;
    sdst[L] = kScales + static_cast<uint32_t>(i) * kScaleBytes;
  });
  const uint32_t lds0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  // copy l of the step that the sources stand at, into the stage at `to`
  auto copy = [&](uint32_t to, auto l) {
    constexpr int L = decltype(l)::value;
    if constexpr (L < kTiles) copy_lds<16>(src[L], lds0 + to + (L * kWaves + wave) * kTileBytes, lane);
    else copy_lds<4>(ssrc[L - kTiles], lds0 + to + sdst[L - kTiles], lane);
  };
  auto advance = [&](bool on) {
    const int d = on ? 1 : 0;
#pragma unroll
    for (int q = 0; q < kTiles; ++q) src[q] += d * (kStepTiles * kTileBytes);
#pragma unroll
    for (int i = 0; i < kScaleCopies; ++i) ssrc[i] += d * (kStepTiles * kScaleBytes);
  };

  f32x16 acc[RM][RN];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < RN; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  struct Frags {
    i32x8 a[RM], b[RN];
    int sa, sb;
  };
  Frags fA, fB;
  // a wave's scales: the bytes of its 1, 2 or 4 stripes among 128 rows' four
  auto read_scales = [&](const uint8_t* s, int stripe, int n, int j) -> int {
    const uint8_t* at = s + ((stripe >> 2) * kStepTiles + j) * kScaleBytes + 4 * lane + (stripe & 3);
    return n == 4 ? *reinterpret_cast<const int*>(at) : n == 2 ? *reinterpret_cast<const uint16_t*>(at) : *at;
  };
  // (the tile's first stripe among its 128 rows' four)
  const int sa0 = TM < kPad ? static_cast<int>(arow / kTileR & 3) : 0, sb0 = TN < kPad ? static_cast<int>(brow / kTileR & 3) : 0;
  // read r of slice j: the scales, then the tiles in the order of their use
  constexpr int kReads = RM + RN + 2;
  auto read = [&](const uint8_t* st, int j, Frags& f, auto r) {
    constexpr int R = decltype(r)::value;
    if constexpr (R == 0) {
      f.sa = read_scales(st + kScales, sa0 + wm * RM, RM, j);
    } else if constexpr (R == 1) {
      f.sb = read_scales(st + kScales + kGroupsA * kScaleBytes, sb0 + wn * RN, RN, j);
    } else if constexpr (R == 2 || R >= RN + 3) {
      constexpr int I = R == 2 ? 0 : R - RN - 2;
      f.a[I] = operand(reinterpret_cast<const i32x4*>(st + ((wm * RM + I) * kStepTiles + j) * kTileBytes)[lane]);
    } else {
      constexpr int I = R - 3;
      f.b[I] = operand(reinterpret_cast<const i32x4*>(st + kOpndA + ((wn * RN + I) * kStepTiles + j) * kTileBytes)[lane]);
    }
  };

  // Step s, on stage s%S of S, with slice 0's operands read during step s-1:
  //   multiply slice 0, reading slice 1 and copying the second half of step
  //   s+S-1 into stage (s+S-1)%S;
  //   barrier: every wave has read all of stage s%S, and its copies of step
  //   s+1 have arrived (those of the S-2 steps after may be on their way);
  //   multiply slice 1, reading slice 0 of step s+1 and copying the first
  //   half of step s+S into stage s%S.
  // With one wave per SIMD nothing else hides an LDS access, so reads and
  // copies are dealt out between the MFMAs: an MFMA lasts 32 cycles, in which
  // LDS serves about one 1 KiB access of each of the four waves.  Copies past
  // the last step repeat it, into stages that nothing reads.
  constexpr int kSlots = RM * RN;
  auto mfma = [&](const Frags& f, auto n) {
    constexpr int I = decltype(n)::value / RN, J = decltype(n)::value % RN;
    acc[I][J] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(f.b[J], f.a[I], acc[I][J], 4, 4, J, f.sb, I, f.sa);
    __builtin_amdgcn_sched_barrier(0);
  };
  // items first .. first+count-1 dealt out evenly over a slice's first `span`
  // MFMAs: those that follow MFMA n
  auto deal = [&](auto n, auto first, auto count, auto span, auto&& f) {
    constexpr int N = decltype(n)::value, C = decltype(count)::value, S = decltype(span)::value;
    constexpr int B = N < S ? (N * C + S - 1) / S : C, E = N + 1 < S ? ((N + 1) * C + S - 1) / S : C;
    static_for<E - B>([&](auto i) { f(Idx<decltype(first)::value + B + decltype(i)::value>{}); });
  };
  constexpr int kHalf = kCopies / 2;
  if (nsteps > 0) {
    static_for<kStages>([&](auto st) {
      // the last stage's second half follows in the loop
      constexpr int S = decltype(st)::value;
      static_for<S + 1 < kStages ? kCopies : kHalf>([&](auto l) { copy(S * kStage, l); });
      if constexpr (S + 1 < kStages) advance(S + 1 < nsteps);
    });
    wait_barrier<(kStages - 2) * kCopies + kHalf>();
    static_for<kReads>([&](auto r) {
      read(lds, 0, fA, r);
      __builtin_amdgcn_sched_barrier(0);
    });
    uint32_t cur = 0, last = (kStages - 1) * kStage;
    for (int s = 0; s < nsteps; ++s) {
      const uint32_t next = cur == (kStages - 1) * kStage ? 0 : cur + kStage;
      static_for<kSlots>([&](auto n) {
        mfma(fA, n);
        deal(n, Idx<0>{}, Idx<kReads>{}, Idx<(kSlots * 3 + 3) / 4>{}, [&](auto r) { read(lds + cur, 1, fB, r); });
        deal(n, Idx<kHalf>{}, Idx<kCopies - kHalf>{}, Idx<kSlots>{}, [&](auto l) { copy(last, l); });
        __builtin_amdgcn_sched_barrier(0);
      });
      advance(s + kStages < nsteps);
      wait_barrier<(kStages - 2) * kCopies>();
      static_for<kSlots>([&](auto n) {
        mfma(fB, n);
        deal(n, Idx<0>{}, Idx<kReads>{}, Idx<kSlots>{}, [&](auto r) { read(lds + next, 0, fA, r); });
        deal(n, Idx<0>{}, Idx<kHalf>{}, Idx<kSlots>{}, [&](auto l) { copy(cur, l); });
        __builtin_amdgcn_sched_barrier(0);
      });
      last = cur;
      cur = next;
    }
    // the last copies have to land before the stores reuse LDS
    wait_barrier<0>();
  }

  T* tile = out + orow * p.ld + static_cast<int64_t>(tj) * TN;
  uint8_t* buf = lds + wave * store_bytes<T, RN>();
  if (p.stream) store_wave<true, RM, RN>(acc, buf, tile, p.ld, rleft, cleft, lane, wm, wn);
  else store_wave<false, RM, RN>(acc, buf, tile, p.ld, rleft, cleft, lane, wm, wn);
}

struct Plan {
  int shape;    // 0: Tiny, 1: Small, 2: Big
  int64_t tiles_i, tiles_j;
  int splits, split_steps;
  int64_t units;  // workgroups, at most
};

LinVariant variant(const Plan& pl) {
  const int size = pl.shape == 2 ? Big::TM : pl.shape == 1 ? Small::TM : Tiny::TM;
  const int threads = pl.shape == 2 ? Big::kThreads : pl.shape == 1 ? Small::kThreads : Tiny::kThreads;
  return {3, size, pl.splits, threads, (pl.units * pl.splits + 7) / 8 * 8};
}

// Tiles and split by estimated time, in us, fitted to measured products (bf16
// outputs, 64 to 8192 rows and 512 to 8192 columns).  A round is 256
// workgroups, one per CU:
//   Big    9 for the first loads and the stores, 0.8 per step and round, bound
//          by the MFMA (4096x4096x4096 39, Small 42)
//   Small  5, and 0.28 per step and round, bound by L2 (2048^3 9.7, Tiny 11.8,
//          Big 18)
//   Tiny   3.6, and 0.13 per step and round, bound by the latency of a step
//          (777x1000x520 4.6, Small 7.4; 301x2500x1999 6.3, Small 9.3)
// Splitting the contraction costs a launch, 3, and the traffic of its partial
// sums at 4 TB/s: it pays for long contractions with few outputs, seldom else
// (512x4096x4096 by Small 12.7, in 2 pieces 18.3).  Tiles too small for a
// launch's 2^32 - 1 threads are left out (a contraction of length 0 over 2^36
// outputs would take Tiny): check_desc keeps Small and Big below that.
Plan make_plan(const LinGeom& g, LinOp op) {
  const int64_t rows = op == LIN_WGRAD ? g.n : g.m, cols = op == LIN_FWD ? g.n : g.k;
  const int64_t contract = op == LIN_FWD ? g.kp : op == LIN_DGRAD ? g.np : g.mp;
  const int64_t used = g.m < g.ew ? g.m : g.ew;
  // steps of a tile: with experts, wgrad contracts one's share of the tokens
  const int64_t all_steps = contract / kPad;
  const double steps = op == LIN_WGRAD ? static_cast<double>(all_steps) / g.ew : static_cast<double>(all_steps);
  Plan best{};
  double best_time = 0.0;
  auto consider = [&](int shape, int64_t pieces) {
    Plan pl{};
    const int tm = shape == 2 ? Big::TM : shape == 1 ? Small::TM : Tiny::TM, tn = shape == 2 ? Big::TN : shape == 1 ? Small::TN : Tiny::TN;
    // every expert with tokens may leave a part of a tile more
    const int64_t extra = op != LIN_WGRAD && g.e > 0 ? used : 0;
    pl.shape = shape;
    pl.tiles_i = (rows + tm - 1) / tm + extra;
    pl.tiles_j = (cols + tn - 1) / tn;
    pl.units = pl.tiles_i * pl.tiles_j * (op == LIN_WGRAD ? g.ew : 1);
    pl.split_steps = static_cast<int>((all_steps + pieces - 1) / pieces);
    pl.splits = pieces > 1 ? static_cast<int>((all_steps + pl.split_steps - 1) / pl.split_steps) : 1;
    const int64_t likely = pl.units - extra * pl.tiles_j / 2;
    const double rounds = static_cast<double>((likely * pl.splits + 255) / 256), each = steps / pl.splits;
    double time = shape == 2 ? rounds * (9.0 + 0.8 * each) : shape == 1 ? 5.0 + rounds * 0.28 * each : 3.6 + rounds * 0.13 * each;
    if (pl.splits > 1) time += 3.0 + 8.0 * static_cast<double>(rows * cols) * pl.splits / 4e6;
    const LinVariant v = variant(pl);
    if (v.workgroups * v.threads > std::numeric_limits<uint32_t>::max()) return;
    if (best.units == 0 || time < best_time) {
      best = pl;
      best_time = time;
    }
  };
  for (int shape : {0, 1, 2}) consider(shape, 1);
  if (g.e == 0)
    for (int64_t s = 2; s <= 16 && 4 * s <= all_steps; s *= 2) consider(0, s);
  return best;
}

}  // namespace

LinVariant lin_product_variant(const LinGeom& g, LinOp op) {
  if (op != LIN_WGRAD && g.m == 0) return {};
  if (op != LIN_WGRAD && lin_few(g)) return lin_few_variant(g, op == LIN_DGRAD, false);
  return variant(make_plan(g, op));
}

// Whether the product writes past the caches: outputs that the last-level cache
// cannot hold (16 experts' 4096x4096 fp32 gradients: 202 us, 258 through the
// caches); smaller ones stay in it for the next layer (4096x4096 bf16: 46 us
// with a quantization of the result, 48 past the caches).  Rows that do not
// start at multiples of 64 bytes go through the caches, which join the lines
// that two stores share (8200x16391x128 bf16: 69 us, 117 past them; 16400 columns
// 66 and 96; 16416, whole 64 bytes, 66 and 62).
bool lin_product_streams(const LinGeom& g, LinOp op, const void* out, mx_dtype dtype, int64_t ld) {
  const int64_t rows = op == LIN_WGRAD ? g.n * g.ew : g.m, cols = op == LIN_FWD ? g.n : g.k;
  const int64_t size = dtype == MX_F32 ? 4 : 2;
  return static_cast<size_t>(rows * cols * size) >= kStreamOutBytes && whole_lines(out, ld * size);
}

size_t lin_product_workspace(const LinGeom& g, LinOp op) {
  if (g.m == 0 || (op != LIN_WGRAD && lin_few(g))) return 0;
  const Plan pl = make_plan(g, op);
  if (pl.splits <= 1) return 0;
  const int64_t rows = op == LIN_WGRAD ? g.n : g.m, cols = op == LIN_FWD ? g.n : g.k;
  return static_cast<size_t>(pl.splits * rows * ((cols + 3) / 4 * 4)) * sizeof(float);
}

hipError_t launch_lin_product(const LinGeom& g, LinOp op, const mx_linear_qtensor* aq, const mx_linear_qtensor* bq,
                              void* out, mx_dtype dtype, int64_t ld, const int32_t* offsets, void* workspace,
                              hipStream_t s) {
  if (op != LIN_WGRAD && g.m == 0) return hipSuccess;
  if (op != LIN_WGRAD && lin_few(g)) return launch_lin_few(g, op == LIN_DGRAD, bq, aq, out, dtype, ld, offsets, s);
  const Plan pl = make_plan(g, op);
  ProductParams p{};
  const mx_role ra = op == LIN_FWD ? MX_ROLE_ACT : MX_ROLE_GRAD, rb = op == LIN_WGRAD ? MX_ROLE_ACT : MX_ROLE_WEIGHT;
  const mx_form fa = op == LIN_WGRAD ? MX_FORM_COLS : MX_FORM_ROWS, fb = op == LIN_FWD ? MX_FORM_ROWS : MX_FORM_COLS;
  p.a = static_cast<const uint8_t*>(fa == MX_FORM_ROWS ? aq->rows : aq->cols);
  p.as = fa == MX_FORM_ROWS ? aq->row_scales : aq->col_scales;
  p.b = static_cast<const uint8_t*>(fb == MX_FORM_ROWS ? bq->rows : bq->cols);
  p.bs = fb == MX_FORM_ROWS ? bq->row_scales : bq->col_scales;
  int64_t c;
  form_dims(g, ra, fa, p.a_rows, c);
  p.akt = c / kTileC;
  p.ktiles = static_cast<int>(c / kTileC);
  form_dims(g, rb, fb, p.bmat, c);
  p.bkt = c / kTileC;
  p.b_rows = p.bmat * form_matrices(g, rb);
  p.rows = op == LIN_WGRAD ? g.n : g.m;
  p.cols = op == LIN_FWD ? g.n : g.k;
  // a split product leaves fp32 sums in the workspace, with rows of whole 16
  // bytes, for k_lin_reduce
  const bool split = pl.splits > 1;
  const int64_t pcols = (p.cols + 3) / 4 * 4;
  p.out = split ? workspace : out;
  p.ld = split ? pcols : ld;
  p.split_out = p.rows * pcols;
  p.stream = !split && lin_product_streams(g, op, out, dtype, ld);
  p.tokens = static_cast<int>(g.m);
  p.offsets = offsets;
  p.experts = g.e;
  p.tiles_i = static_cast<int>(pl.tiles_i);
  p.tiles_j = static_cast<int>(pl.tiles_j);
  p.splits = pl.splits;
  p.split_steps = pl.split_steps;
  const LinVariant v = variant(pl);
  auto multiply = [&](auto t) {
    using T = decltype(t);
    auto launch = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(v.workgroups)), dim3(v.threads), 0, s, p); };
    auto with = [&](auto contract) {
      constexpr bool C = decltype(contract)::value;
      pl.shape == 2 ? launch(k_lin_product<T, Big, C>) : pl.shape == 1 ? launch(k_lin_product<T, Small, C>) : launch(k_lin_product<T, Tiny, C>);
    };
    op == LIN_WGRAD ? with(std::true_type{}) : with(std::false_type{});
  };
  auto reduce = [&](auto t) {
    using T = decltype(t);
    const int64_t n = p.rows * pcols / 4;
    const unsigned wgs = static_cast<unsigned>(n / 256 < 2048 ? (n + 255) / 256 : 2048);
    hipLaunchKernelGGL(k_lin_reduce<T>, dim3(wgs), dim3(256), 0, s, static_cast<const float*>(workspace), p.splits, p.rows, p.cols, pcols,
                       static_cast<T*>(out), ld);
  };
  auto go = [&](auto t) {
    if (!split) multiply(t);
    else {
      multiply(float{});
      reduce(t);
    }
  };
  switch (dtype) {
    case MX_BF16: go(bf16_t{}); break;
    case MX_F16: go(f16_t{}); break;
    default: go(float{}); break;
  }
  return hipGetLastError();
}

}  // namespace mx
