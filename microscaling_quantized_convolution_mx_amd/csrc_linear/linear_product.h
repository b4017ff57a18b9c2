// What the products of the linear layers in 4 and 8 bits share on the device:
// which tile a workgroup takes, its stores, and the sum of a split contraction's
// pieces.
#pragma once

#include <utility>

#include "internal.h"
#include "linear.h"

namespace mx {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int I>
struct Idx {
  static constexpr int value = I;
};
template <int N, class F>
__device__ __forceinline__ void static_for(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(Idx<I>{}), ...); }(std::make_integer_sequence<int, N>());
}

struct ProductParams {
  const uint8_t *a, *as, *b, *bs;  // codes and scales
  void* out;
  int64_t akt, bkt;        // column tiles of a stripe
  int64_t bmat;            // ROWS: padded rows of one weight matrix in b
  int64_t a_rows, b_rows;  // padded rows of a and b (of all matrices)
  int64_t rows, cols;      // of out (ROWS: rows = tokens; CONTRACT: of one expert's matrix)
  int64_t ld;
  int64_t split_out;       // elements of out from one piece of a split product to the next
  int stream;              // out is written past the caches
  int ktiles;              // ROWS and one layer: column tiles to contract
  int tokens;
  const int32_t* offsets;
  int experts;
  int tiles_i, tiles_j;    // output tiles (ROWS with experts: tiles_i is an upper bound over all of them)
  int splits, split_steps; // pieces of the contraction and steps of each
};

// A value that all lanes have alike.
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
}

// What a workgroup takes.
struct Work {
  int64_t arow, brow;    // first padded rows of the tile in a and b
  int64_t orow;          // first output row
  int64_t rleft, cleft;  // rows and columns left of the matrix from the tile on
  int64_t k0;            // first column tile
  int64_t out;           // elements from p.out to its expert's matrix, or its piece of a split product
  int nsteps;            // steps of 128 columns
  int tj;                // column tile of the output
};

// Work: (expert, row tile, column tile, split).  Blocks go to the 8 XCDs in
// turn; XCD x takes the x-th eighth of the work, so that what its blocks
// share stays in its L2.  False where the block has none.
// SPREAD (CONTRACT with experts): XCD x takes the x-th eighth of every expert's
// tiles instead, so that experts with many tokens are all XCDs' work alike; the
// grid has room for a multiple of 8 tiles of each.
template <int TM, int TN, bool CONTRACT, bool SPREAD = false>
__device__ __forceinline__ bool find_work(const ProductParams& p, Work& o) {
  int ti, tj, sp = 0;
  int64_t arow = 0, brow = 0, orow = 0, rleft, k0 = 0, out = 0;
  int ksteps;  // steps of the whole contraction
  {
    int64_t total;
    if (CONTRACT || p.experts == 0) total = static_cast<int64_t>(p.tiles_i) * p.tiles_j * (CONTRACT && p.experts > 0 ? p.experts : p.splits);
    else {
      Segment s;
      int ti_all = 0;
      find_segment(p.offsets, p.experts, p.tokens, -1, TM, s, &ti_all);
      total = static_cast<int64_t>(ti_all) * p.tiles_j;
    }
    const int64_t plane = static_cast<int64_t>(p.tiles_i) * p.tiles_j;
    const int64_t per = (total + 7) / 8;
    const int64_t x = blockIdx.x & 7, i = blockIdx.x >> 3;
    int64_t w = x * per + i;
    if (SPREAD && CONTRACT && p.experts > 0) {
      const int64_t part = (plane + 7) / 8, e = i / part, in = x * part + (i - e * part);
      if (e >= p.experts || in >= plane) return false;
      w = e * plane + in;
    } else if (i >= per || w >= total) {
      return false;
    }
    // groups of 4 row tiles, walked column by column
    int rows_t = p.tiles_i;
    int z = 0;
    if (CONTRACT || p.experts == 0) {
      z = static_cast<int>(w / plane);
      w -= z * plane;
    } else {
      rows_t = static_cast<int>(total / p.tiles_j);
    }
    constexpr int G = 4;
    const int64_t band = static_cast<int64_t>(G) * p.tiles_j;
    const int bi = static_cast<int>(w / band);
    const int r = static_cast<int>(w - bi * band);
    const int h = min(G, rows_t - bi * G);
    ti = bi * G + r % h;
    tj = r / h;
    if constexpr (CONTRACT) {
      arow = static_cast<int64_t>(ti) * TM;
      orow = arow;
      rleft = p.rows - orow;
      if (p.experts > 0) {
        Segment s;
        find_segment(p.offsets, p.experts, p.tokens, z, 0, s);
        k0 = s.prow / kTileC;
        ksteps = (s.len + kPad - 1) / kPad;
        out += static_cast<int64_t>(z) * p.rows * p.ld;
      } else {
        ksteps = p.ktiles / kStepTiles;
        sp = z;
      }
      brow = static_cast<int64_t>(tj) * TN;
    } else {
      ksteps = p.ktiles / kStepTiles;
      if (p.experts > 0) {
        Segment s;
        find_segment(p.offsets, p.experts, p.tokens, ti, TM, s);
        arow = s.prow + static_cast<int64_t>(s.unit) * TM;
        orow = s.row0 + static_cast<int64_t>(s.unit) * TM;
        rleft = s.len - static_cast<int64_t>(s.unit) * TM;
        brow = s.e * p.bmat;
      } else {
        sp = z;
        arow = orow = static_cast<int64_t>(ti) * TM;
        rleft = p.rows - orow;
      }
      brow += static_cast<int64_t>(tj) * TN;
    }
  }
  int s_begin = 0, nsteps = ksteps;
  if (p.splits > 1) {
    s_begin = min(ksteps, sp * p.split_steps);
    nsteps = min(ksteps, s_begin + p.split_steps) - s_begin;
    out += sp * p.split_out;
  }
  k0 += static_cast<int64_t>(s_begin) * kStepTiles;
  // what the experts' offsets say is the same in all lanes: in scalar registers from here on
  o.arow = uniform(arow);
  o.brow = uniform(brow);
  o.orow = uniform(orow);
  o.rleft = uniform(rleft);
  o.cleft = p.cols - static_cast<int64_t>(tj) * TN;
  o.k0 = uniform(k0);
  o.nsteps = __builtin_amdgcn_readfirstlane(nsteps);
  o.tj = tj;
  o.out = out;
  return true;
}

// Output tile, waves and LDS stages of a workgroup.
template <int M, int N, int A, int B, int S>
struct Shape {
  static constexpr int TM = M, TN = N, WM = A, WN = B, kStages = S;
  static constexpr int kThreads = 64 * A * B;
};
// LDS that a wave's stores go through: 32 rows of its outputs, 16 bytes apart
// from each other so that neither the writes nor the reads conflict.
template <class U, int RN>
__host__ __device__ constexpr int store_bytes() { return 32 * (RN * 32 * static_cast<int>(sizeof(U)) + 16); }

// Stores the wave's RM x RN results of 32x32.  The MFMA leaves lane l with row l%32
// and 4 columns each at 8v + 4(l/32), v = 0..3: stored from there, a memory
// instruction would write 32 short pieces.  Through LDS, 32 rows at a time,
// it writes whole rows, 16 bytes per lane.
// dst: the tile's first output; rleft, cleft: rows and columns from there on
// that exist.
// STREAM: past the caches.
template <bool STREAM, int RM, int RN, class U>
__device__ __forceinline__ void store_wave(const f32x16 (&acc)[RM][RN], uint8_t* buf, U* dst, int64_t ld, int64_t rleft,
                                           int64_t cleft, int lane, int wm, int wn) {
  constexpr int W = RN * 32;                                  // columns of the wave
  constexpr int kRow = W * static_cast<int>(sizeof(U)) + 16;  // bytes between rows in LDS
  constexpr int N = 16 / static_cast<int>(sizeof(U));         // elements of 16 bytes
  constexpr int P = W / N;                                    // 16-byte pieces of a row
  const int64_t c0 = wn * W;
  cleft -= c0;
  rleft -= wm * RM * 32;
  dst += static_cast<int64_t>(wm * RM * 32) * ld + c0;
#pragma unroll
  for (int i = 0; i < RM; ++i) {
#pragma unroll
    for (int j = 0; j < RN; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        struct alignas(4 * sizeof(U)) { U e[4]; } q;
#pragma unroll
        for (int w = 0; w < 4; ++w) q.e[w] = from_f32<U>(acc[i][j][4 * v + w]);
        __builtin_memcpy(__builtin_assume_aligned(buf + (lane & 31) * kRow + (32 * j + 8 * v + 4 * (lane >> 5)) * sizeof(U), 4 * sizeof(U)), &q, sizeof(q));
      }
    __builtin_amdgcn_wave_barrier();
    U* d = dst + static_cast<int64_t>(32 * i) * ld;
    const int64_t left = rleft - 32 * i;
#pragma unroll
    for (int s = 0; s < 32 * P / 64; ++s) {
      const int r = (s * 64 + lane) / P, c = (s * 64 + lane) % P * N;
      const i32x4 q = *reinterpret_cast<const i32x4*>(buf + r * kRow + c * sizeof(U));
      if (r < left) {
        if (c + N <= cleft) {
          if constexpr (STREAM) stream16(d + r * ld + c, q);
          else store16(d + r * ld + c, q);
        } else {
          for (int e = 0; e < N; ++e)
            if (c + e < cleft) d[r * ld + c + e] = reinterpret_cast<const U*>(buf + r * kRow + c * sizeof(U))[e];
        }
      }
    }
    __builtin_amdgcn_wave_barrier();
  }
}

// Waits until at most N of the wave's copies and none of its LDS reads are on
// their way, then for the workgroup's other waves to have come as far.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  static_assert(N < 64);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" : : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Sums the pieces of a split product in their order, 4 columns per thread.
template <class T>
__global__ __launch_bounds__(256) void k_lin_reduce(const float* __restrict__ partial, int splits, int64_t rows, int64_t cols,
                                                     int64_t pcols, T* __restrict__ out, int64_t ld) {
  const int64_t n = rows * pcols / 4;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256) {
    f32x4 s = reinterpret_cast<const f32x4*>(partial)[i];
    for (int q = 1; q < splits; ++q) s += reinterpret_cast<const f32x4*>(partial)[q * n + i];
    const int64_t r = 4 * i / pcols, c = 4 * i - r * pcols;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < cols) out[r * ld + c + e] = from_f32<T>(s[e]);
  }
}

}  // namespace
}  // namespace mx
