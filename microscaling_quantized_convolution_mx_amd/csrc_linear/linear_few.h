// What the few-token kernels of the linear layers in 4 and 8 bits share: which
// tokens and stripes a workgroup takes, and the sum of its waves' results.
#pragma once

#include "linear.h"

namespace mx {
namespace {

constexpr int kMaxWaves = 8;
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

// What a workgroup takes.
struct FewWork {
  int st;        // first stripe
  int e, nt;     // expert, tokens
  int64_t row0;  // first row of X and Y
  int64_t prow;  // ... of the quantized form
};

// Work: (pass of tokens, sn stripes).  An expert with many tokens has many
// passes, each of them workgroups of its own.  Blocks go to the 8 XCDs in turn:
// an XCD takes the x-th part of every pass' stripes, or, of many passes, every
// eighth one (make_few).  pass: tokens of one.  False where the block has none.
__device__ __forceinline__ bool find_pass(const FewParams& p, int sn, int pass, FewWork& o) {
  const int x = static_cast<int>(blockIdx.x & 7), i = static_cast<int>(blockIdx.x >> 3), d = i / p.part;
  const int u = p.whole ? d * 8 + x : d;
  o.st = (i - d * p.part + (p.whole ? 0 : x * p.part)) * sn;
  if (u >= p.passes || o.st * kTileR >= p.n) return false;
  o.e = 0;
  o.nt = p.tokens;  // without experts there is one pass
  o.row0 = o.prow = 0;
  if (p.experts > 0) {
    Segment s;
    if (!find_segment(p.offsets, p.experts, p.tokens, u, pass, s)) return false;
    const int t0 = __builtin_amdgcn_readfirstlane(s.unit) * pass;
    o.e = __builtin_amdgcn_readfirstlane(s.e);
    o.nt = min(pass, __builtin_amdgcn_readfirstlane(s.len) - t0);
    o.row0 = s.row0 + t0;
    o.prow = static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(s.prow))) + t0;
  }
  return true;
}

// Joins the waves' sums in their order, 32 tokens x 32 lines at a time: a
// lane holds token l32, lines 8(v/4) + 4 half + v%4.  sums: LDS.
template <int SN>
__device__ __forceinline__ void join_sums(const FewParams& p, const f32x16 (&acc)[SN], float* sums, int nt, int64_t row0, int st) {
  const int tid = threadIdx.x, threads = blockDim.x, waves = threads >> 6;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), half = tid >> 5 & 1, l32 = tid & 31;
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

}  // namespace
}  // namespace mx
