// The tokens' way to their experts and back: a stable sort of the choices by
// expert, and the moves of rows that it orders.
//
// Sort.  Choices are counted and placed 64 at a time by a wave: a ballot for
// each bit of the expert's number gives every lane the mask of the lanes that
// chose the same one, whose lower bits are its rank among them.  Each wave takes
// consecutive choices and has counters of its own in LDS, which become its
// experts' next places once the counts of the waves and workgroups before it,
// and of the experts before each, are added.  So places follow the order of the
// choices, without atomics.  Few choices are one workgroup's; for more, a first
// kernel leaves each workgroup's counts and the second adds up those before it.
//
// 16384 tokens' 4 choices of 64 experts take 9 to 10 us, 32 tokens' 2 choices 3 to 4.
//
// Moves.  Bound by memory traffic: a token's row is read, or written, once for
// all of its choices, and each of their rows once.  A token is some lanes' of a
// workgroup, 16 bytes each at a time.  16384 tokens of 4 choices, 2048 bf16
// features, each repeated in a graph: gather 64 us (5.3 TB/s), its gradient 62, combine
// 62, its gradient 115 (5.2); one after the other, on what the caches hold of the call
// before, 52, 75, 89 and 104.  (A wave for each token: combine 84, its gradient 131.)
#include <algorithm>
#include <type_traits>

#include "layer.h"
#include "linear8_codes.h"

namespace mx {
namespace {

constexpr int kSortWaves = 16, kSortThreads = 64 * kSortWaves;

struct SortParams {
  const int32_t* expert;
  int32_t *offsets, *rows, *order;
  int32_t* counts;  // [groups][experts] of each workgroup
  int n, experts;
  int groups, chunk;  // workgroups, choices of each (a multiple of 64 per wave)
};

// What a wave does with 64 of its choices: f(index, expert or -1, mask of the
// lanes with the same expert).
template <class F>
__device__ __forceinline__ void each_choice(const SortParams& p, int64_t begin, int64_t end, int bits, F&& f) {
  const int lane = threadIdx.x & 63;
  for (int64_t b = begin; b < end; b += 64) {
    const int64_t i = b + lane;
    const int raw = i < end ? p.expert[i] : -1;
    const bool valid = static_cast<uint32_t>(raw) < static_cast<uint32_t>(p.experts);
    uint64_t same = __ballot(valid);
    for (int k = 0; k < bits; ++k) {
      const bool set = raw >> k & 1;
      const uint64_t m = __ballot(set);
      same &= set ? m : ~m;
    }
    f(i, i < end, valid ? raw : -1, same);
  }
}

// Counts the wave's choices by expert in `cnt`.
__device__ __forceinline__ void count_choices(const SortParams& p, int64_t begin, int64_t end, int bits, int* cnt) {
  const int lane = threadIdx.x & 63;
  each_choice(p, begin, end, bits, [&](int64_t, bool, int e, uint64_t same) {
    if (e >= 0 && __builtin_ctzll(same) == lane) cnt[e] += __builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
  });
}

__device__ __forceinline__ void wave_range(const SortParams& p, int64_t& begin, int64_t& end) {
  const int64_t first = static_cast<int64_t>(blockIdx.x) * p.chunk, last = min<int64_t>(first + p.chunk, p.n);
  const int64_t each = p.chunk / kSortWaves;
  begin = min(first + (threadIdx.x >> 6) * each, last);
  end = min(begin + each, last);
}

__device__ __forceinline__ int expert_bits(int experts) { return experts > 1 ? 32 - __builtin_clz(experts - 1) : 0; }

__global__ __launch_bounds__(kSortThreads) void k_route_count(const SortParams p) {
  extern __shared__ int cnt[];
  for (int i = threadIdx.x; i < kSortWaves * p.experts; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int64_t begin, end;
  wave_range(p, begin, end);
  count_choices(p, begin, end, expert_bits(p.experts), cnt + (threadIdx.x >> 6) * p.experts);
  __syncthreads();
  for (int e = threadIdx.x; e < p.experts; e += kSortThreads) {
    int s = 0;
    for (int w = 0; w < kSortWaves; ++w) s += cnt[w * p.experts + e];
    p.counts[static_cast<int64_t>(blockIdx.x) * p.experts + e] = s;
  }
}

// Experts are at most as many as threads: thread e is expert e's.
static_assert(MX_LINEAR_MAX_EXPERTS <= kSortThreads);

__global__ __launch_bounds__(kSortThreads) void k_route_place(const SortParams p) {
  extern __shared__ int cnt[];  // [waves][experts]: counts, then next places
  __shared__ int part[2][kSortThreads], wsum[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6, e = tid;
  int* mine = cnt + wave * p.experts;
  for (int i = tid; i < kSortWaves * p.experts; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  int64_t begin, end;
  wave_range(p, begin, end);
  const int bits = expert_bits(p.experts);
  count_choices(p, begin, end, bits, mine);
  int all = 0, before = 0;  // of expert e, in all workgroups and in those before this one
  if (p.groups > 1) {
    // the threads share the workgroups among them: each takes every q-th one's counts of one expert
    const int span = 1 << bits, q = kSortThreads >> bits, x = tid & (span - 1), k = tid >> bits;
    int a = 0, b = 0;
    if (x < p.experts) {
#pragma unroll 8
      for (int g = k; g < p.groups; g += q) {
        const int v = p.counts[static_cast<int64_t>(g) * p.experts + x];
        a += v;
        b += g < static_cast<int>(blockIdx.x) ? v : 0;
      }
    }
    part[0][tid] = a;
    part[1][tid] = b;
    __syncthreads();
    if (e < p.experts) {
      for (int i = 0; i < q; ++i) {
        all += part[0][i * span + e];
        before += part[1][i * span + e];
      }
    }
  }
  __syncthreads();
  if (p.groups == 1 && e < p.experts)
    for (int w = 0; w < kSortWaves; ++w) all += cnt[w * p.experts + e];
  // places of the experts before e
  const int scan = wave_scan_add(all);
  if ((tid & 63) == 63) wsum[wave] = scan;
  __syncthreads();
  int start = scan - all, total = 0;
  for (int w = 0; w < kSortWaves; ++w) {
    start += w < wave ? wsum[w] : 0;
    total += wsum[w];
  }
  if (e < p.experts) {
    int at = start + before;
    for (int w = 0; w < kSortWaves; ++w) {
      const int v = cnt[w * p.experts + e];
      cnt[w * p.experts + e] = at;
      at += v;
    }
    if (blockIdx.x == 0) p.offsets[e] = start;
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.experts] = total;
  __syncthreads();
  const int lane = tid & 63;
  each_choice(p, begin, end, bits, [&](int64_t i, bool in, int x, uint64_t same) {
    int at = -1;
    if (x >= 0) at = mine[x] + __builtin_popcountll(same & ((uint64_t{1} << lane) - 1));
    __builtin_amdgcn_wave_barrier();
    if (x >= 0 && __builtin_ctzll(same) == lane) mine[x] = at + __builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
    if (in) {
      p.rows[i] = at;
      if (p.order) {
        if (at >= 0) p.order[at] = static_cast<int32_t>(i);
        if (i >= total) p.order[i] = -1;
      }
    }
  });
}

struct MoveParams {
  const void *a, *y;   // the tokens' matrix (or the rows', where it is the one read), and combine_bwd's rows
  void* out;
  int64_t lda, ldy, ldo;
  const int32_t* rows;
  const float* weight;
  float* dweight;
  int tokens, choices, features;
  int lanes;           // of a token, a power of two: log2
  int limit;           // rows of the rows' matrices
};

// Elements of 16 bytes of T, raw.
template <class T>
constexpr int kPiece = 16 / static_cast<int>(sizeof(T));

template <class T>
__global__ __launch_bounds__(256) void k_route_gather(const MoveParams p) {
  constexpr int N = kPiece<T>;
  const int per = 256 >> p.lanes, l = threadIdx.x & ((1 << p.lanes) - 1);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + (threadIdx.x >> p.lanes); t < p.tokens; t += static_cast<int64_t>(gridDim.x) * per) {
    const int32_t* rows = p.rows + t * p.choices;
    const T* x = static_cast<const T*>(p.a) + t * p.lda;
    for (int64_t c = static_cast<int64_t>(l) * N; c < p.features; c += N << p.lanes) {
      const bool whole = c + N <= p.features;
      i32x4 v{};
      if (whole) v = load16(x + c);
      for (int j = 0; j < p.choices; ++j) {
        const int r = rows[j];
        if (static_cast<uint32_t>(r) >= static_cast<uint32_t>(p.limit)) continue;
        T* d = static_cast<T*>(p.out) + r * p.ldo + c;
        if (whole) store16(d, v);
        else
          for (int64_t i = c; i < p.features; ++i) d[i - c] = x[i];
      }
    }
  }
}

// N: choices whose loads are on their way together.
template <class T, bool WEIGHTED, int N>
__global__ __launch_bounds__(256) void k_route_combine(const MoveParams p) {
  const int per = 256 >> p.lanes, l = threadIdx.x & ((1 << p.lanes) - 1);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + (threadIdx.x >> p.lanes); t < p.tokens; t += static_cast<int64_t>(gridDim.x) * per) {
    const int32_t* rows = p.rows + t * p.choices;
    const float* weight = WEIGHTED ? p.weight + t * p.choices : nullptr;
    for (int64_t c = static_cast<int64_t>(l) * 8; c < p.features; c += 8 << p.lanes) {
      float s[8] = {};
      for (int j0 = 0; j0 < p.choices; j0 += N) {
        Raw8<T> raw[N];
        bool has[N];
        float w[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int q = min(j0 + j, p.choices - 1), r = rows[q];
          has[j] = j0 + j < p.choices && static_cast<uint32_t>(r) < static_cast<uint32_t>(p.limit);
          raw[j] = load_raw8(static_cast<const T*>(p.a) + (has[j] ? r : 0) * p.lda, c, has[j] ? p.features : 0);
          w[j] = WEIGHTED ? weight[q] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
          float v[8];
          unpack8(raw[j], v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (has[j]) s[i] += WEIGHTED ? w[j] * v[i] : v[i];
        }
      }
      store_row8(static_cast<T*>(p.out) + t * p.ldo, c, p.features, s);
    }
  }
}

// N: choices whose rows are read, and sums held, together.  GROUP: a token is the
// workgroup's, whose waves join their sums in LDS; else a wave's or less.
template <class T, int N, bool GROUP>
__global__ __launch_bounds__(256) void k_route_combine_bwd(const MoveParams p) {
  __shared__ float part[2][N][4];
  const int lanes = GROUP ? 8 : p.lanes, per = 256 >> lanes, width = 1 << lanes, l = threadIdx.x & (width - 1);
  int turn = 0;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * per + (threadIdx.x >> lanes); t < p.tokens; t += static_cast<int64_t>(gridDim.x) * per) {
    const T* dout = static_cast<const T*>(p.a) + t * p.lda;
    for (int j0 = 0; j0 < p.choices; j0 += N, turn ^= 1) {
      int r[N];
      float w[N], s[N];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const bool in = j0 + j < p.choices;
        r[j] = in ? p.rows[t * p.choices + j0 + j] : -1;
        if (static_cast<uint32_t>(r[j]) >= static_cast<uint32_t>(p.limit)) r[j] = -1;
        w[j] = in ? p.weight[t * p.choices + j0 + j] : 0.0f;
        s[j] = 0.0f;
      }
      for (int64_t c = static_cast<int64_t>(l) * 8; c < p.features; c += 8 << lanes) {
        const Raw8<T> graw = load_raw8(dout, c, p.features);
        Raw8<T> yraw[N];
        if (p.dweight) {
#pragma unroll
          for (int j = 0; j < N; ++j)
            yraw[j] = load_raw8(static_cast<const T*>(p.y) + max(r[j], 0) * p.ldy, c, r[j] < 0 ? 0 : p.features);
        }
        float g[8];
        unpack8(graw, g);
#pragma unroll
        for (int j = 0; j < N; ++j) {
          if (r[j] < 0) continue;
          if (p.dweight) {
            float v[8];
            unpack8(yraw[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) s[j] += g[i] * v[i];
          }
          if (p.out) {
            float d[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] = w[j] * g[i];
            store_row8(static_cast<T*>(p.out) + r[j] * p.ldo, c, p.features, d);
          }
        }
      }
      if (p.dweight) {
#pragma unroll
        for (int j = 0; j < N; ++j)
          for (int d = 1; d < min(width, 64); d *= 2) s[j] += __shfl_xor(s[j], d);
        if constexpr (GROUP) {
          // (the halves of `part` are used in turn: a wave that writes one again
          // has passed the barrier between)
          if ((l & 63) == 0) {
#pragma unroll
            for (int j = 0; j < N; ++j) part[turn][j][l >> 6] = s[j];
          }
          __syncthreads();
          if (l < N && j0 + l < p.choices)
            p.dweight[t * p.choices + j0 + l] = (part[turn][l][0] + part[turn][l][1]) + (part[turn][l][2] + part[turn][l][3]);
        } else {
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (l == 0 && j0 + j < p.choices) p.dweight[t * p.choices + j0 + j] = s[j];
        }
      }
    }
  }
}

// log2 of the lanes of a token: what its row needs, at most `most`.
int lanes_of(int64_t pieces, int most) {
  int l = 3;
  while (l < most && pieces > (int64_t{1} << l)) ++l;
  return l;
}

unsigned move_groups(const MoveParams& p) {
  const int64_t per = 256 >> p.lanes;
  return static_cast<unsigned>(std::min<int64_t>((p.tokens + per - 1) / per, 1 << 20));
}

SortParams make_sort(const mx_route_desc& d) {
  SortParams p{};
  p.n = d.tokens * d.choices;
  p.experts = d.experts;
  // one workgroup for as many as four rounds of its waves; else each has one round, until there are 256 of them
  const int64_t round = kSortThreads;
  p.groups = p.n <= 4 * round ? 1 : static_cast<int>(std::min<int64_t>((p.n + round - 1) / round, 256));
  const int64_t each = (static_cast<int64_t>(p.n) + p.groups - 1) / p.groups;
  p.chunk = static_cast<int>((each + round - 1) / round * round);
  return p;
}

// go(choices that are taken together) as a compile-time constant: registers of
// choices that there are not would leave fewer waves on a CU (16384 tokens of 2
// choices, 4096 features, combine 79 us, 89 with room for 4 and 184 for 8; 8
// choices of 2048 features 120 by fours and 133 by eights)
template <class F>
void by_choices(int choices, F&& go) {
  if (choices == 1) go(std::integral_constant<int, 1>{});
  else if (choices == 2) go(std::integral_constant<int, 2>{});
  else go(std::integral_constant<int, 4>{});
}

template <class F>
void by_type(mx_dtype t, F&& go) {
  if (t == MX_BF16) go(bf16_t{});
  else if (t == MX_F16) go(f16_t{});
  else go(float{});
}

}  // namespace

size_t route_workspace(const mx_route_desc& d) {
  const SortParams p = make_sort(d);
  return p.groups > 1 ? sizeof(int32_t) * static_cast<size_t>(p.groups) * static_cast<size_t>(p.experts) : 0;
}

hipError_t launch_route_sort(const mx_route_desc& d, const int32_t* expert, int32_t* offsets, int32_t* rows, int32_t* order,
                             void* workspace, hipStream_t s) {
  SortParams p = make_sort(d);
  p.expert = expert;
  p.offsets = offsets;
  p.rows = rows;
  p.order = order;
  p.counts = static_cast<int32_t*>(workspace);
  const size_t lds = sizeof(int) * kSortWaves * static_cast<size_t>(p.experts);
  if (p.groups > 1) hipLaunchKernelGGL(k_route_count, dim3(p.groups), dim3(kSortThreads), lds, s, p);
  hipLaunchKernelGGL(k_route_place, dim3(p.groups), dim3(kSortThreads), lds, s, p);
  return hipGetLastError();
}

hipError_t launch_route_gather(const mx_route_desc& d, const void* x, int64_t ldx, const int32_t* rows, void* out, int64_t ldo,
                               mx_dtype dtype, hipStream_t s) {
  if (d.tokens == 0) return hipSuccess;
  MoveParams p{};
  p.a = x;
  p.lda = ldx;
  p.rows = rows;
  p.out = out;
  p.ldo = ldo;
  p.tokens = d.tokens;
  p.choices = d.choices;
  p.features = d.features;
  p.limit = d.tokens * d.choices;
  const int n = dtype == MX_F32 ? 4 : 8;
  p.lanes = lanes_of((static_cast<int64_t>(d.features) + n - 1) / n, 8);
  auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(move_groups(p)), dim3(256), 0, s, p); };
  dtype == MX_F32 ? go(k_route_gather<float>) : go(k_route_gather<bf16_t>);  // (copies: any type of the size will do)
  return hipGetLastError();
}

hipError_t launch_route_combine(const mx_route_desc& d, const void* y, int64_t ldy, const int32_t* rows, const float* weight,
                                void* out, int64_t ldo, mx_dtype dtype, hipStream_t s) {
  if (d.tokens == 0) return hipSuccess;
  MoveParams p{};
  p.a = y;
  p.lda = ldy;
  p.rows = rows;
  p.weight = weight;
  p.out = out;
  p.ldo = ldo;
  p.tokens = d.tokens;
  p.choices = d.choices;
  p.features = d.features;
  p.limit = d.tokens * d.choices;
  p.lanes = lanes_of((static_cast<int64_t>(d.features) + 7) / 8, 8);
  by_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(move_groups(p)), dim3(256), 0, s, p); };
    by_choices(d.choices, [&](auto n) {
      constexpr int N = decltype(n)::value;
      weight ? go(k_route_combine<T, true, N>) : go(k_route_combine<T, false, N>);
    });
  });
  return hipGetLastError();
}

hipError_t launch_route_combine_bwd(const mx_route_desc& d, const void* dout, int64_t ldo, const void* y, int64_t ldy,
                                    const int32_t* rows, const float* weight, void* dy, int64_t lddy, float* dweight,
                                    mx_dtype dtype, hipStream_t s) {
  if (d.tokens == 0) return hipSuccess;
  MoveParams p{};
  p.a = dout;
  p.lda = ldo;
  p.y = y;
  p.ldy = ldy;
  p.rows = rows;
  p.weight = weight;
  p.out = dy;
  p.ldo = lddy;
  p.dweight = dweight;
  p.tokens = d.tokens;
  p.choices = d.choices;
  p.features = d.features;
  p.limit = d.tokens * d.choices;
  // a token is a wave's at most, or the workgroup's
  p.lanes = lanes_of((static_cast<int64_t>(d.features) + 7) / 8, 8);
  if (p.lanes == 7) p.lanes = 8;
  by_type(dtype, [&](auto t) {
    using T = decltype(t);
    auto go = [&](auto kern) { hipLaunchKernelGGL(kern, dim3(move_groups(p)), dim3(256), 0, s, p); };
    by_choices(d.choices, [&](auto n) {
      constexpr int N = decltype(n)::value;
      p.lanes == 8 ? go(k_route_combine_bwd<T, N, true>) : go(k_route_combine_bwd<T, N, false>);
    });
  });
  return hipGetLastError();
}

}  // namespace mx
