// Global norm over many gradients and clipping by it (mxlinear.h).
//
// Two launches for up to kTensors tensors (each further kTensors add two):
//   k_grad_sum   reads every gradient once; a workgroup sums the squares of
//                its chunks and leaves one fp64 partial
//   k_grad_clip  every workgroup adds all partials in the same order (up to 8
//                KiB from L2 for each kTensors tensors), so all of them hold the
//                same norm without a launch between, then scales its chunks
// Bound by memory: two reads and one write; 818 MB of gradients in 240 tensors
// that start anywhere take 574 us (4.3 TB/s; the norm alone 150 us, 5.5 TB/s).
// The partials' reads grow with the square of the tensors' number: 24 KiB for
// each workgroup of three launches there, 0.9 MB in 105 launches for ten thousand
// large tensors.  Sums are fp64: the squares of any finite fp32 fit, and the
// adds are far below the vector units' rate.
//
// The tensors' addresses and sizes travel in the kernel's arguments, so no
// table has to be copied to the device.  Work is dealt in chunks over all
// tensors; a workgroup takes every gridDim.x-th chunk.  Chunks are of 8192
// elements, or of 2048 where that leaves CUs idle.
#include "internal.h"
#include "linear.h"

namespace mx {
namespace {

constexpr int kTensors = 96;       // per launch: the arguments stay below 4 KiB
constexpr int kThreads = 256;
constexpr int kChunk = 8192, kSmallChunk = 2048;  // elements
constexpr int kMaxGroups = 1024;   // workgroups, and partials, per launch

struct Batch {
  const void* grad[kTensors];
  void* out[kTensors];
  int64_t numel[kTensors];
  int32_t first[kTensors + 1];  // first chunk of each tensor
  uint8_t dtype[kTensors];
  int32_t count;
  int32_t chunk;   // elements of a chunk
  int32_t stream;  // whether the outputs pass the last-level cache
};

template <class T> struct Pack { static constexpr int N = 16 / sizeof(T); };

template <class T>
__device__ __forceinline__ void unpack(uint4 v, float* x) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < Pack<T>::N; ++i) x[i] = to_f32(e[i]);
}

// the tensor of chunk c: the last one that starts at it or before.  Every lane
// compares two of them.
__device__ __forceinline__ int tensor_of(const Batch& b, int c) {
  static_assert(kTensors <= 128);
  const int lane = threadIdx.x & 63;
  const uint64_t lo = __ballot(lane < b.count && b.first[min(lane, kTensors)] <= c);
  const uint64_t hi = __ballot(lane + 64 < b.count && b.first[min(lane + 64, kTensors)] <= c);
  return __popcll(lo) + __popcll(hi) - 1;
}

// Elements before the first multiple of 16 bytes (n at most).  Gradients that
// are parts of a bucket start anywhere, so this is the usual case.
template <class T>
__device__ __forceinline__ int64_t head_of(const T* g, int64_t n) {
  const int64_t h = static_cast<int64_t>((0 - reinterpret_cast<uintptr_t>(g)) % 16 / sizeof(T));
  return h < n ? h : n;
}

template <class T>
__device__ __forceinline__ double sum_chunk(const T* __restrict__ g, int64_t n) {
  constexpr int N = Pack<T>::N;
  double s = 0.0;
  auto add = [&](float v) { s = __builtin_fma(static_cast<double>(v), static_cast<double>(v), s); };
  const int64_t head = head_of(g, n), packs = (n - head) / N;
  const uint4* v = reinterpret_cast<const uint4*>(g + head);
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < packs; i += kThreads) {
    float x[N];
    unpack<T>(v[i], x);
#pragma unroll
    for (int j = 0; j < N; ++j) add(x[j]);
  }
  // fewer than N elements before and after
  const int64_t t = head + packs * N + threadIdx.x;
  if (threadIdx.x < head) add(to_f32(g[threadIdx.x]));
  if (t < n) add(to_f32(g[t]));
  return s;
}

template <class T>
__device__ __forceinline__ void scale_chunk(const T* g, T* o, int64_t n, float f, bool stream) {
  constexpr int N = Pack<T>::N;
  if ((reinterpret_cast<uintptr_t>(g) - reinterpret_cast<uintptr_t>(o)) % 16 != 0) {
    for (int64_t i = threadIdx.x; i < n; i += kThreads) o[i] = from_f32<T>(to_f32(g[i]) * f);
    return;
  }
  const int64_t head = head_of(g, n), packs = (n - head) / N;
  const uint4* v = reinterpret_cast<const uint4*>(g + head);
  uint4* w = reinterpret_cast<uint4*>(o + head);
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < packs; i += kThreads) {
    float x[N];
    unpack<T>(v[i], x);
    uint4 q;
    T* e = reinterpret_cast<T*>(&q);
#pragma unroll
    for (int j = 0; j < N; ++j) e[j] = from_f32<T>(x[j] * f);
    if (stream) stream16(w + i, __builtin_bit_cast(i32x4, q));
    else w[i] = q;
  }
  const int64_t t = head + packs * N + threadIdx.x;
  if (threadIdx.x < head) o[threadIdx.x] = from_f32<T>(to_f32(g[threadIdx.x]) * f);
  if (t < n) o[t] = from_f32<T>(to_f32(g[t]) * f);
}

// Sum over the workgroup, the same in every thread, in a fixed order.
__device__ __forceinline__ double group_sum(double s) {
  __shared__ double part[kThreads / 64];
#pragma unroll
  for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = 0.0;
#pragma unroll
  for (int i = 0; i < kThreads / 64; ++i) s += part[i];
  __syncthreads();
  return s;
}

__global__ __launch_bounds__(kThreads) void k_grad_sum(const Batch b, double* __restrict__ partial) {
  double s = 0.0;
  for (int c = blockIdx.x; c < b.first[b.count]; c += gridDim.x) {
    const int t = tensor_of(b, c);
    const int64_t at = static_cast<int64_t>(c - b.first[t]) * b.chunk;
    const int64_t n = min(static_cast<int64_t>(b.chunk), b.numel[t] - at);
    if (b.dtype[t] == MX_BF16) s += sum_chunk(static_cast<const bf16_t*>(b.grad[t]) + at, n);
    else if (b.dtype[t] == MX_F16) s += sum_chunk(static_cast<const f16_t*>(b.grad[t]) + at, n);
    else s += sum_chunk(static_cast<const float*>(b.grad[t]) + at, n);
  }
  s = group_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// write: this launch's first workgroup stores the norm
__global__ __launch_bounds__(kThreads) void k_grad_clip(const Batch b, const double* __restrict__ partial, int partials,
                                                         float max_norm, float* __restrict__ norm, int write) {
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kThreads) s += partial[i];
  s = group_sum(s);
  const float nrm = static_cast<float>(__builtin_sqrt(s));
  if (write && blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  if (b.count == 0) return;
  const float q = max_norm / (nrm + 1e-6f);
  const float f = q < 1.0f || q != q ? q : 1.0f;
  for (int c = blockIdx.x; c < b.first[b.count]; c += gridDim.x) {
    const int t = tensor_of(b, c);
    if (f == 1.0f && b.grad[t] == b.out[t]) continue;
    const int64_t at = static_cast<int64_t>(c - b.first[t]) * b.chunk;
    const int64_t n = min(static_cast<int64_t>(b.chunk), b.numel[t] - at);
    if (b.dtype[t] == MX_BF16) scale_chunk(static_cast<const bf16_t*>(b.grad[t]) + at, static_cast<bf16_t*>(b.out[t]) + at, n, f, b.stream != 0);
    else if (b.dtype[t] == MX_F16) scale_chunk(static_cast<const f16_t*>(b.grad[t]) + at, static_cast<f16_t*>(b.out[t]) + at, n, f, b.stream != 0);
    else scale_chunk(static_cast<const float*>(b.grad[t]) + at, static_cast<float*>(b.out[t]) + at, n, f, b.stream != 0);
  }
}

// The next batch of non-empty tensors from i on.  The caller has checked that
// all chunks together fit an int32.
void fill(const mx_grad_list* l, int& i, Batch& b, int chunk, bool stream = false) {
  b.chunk = chunk;
  b.stream = stream ? 1 : 0;
  b.count = 0;
  int64_t chunks = 0;
  for (; i < l->count && b.count < kTensors; ++i) {
    if (l->numel[i] <= 0) continue;
    const int64_t more = (l->numel[i] + chunk - 1) / chunk;
    b.grad[b.count] = l->grads[i];
    b.out[b.count] = l->out ? l->out[i] : nullptr;
    b.numel[b.count] = l->numel[i];
    b.dtype[b.count] = static_cast<uint8_t>(l->dtypes[i]);
    b.first[b.count] = static_cast<int32_t>(chunks);
    chunks += more;
    b.first[++b.count] = static_cast<int32_t>(chunks);
  }
}

unsigned groups(const Batch& b) {
  const int c = b.first[b.count];
  return static_cast<unsigned>(c < kMaxGroups ? c : kMaxGroups);
}

}  // namespace

size_t grad_workspace_bytes(int32_t count) {
  return (static_cast<size_t>(count) + kTensors - 1) / kTensors * kMaxGroups * sizeof(double);
}

hipError_t launch_grad_clip(const mx_grad_list* l, bool clip, float max_norm, float* norm, void* workspace, hipStream_t s) {
  double* partial = static_cast<double*>(workspace);
  int partials = 0;
  static_assert(sizeof(Batch) + 64 <= 4096);
  int64_t total = 0;
  for (int i = 0; i < l->count; ++i) total += l->numel[i];
  const int chunk = total < static_cast<int64_t>(kChunk) * kMaxGroups ? kSmallChunk : kChunk;
  Batch b;
  for (int i = 0; i < l->count;) {
    fill(l, i, b, chunk);
    if (b.count == 0) break;
    const unsigned wgs = groups(b);
    hipLaunchKernelGGL(k_grad_sum, dim3(wgs), dim3(kThreads), 0, s, b, partial + partials);
    partials += static_cast<int>(wgs);
  }
  bool first = true;
  // outputs that the last-level cache cannot hold are written past it: 250M
  // values take 572 us instead of 602
  size_t bytes = 0;
  for (int i = 0; i < l->count; ++i) bytes += static_cast<size_t>(l->numel[i]) * (l->dtypes[i] == MX_F32 ? 4 : 2);
  for (int i = 0; clip && i < l->count;) {
    fill(l, i, b, chunk, bytes > kStreamOutBytes);
    if (b.count == 0) break;
    hipLaunchKernelGGL(k_grad_clip, dim3(groups(b)), dim3(kThreads), 0, s, b, partial, partials, max_norm, norm, first ? 1 : 0);
    first = false;
  }
  if (first) {
    b.count = 0;
    hipLaunchKernelGGL(k_grad_clip, dim3(1), dim3(kThreads), 0, s, b, partial, partials, max_norm, norm, 1);
  }
  return hipGetLastError();
}

}  // namespace mx
