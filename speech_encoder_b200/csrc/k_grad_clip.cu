// Global gradient norm over many tensors, and clipping:
//   norm = scale sqrt(sum g^2),  out = g scale min(1, max_norm / (norm + 1e-6)).
// Two passes over the gradients (the factor needs the whole sum), bound by HBM.
// The tensors' table travels in the kernels' parameters, so the calls need no
// copy to the device and may be captured; a list longer than one table is
// walked by several launches.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "w2v_internal.h"

namespace w2v {
namespace {

constexpr int kClipThreads = 256;
constexpr int kChunk = 8192;        // elements of one tensor that a block takes at a time
constexpr int kTable = 512;         // tensors per launch
constexpr int kBlocks = 4 * kNumSMs;  // of 256 threads, resident at once

struct ClipTable {
  const void* src[kTable];
  void* dst[kTable];
  int64_t n[kTable];
  int first[kTable + 1];            // first chunk of each tensor, total at the end
  uint8_t type[kTable];
  int count;
};

// The tensor that holds `chunk`: the last one whose first chunk is not above it.
__device__ __forceinline__ int find_tensor(const ClipTable& t, int chunk) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

template <typename T>
struct Elem;
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float get(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half put(float v) { return __float2half_rn(v); }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 put(float v) { return __float2bfloat16_rn(v); }
};

template <typename T>
struct alignas(16) Vec16 {
  T v[16 / sizeof(T)];
};

// Elements [from, to) of chunk c: chunks start on 16-byte boundaries of src, the
// first one also takes the elements before its boundary.
template <typename T>
__device__ __forceinline__ void chunk_range(const T* src, int64_t n, int c, int64_t* head, int64_t* from, int64_t* to) {
  int64_t hd = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(src) & 15)) & 15) / sizeof(T);
  if (hd > n) hd = n;
  *head = hd;
  *from = hd + static_cast<int64_t>(c) * kChunk;
  const int64_t end = *from + kChunk;
  *to = end < n ? end : n;
}

// A whole chunk's 16-byte vectors per thread: all loaded before any is used.
template <typename T>
constexpr int kVecs = kChunk * static_cast<int>(sizeof(T)) / 16 / kClipThreads;

template <typename T>
__device__ __forceinline__ double square(T v) {
  const double x = Elem<T>::get(v);
  return x * x;
}

// Squares of one thread's part of a chunk.  32 of them are added in fp32 where that
// is safe: a sum between 1e-20 and 1e37 has no overflowed square, and squares lost
// below fp32's range (each below 1e-38) do not show in it.  Otherwise, and across
// parts, in fp64 (all in fp64 took 257 us for 1.2 GB, bound by its conversions).
template <typename T>
__device__ __forceinline__ double chunk_squares(const void* srcv, int64_t n, int c) {
  constexpr int V = 16 / sizeof(T);
  const T* src = static_cast<const T*>(srcv);
  int64_t head, from, to;
  chunk_range<T>(src, n, c, &head, &from, &to);
  double s = 0.0;
  if (c == 0 && threadIdx.x < head) s = square<T>(src[threadIdx.x]);
  if (to <= from) return s;
  const int vecs = static_cast<int>(to - from) / V;
  const Vec16<T>* p = reinterpret_cast<const Vec16<T>*>(src + from);
  Vec16<T> u[kVecs<T>];
#pragma unroll
  for (int i = 0; i < kVecs<T>; ++i) {
    const int at = threadIdx.x + i * kClipThreads;
    if (at < vecs) {
      u[i] = p[at];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) u[i].v[k] = Elem<T>::put(0.f);
    }
  }
  float q[V];
#pragma unroll
  for (int k = 0; k < V; ++k) q[k] = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs<T>; ++i) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const float x = Elem<T>::get(u[i].v[k]);
      q[k] = fmaf(x, x, q[k]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) sum += q[k];
  if (sum > 1e-20f && sum < 1e37f) {
    s += sum;
  } else {
#pragma unroll
    for (int i = 0; i < kVecs<T>; ++i) {
#pragma unroll
      for (int k = 0; k < V; ++k) s += square<T>(u[i].v[k]);
    }
  }
  const int64_t at = from + static_cast<int64_t>(vecs) * V + threadIdx.x;
  if (at < to) s += square<T>(src[at]);
  return s;
}

// out = g f lift; lift is 1, or the power of two that keeps f out of fp32's subnormals.
template <typename T>
__device__ __forceinline__ void chunk_scale(const void* srcv, void* dstv, int64_t n, int c, float f, float lift) {
  constexpr int V = 16 / sizeof(T);
  const T* src = static_cast<const T*>(srcv);
  T* dst = static_cast<T*>(dstv);
  int64_t head, from, to;
  chunk_range<T>(src, n, c, &head, &from, &to);
  if (c == 0 && threadIdx.x < head) dst[threadIdx.x] = Elem<T>::put(Elem<T>::get(src[threadIdx.x]) * f * lift);
  if (to <= from) return;
  const int vecs = static_cast<int>(to - from) / V;
  const bool same = ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst)) & 15) == 0;
  const Vec16<T>* p = reinterpret_cast<const Vec16<T>*>(src + from);
  Vec16<T> u[kVecs<T>];
#pragma unroll
  for (int i = 0; i < kVecs<T>; ++i) {
    const int at = threadIdx.x + i * kClipThreads;
    if (at < vecs) u[i] = p[at];
  }
#pragma unroll
  for (int i = 0; i < kVecs<T>; ++i) {
    const int at = threadIdx.x + i * kClipThreads;
    if (at >= vecs) break;
#pragma unroll
    for (int k = 0; k < V; ++k) u[i].v[k] = Elem<T>::put(Elem<T>::get(u[i].v[k]) * f * lift);
    if (same) {
      reinterpret_cast<Vec16<T>*>(dst + from)[at] = u[i];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) dst[from + static_cast<int64_t>(at) * V + k] = u[i].v[k];
    }
  }
  const int64_t at = from + static_cast<int64_t>(vecs) * V + threadIdx.x;
  if (at < to) dst[at] = Elem<T>::put(Elem<T>::get(src[at]) * f * lift);
}

// Sum over the block, the same in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double s) {
  __shared__ double red[kClipThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = red[0];
#pragma unroll
  for (int i = 1; i < kClipThreads / 32; ++i) s += red[i];
  return s;
}

// The sum is fp64: squares of fp32 and bf16 values leave fp32's range from 1.8e19
// and below 1e-23, and there may be 10^9 of them.
__global__ void __launch_bounds__(kClipThreads)
grad_squares_kernel(const __grid_constant__ ClipTable t, double* __restrict__ partial) {
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  double s = 0.0;
  for (int c = blockIdx.x; c < t.first[t.count]; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const int k = c - t.first[i];
    if (t.type[i] == 2)
      s += chunk_squares<float>(t.src[i], t.n[i], k);
    else if (t.type[i] == 1)
      s += chunk_squares<__nv_bfloat16>(t.src[i], t.n[i], k);
    else
      s += chunk_squares<__half>(t.src[i], t.n[i], k);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

__global__ void __launch_bounds__(kClipThreads)
grad_scale_kernel(const __grid_constant__ ClipTable t, const double* __restrict__ partial, int partials, float scale,
                  float max_norm, float* __restrict__ norm_out) {
  if (threadIdx.x == 0) pdl_launch_dependents();
  pdl_wait();
  double s = 0.0;
  for (int i = threadIdx.x; i < partials; i += kClipThreads) s += partial[i];
  const double norm = sqrt(block_sum(s)) * fabs(static_cast<double>(scale));
  const float written = static_cast<float>(norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm_out = written;
  double by = static_cast<double>(max_norm) / (norm + 1e-6);
  if (!(by < 1.0) || !(written < INFINITY)) by = 1.0;  // not clipped, or no finite norm for the caller to read
  by *= static_cast<double>(scale);
  // A factor below 2^-126 (a norm near fp32's end) would keep but a few bits as an fp32.
  const float lift = by < 0x1p-126 ? 0x1p-126f : 1.0f;
  const float f = static_cast<float>(by / static_cast<double>(lift));
  // from the end, where the first pass has just been: what it left in L2 is not
  // read from memory again
  for (int c = t.first[t.count] - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= static_cast<int>(gridDim.x)) {
    const int i = find_tensor(t, c);
    const int k = c - t.first[i];
    if (f == 1.0f && lift == 1.0f && t.src[i] == t.dst[i]) continue;  // in place and unchanged
    if (t.type[i] == 2)
      chunk_scale<float>(t.src[i], t.dst[i], t.n[i], k, f, lift);
    else if (t.type[i] == 1)
      chunk_scale<__nv_bfloat16>(t.src[i], t.dst[i], t.n[i], k, f, lift);
    else
      chunk_scale<__half>(t.src[i], t.dst[i], t.n[i], k, f, lift);
  }
}

}  // namespace

size_t grad_clip_ws_bytes(int n) {
  const size_t tables = n <= kTable ? 1 : (static_cast<size_t>(n) + kTable - 1) / kTable;
  return tables * kBlocks * sizeof(double);
}

cudaError_t launch_grad_clip(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                             const int* types, float scale, float max_norm, float* norm, void* ws, cudaStream_t st) {
  double* partial = static_cast<double*>(ws);
  const int tables = n <= kTable ? 1 : (n + kTable - 1) / kTable;
  ClipTable t;
  auto fill = [&](int k) {
    const int base = k * kTable;
    t.count = n - base < kTable ? n - base : kTable;
    int chunks = 0;
    for (int i = 0; i < t.count; ++i) {
      t.src[i] = grads[base + i];
      t.dst[i] = outs[base + i];
      t.n[i] = counts[base + i];
      t.type[i] = static_cast<uint8_t>(types[base + i]);
      t.first[i] = chunks;
      // chunks of the elements after those before the first 16-byte boundary
      // (an upper bound on them: all; a chunk past the end does nothing)
      chunks += static_cast<int>((t.n[i] + kChunk - 1) / kChunk);
    }
    t.first[t.count] = chunks;
    if (t.count == 0) {
      t.count = 1;
      t.first[1] = 0;
    }
    return chunks;
  };
  for (int k = 0; k < tables; ++k) {
    fill(k);
    const cudaError_t r = launch_pdl(grad_squares_kernel, dim3(kBlocks), dim3(kClipThreads), 0, st, t,
                                     partial + static_cast<int64_t>(k) * kBlocks);
    if (r != cudaSuccess) return r;
  }
  for (int k = tables - 1; k >= 0; --k) {
    if (tables > 1) fill(k);
    const cudaError_t r = launch_pdl(grad_scale_kernel, dim3(kBlocks), dim3(kClipThreads), 0, st, t,
                                     static_cast<const double*>(partial), tables * kBlocks, scale, max_norm, norm);
    if (r != cudaSuccess) return r;
  }
  return cudaSuccess;
}

}  // namespace w2v
