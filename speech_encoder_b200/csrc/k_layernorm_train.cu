// LayerNorm for training: the forward pass that keeps each row's mean and
// 1 / sqrt(var + eps), and the backward pass with the affine gradients, both with
// an optional GELU f after the affine map:
//   xh = (x - mean) rstd,  z = xh gamma + beta,  y = f(z)
//   dz = dy f'(z),  w = dz gamma,
//   dx = rstd (w - mean_c(w) - xh mean_c(w xh)) + dres,
//   dgamma = sum_rows dz xh,  dbeta = sum_rows dz
// fp32 throughout; only y and dx are rounded to their types.  Both passes are
// bound by HBM: each row is read once into registers and used from there.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "w2v_internal.h"

namespace w2v {
namespace {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// V consecutive elements as one access of V * sizeof(T) bytes.
template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T v[V];
};

template <typename T, int V>
__device__ __forceinline__ void load_vec(const T* p, float* out) {
  const Vec<T, V> u = *reinterpret_cast<const Vec<T, V>*>(p);
#pragma unroll
  for (int i = 0; i < V; ++i) out[i] = to_f32<T>(u.v[i]);
}

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float* in) {
  Vec<T, V> u;
#pragma unroll
  for (int i = 0; i < V; ++i) u.v[i] = from_f32<T>(in[i]);
  *reinterpret_cast<Vec<T, V>*>(p) = u;
}

// GELU with the accuracy of fp32: the tanh form as z sigmoid(2u),
// u = sqrt(2/pi) (z + 0.044715 z^3).
__device__ __forceinline__ float gelu_value(float z, int act) {
  if (act == 1) return gelu_erf(z);
  const float k = 0.7978845608028654f;
  return z * rcp_approx(1.0f + __expf(-2.0f * z * fmaf(0.044715f * k, z * z, k)));
}

// f'(z): Phi(z) + z phi(z), or s + z s (1 - s) 2 u'(z) with s = sigmoid(2u).
__device__ __forceinline__ float gelu_slope(float z, int act) {
  if (act == 1)
    return fmaf(z * 0.3989422804014327f, __expf(-0.5f * z * z), 0.5f * (1.0f + erff(z * 0.70710678118654752f)));
  const float k = 0.7978845608028654f, z2 = z * z;
  const float s = rcp_approx(1.0f + __expf(-2.0f * z * fmaf(0.044715f * k, z2, k)));
  return fmaf(z * s * (1.0f - s), 2.0f * fmaf(3.0f * 0.044715f * k, z2, k), s);
}

// Sum over the G threads of a row (a warp, or the whole block).
template <int G>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (G == 32) return v;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < G / 32; ++i) s += red[i];
  return s;
}

constexpr int kLnThreads = 256;

// G threads a row, each with NCH chunks of V elements (chunk i at column
// (thread + G i) V).
template <typename X, typename Y, int V, int NCH, int G>
__global__ void __launch_bounds__(kLnThreads)
layernorm_fwd_kernel(const X* __restrict__ x, int64_t x_ld, Y* __restrict__ y, int64_t y_ld, int64_t rows, int cols,
                     const float* __restrict__ gamma, const float* __restrict__ beta, float eps, int act,
                     float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float red[kLnThreads / 32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int lane = threadIdx.x % G;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kLnThreads / G) + threadIdx.x / G;
  pdl_wait();
  if (row >= rows) return;  // whole groups
  const X* xr = x + row * x_ld;
  float v[NCH * V];
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (lane + G * i) * V;
    if (c < cols) {
      load_vec<X, V>(xr + c, v + i * V);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) v[i * V + k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < V; ++k) s += v[i * V + k];
  }
  const float inv = 1.0f / cols;
  const float mean = group_sum<G>(s, red) * inv;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if ((lane + G * i) * V < cols) {
#pragma unroll
      for (int k = 0; k < V; ++k) q += (v[i * V + k] - mean) * (v[i * V + k] - mean);
    }
  }
  const float rstd = 1.0f / sqrtf(group_sum<G>(q, red) * inv + eps);
  if (lane == 0) {
    mean_out[row] = mean;
    rstd_out[row] = rstd;
  }
  Y* yr = y + row * y_ld;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (lane + G * i) * V;
    if (c < cols) {
      float g[V], b[V];
      load_vec<float, V>(gamma + c, g);
      load_vec<float, V>(beta + c, b);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float z = fmaf((v[i * V + k] - mean) * rstd, g[k], b[k]);
        g[k] = act ? gelu_value(z, act) : z;
      }
      store_vec<Y, V>(yr + c, g);
    }
  }
}

// Persistent blocks: each thread keeps its columns' dgamma and dbeta over all
// the rows it sees; the block adds its groups' sums in order and leaves one
// partial per block, which layernorm_affine_kernel adds up in block order.
template <typename X, typename Y, int V, int NCH, int G>
__global__ void __launch_bounds__(kLnThreads)
layernorm_bwd_kernel(const Y* __restrict__ dy, int64_t dy_ld, const X* __restrict__ x, int64_t x_ld, int64_t rows,
                     int cols, const float* __restrict__ gamma, const float* __restrict__ beta,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int act,
                     const X* dres, int64_t dres_ld, X* dx, int64_t dx_ld,
                     float* __restrict__ partial) {
  extern __shared__ float acc[];  // [2][cols] when several groups share the block
  __shared__ float red[kLnThreads / 32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int kGroups = kLnThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  float dg[NCH * V], db[NCH * V];
#pragma unroll
  for (int i = 0; i < NCH * V; ++i) dg[i] = db[i] = 0.f;
  const float inv = 1.0f / cols;
  pdl_wait();
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group; row < rows;
       row += static_cast<int64_t>(gridDim.x) * kGroups) {
    const float m = mean[row], r = rstd[row];
    float xh[NCH * V], w[NCH * V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (lane + G * i) * V;
      if (c < cols) {
        load_vec<X, V>(x + row * x_ld + c, xh + i * V);
        load_vec<Y, V>(dy + row * dy_ld + c, w + i * V);
      }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (lane + G * i) * V;
      if (c < cols) {
        float g[V], b[V];
        load_vec<float, V>(gamma + c, g);
        if (act) load_vec<float, V>(beta + c, b);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int e = i * V + k;
          xh[e] = (xh[e] - m) * r;
          if (act) w[e] *= gelu_slope(fmaf(xh[e], g[k], b[k]), act);
          dg[e] = fmaf(w[e], xh[e], dg[e]);
          db[e] += w[e];
          w[e] *= g[k];
          s1 += w[e];
          s2 = fmaf(w[e], xh[e], s2);
        }
      }
    }
    s1 = group_sum<G>(s1, red) * inv;
    s2 = group_sum<G>(s2, red) * inv;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (lane + G * i) * V;
      if (c < cols) {
        float o[V];
        if (dres) {
          load_vec<X, V>(dres + row * dres_ld + c, o);
        } else {
#pragma unroll
          for (int k = 0; k < V; ++k) o[k] = 0.f;
        }
#pragma unroll
        for (int k = 0; k < V; ++k) o[k] = fmaf(r, w[i * V + k] - s1 - xh[i * V + k] * s2, o[k]);
        store_vec<X, V>(dx + row * dx_ld + c, o);
      }
    }
  }
  float* mine = partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
  for (int turn = 0; turn < kGroups; ++turn) {
    if (group == turn) {
      const bool first = turn == 0, last = turn == kGroups - 1;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const int c = (lane + G * i) * V + k;
          if (c < cols) {
            const float a = dg[i * V + k] + (first ? 0.f : acc[c]), d = db[i * V + k] + (first ? 0.f : acc[cols + c]);
            (last ? mine : acc)[c] = a;
            (last ? mine : acc)[cols + c] = d;
          }
        }
      }
    }
    if (kGroups > 1) __syncthreads();
  }
}

// dgamma and dbeta: the blocks' partials added in a fixed order.  A block takes
// 32 columns of the 2 cols; 8 warps add every eighth partial, then warp 0 the 8.
__global__ void __launch_bounds__(256)
layernorm_affine_kernel(const float* __restrict__ partial, int blocks, int cols, float* __restrict__ dgamma,
                        float* __restrict__ dbeta) {
  __shared__ float red[8][32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c = blockIdx.x * 32 + lane;
  pdl_wait();
  float s = 0.f;
  if (c < 2 * cols)
    for (int i = warp; i < blocks; i += 8) s += partial[static_cast<int64_t>(i) * 2 * cols + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * cols) {
    s = red[0][lane];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += red[i][lane];
    (c < cols ? dgamma + c : dbeta + (c - cols))[0] = s;
  }
}

// Calls fn with the compile-time shape for this row: vector accesses when the
// width, every stride and every pointer allow 16-byte chunks of X (and the same
// number of elements of Y and fp32), single elements otherwise.
template <typename X, int G, typename F>
cudaError_t by_chunks(bool vec, int cols, F&& fn) {
  constexpr int V = 16 / sizeof(X);
  constexpr int kStep = sizeof(X) == 4 ? 2 : 1;  // chunks per thread: 1..4 (16-bit), 2, 4, 6, 8 (fp32)
  if (!vec) return fn(std::integral_constant<int, 1>(), std::integral_constant<int, 32>());
  const int n = (cols + G * V * kStep - 1) / (G * V * kStep);
  std::integral_constant<int, V> v;
  if (n <= 1) return fn(v, std::integral_constant<int, kStep>());
  if (n == 2) return fn(v, std::integral_constant<int, 2 * kStep>());
  if (n == 3) return fn(v, std::integral_constant<int, 3 * kStep>());
  return fn(v, std::integral_constant<int, 4 * kStep>());
}

// Threads a row: one warp up to 1024 columns (32 values a thread), a block of
// 256 above, up to kLnMaxCols.
constexpr int kWarpCols = 1024;

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int bwd_blocks(int64_t rows, int cols) {
  const int per = cols <= kWarpCols ? kLnThreads / 32 : 1;
  const int64_t want = (rows + per - 1) / per;
  return static_cast<int>(want < 2 * kNumSMs ? (want < 1 ? 1 : want) : 2 * kNumSMs);
}

template <typename X, typename Y, int G>
cudaError_t fwd(const LnTrain& s, const void* xp, void* yp, float eps, float* mean, float* rstd, cudaStream_t st) {
  constexpr int V = 16 / sizeof(X);
  const bool vec = s.cols % V == 0 && s.x_ld % V == 0 && s.y_ld % V == 0 && aligned(xp, 16) &&
                   aligned(yp, V * sizeof(Y)) && aligned(s.gamma, 4 * V) && aligned(s.beta, 4 * V);
  const int64_t per = kLnThreads / G;
  const dim3 grid(static_cast<unsigned>((s.rows + per - 1) / per));
  return by_chunks<X, G>(vec, s.cols, [&](auto v, auto nch) {
    return launch_pdl(layernorm_fwd_kernel<X, Y, decltype(v)::value, decltype(nch)::value, G>, grid, dim3(kLnThreads),
                      0, st, static_cast<const X*>(xp), s.x_ld, static_cast<Y*>(yp), s.y_ld, s.rows, s.cols, s.gamma,
                      s.beta, eps, s.act, mean, rstd);
  });
}

struct BwdPtrs {
  const void* dy;
  const void* x;
  const float* mean;
  const float* rstd;
  const void* dres;
  int64_t dres_ld;
  void* dx;
  int64_t dx_ld;
  float* partial;
};

template <typename X, typename Y, int G>
cudaError_t bwd(const LnTrain& s, const BwdPtrs& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(X);
  const bool vec = s.cols % V == 0 && s.x_ld % V == 0 && s.y_ld % V == 0 && p.dx_ld % V == 0 &&
                   (!p.dres || (p.dres_ld % V == 0 && aligned(p.dres, 16))) && aligned(p.x, 16) && aligned(p.dx, 16) &&
                   aligned(p.dy, V * sizeof(Y)) && aligned(s.gamma, 4 * V) && aligned(s.beta, 4 * V);
  const size_t smem = G == 32 ? 2 * static_cast<size_t>(s.cols) * sizeof(float) : 0;
  return by_chunks<X, G>(vec, s.cols, [&](auto v, auto nch) {
    return launch_pdl(layernorm_bwd_kernel<X, Y, decltype(v)::value, decltype(nch)::value, G>,
                      dim3(bwd_blocks(s.rows, s.cols)), dim3(kLnThreads), smem, st, static_cast<const Y*>(p.dy), s.y_ld,
                      static_cast<const X*>(p.x), s.x_ld, s.rows, s.cols, s.gamma, s.beta, p.mean, p.rstd, s.act,
                      static_cast<const X*>(p.dres), p.dres_ld, static_cast<X*>(p.dx), p.dx_ld, p.partial);
  });
}

template <typename F>
cudaError_t by_types(int x_type, int y_type, F&& fn) {
  if (x_type == 0 && y_type == 0) return fn(__half(), __half());
  if (x_type == 1 && y_type == 1) return fn(__nv_bfloat16(), __nv_bfloat16());
  if (x_type == 2 && y_type == 2) return fn(float(), float());
  if (x_type == 2 && y_type == 0) return fn(float(), __half());
  if (x_type == 2 && y_type == 1) return fn(float(), __nv_bfloat16());
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_layernorm_fwd(const LnTrain& s, const void* x, void* y, float eps, float* mean, float* rstd,
                                 cudaStream_t st) {
  if (s.rows == 0) return cudaSuccess;
  return by_types(s.x_type, s.y_type, [&](auto xt, auto yt) {
    using X = decltype(xt);
    using Y = decltype(yt);
    return s.cols <= kWarpCols ? fwd<X, Y, 32>(s, x, y, eps, mean, rstd, st)
                               : fwd<X, Y, kLnThreads>(s, x, y, eps, mean, rstd, st);
  });
}

size_t layernorm_bwd_ws_bytes(int64_t rows, int cols) {
  return static_cast<size_t>(bwd_blocks(rows, cols)) * 2 * cols * sizeof(float);
}

cudaError_t launch_layernorm_bwd(const LnTrain& s, const void* dy, const void* x, const float* mean,
                                 const float* rstd, const void* dres, int64_t dres_ld, void* dx, int64_t dx_ld,
                                 float* dgamma, float* dbeta, void* ws, cudaStream_t st) {
  const BwdPtrs p = {dy, x, mean, rstd, dres, dres_ld, dx, dx_ld, static_cast<float*>(ws)};
  const cudaError_t r = by_types(s.x_type, s.y_type, [&](auto xt, auto yt) {
    using X = decltype(xt);
    using Y = decltype(yt);
    return s.cols <= kWarpCols ? bwd<X, Y, 32>(s, p, st) : bwd<X, Y, kLnThreads>(s, p, st);
  });
  if (r != cudaSuccess) return r;
  return launch_pdl(layernorm_affine_kernel, dim3((2 * s.cols + 31) / 32), dim3(256), 0, st, p.partial,
                    bwd_blocks(s.rows, s.cols), s.cols, dgamma, dbeta);
}

}  // namespace w2v
