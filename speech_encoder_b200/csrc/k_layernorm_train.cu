// LayerNorm for training: the forward pass that keeps each row's mean and
// 1 / sqrt(var + eps), and the backward pass with the affine gradients, both with
// an optional GELU f after the affine map:
//   xh = (x - mean) rstd,  z = xh gamma + beta,  y = f(z)
//   dz = dy f'(z),  w = dz gamma,
//   dx = rstd (w - mean_c(w) - xh mean_c(w xh)) + dres,
//   dgamma = sum_rows dz xh,  dbeta = sum_rows dz
// fp32 throughout; only y and dx are rounded to their types.  Each row is read
// once and used from registers; without a GELU the passes come within 1.2 to 1.5 of
// the time that HBM needs, with one instruction issue bounds them (51199 x 512 fp16:
// forward 20 us and 25 with the exact GELU against 16, backward 36 and 47 against 24).
#include <cuda_bf16.h>

#include <algorithm>

#include "ptx.cuh"
#include "w2v_internal.h"

namespace w2v {
namespace {

constexpr int kLnThreads = 256;

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

// A thread's elements of a row: NCH chunks of V, chunk i at column (lane + G i) V;
// columns past the end read as zero and are not written.
template <typename T, int V, int NCH, int G>
__device__ __forceinline__ void load_row(const T* p, int lane, int cols, Vec<T, V> (&u)[NCH]) {
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (lane + G * i) * V;
    if (c < cols) {
      u[i] = *reinterpret_cast<const Vec<T, V>*>(p + c);
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) u[i].v[k] = from_f32<T>(0.f);
    }
  }
}

template <typename T, int V, int NCH>
__device__ __forceinline__ void widen(const Vec<T, V> (&u)[NCH], float2 (&out)[NCH * V / 2]) {
#pragma unroll
  for (int e = 0; e < NCH * V; e += 2)
    out[e / 2] = make_float2(to_f32<T>(u[e / V].v[e % V]), to_f32<T>(u[(e + 1) / V].v[(e + 1) % V]));
}

template <typename T, int V, int NCH, int G>
__device__ __forceinline__ void store_row(T* p, int lane, int cols, const float2 (&in)[NCH * V / 2]) {
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (lane + G * i) * V;
    if (c < cols) {
      Vec<T, V> u;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int e = i * V + k;
        u.v[k] = from_f32<T>(e & 1 ? in[e / 2].y : in[e / 2].x);
      }
      *reinterpret_cast<Vec<T, V>*>(p + c) = u;
    }
  }
}

// Elements e .. e + 3 of a thread's part of a vector over the columns.
template <int V, int G>
__device__ __forceinline__ float4 load4(const float* p, int lane, int cols, int e) {
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (V >= 4) {
    const int c = (lane + G * (e / V)) * V;
    if (c < cols) r = *reinterpret_cast<const float4*>(p + c + e % V);
  } else {
    if (lane + G * e < cols) r.x = p[lane + G * e];
    if (lane + G * (e + 1) < cols) r.y = p[lane + G * (e + 1)];
    if (lane + G * (e + 2) < cols) r.z = p[lane + G * (e + 2)];
    if (lane + G * (e + 3) < cols) r.w = p[lane + G * (e + 3)];
  }
  return r;
}

// Asynchronous copy of one chunk to this thread's own place in shared memory, and
// the wait for all but the newest N rows of them: no other thread is involved.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if (BYTES < 8) return;  // (rows of single elements are not copied this way)
  if (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// This thread's chunks of a row from its place in a stage, kLnThreads chunks apart.
template <typename T, int V, int NCH, int G>
__device__ __forceinline__ void read_ring(const Vec<T, V>* slot, int lane, int cols, float2 (&out)[NCH * V / 2]) {
  Vec<T, V> u[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    if ((lane + G * i) * V < cols) {
      u[i] = slot[i * kLnThreads];
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) u[i].v[k] = from_f32<T>(0.f);
    }
  }
  widen<T, V, NCH>(u, out);
}

__device__ __forceinline__ float ld_dsmem(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A constant for both elements of a pair, held in registers: a packed instruction
// takes no immediates, and left to itself the compiler moves each constant into a
// pair of registers before each use.
__device__ __forceinline__ float2 held(float v) {
  float2 r;
  asm("mov.f32 %0, %2;\n\tmov.f32 %1, %2;" : "=f"(r.x), "=f"(r.y) : "f"(v));
  return r;
}

// GELU f and its slope f' on pairs of elements in packed fp32 instructions (with
// scalar ones both passes over 51199 x 512 were bound by instruction issue).  WIDE:
// for results that stay fp32.
template <int ACT, bool WIDE>
struct Gelu {
  __device__ __forceinline__ float2 value(float2 z) const { return z; }
  __device__ __forceinline__ float2 slope(float2) const { return both(1.0f); }
};

// Phi(-|z|) of the exact form, and e = exp(-z^2 / 2): they share one exponential, as
// Phi(-|z|) = e g(t) with t = 1 / (1 + p |z|) and g a polynomial without a constant.
// Coefficients by linear programming over a grid of z in [0, 13] or [0, 14], p by search.
template <bool WIDE>
struct NormalTail;

// Results of 16 bits: degree 6, the smallest largest excess over absolute and relative
// bounds of 1 : 1000 (6.4e-8 and 6.4e-5).  Measured over [-13, 13]: the slope within
// 2.5e-7, and f, rounded, within 1.16 half steps of fp16 and 1.03 of bf16 (2.9 and 18
// with a polynomial of degree 5 for the absolute error alone).
template <>
struct NormalTail<false> {
  static constexpr float p = 0.2925f;
  float2 a = held(-0.5f * 1.4426950408889634f);
  float2 c6 = held(-0.08600358808141047f), c5 = held(0.26645464523659707f), c4 = held(-0.07094969882740387f);
  float2 c3 = held(0.16799627886898685f), c2 = held(0.10494842715972288f), c1 = held(0.11755387193946223f);
  __device__ __forceinline__ float2 g(float2 t) const {
    return ffma2(ffma2(ffma2(ffma2(ffma2(t, c6, c5), t, c4), t, c3), t, c2), t, c1);
  }
};

// Results of fp32: degree 8, the smallest largest relative error (6.6e-8), so a few
// roundings of fp32 at every z, and z^2 2^-23 of the exponent's.  Measured: Phi within
// 2.2e-7, f within 1.5e-6 of its own value down to z = -5, the slope within 2.3e-7.
// Packed like the other; fp32 rows wait for memory and hardly show it (25600 x 512
// forward 18.7 us for either degree, backward 33.2 for 33.0).
template <>
struct NormalTail<true> {
  static constexpr float p = 0.305f;
  float2 a = held(-0.5f * 1.4426950408889634f);
  float2 c8 = held(0.03663970305112069f), c7 = held(-0.15273976910813133f), c6 = held(0.1853005931000754f);
  float2 c5 = held(-0.03761743553585788f), c4 = held(0.12085047515807737f), c3 = held(0.10346547345964746f);
  float2 c2 = held(0.12246101027285013f), c1 = held(0.12164002060621362f);
  __device__ __forceinline__ float2 g(float2 t) const {
    const float2 high = ffma2(ffma2(ffma2(ffma2(t, c8, c7), t, c6), t, c5), t, c4);
    return ffma2(ffma2(ffma2(high, t, c3), t, c2), t, c1);
  }
};

// Exact form; h = Phi(-|z|).
template <bool WIDE>
struct Gelu<1, WIDE> : NormalTail<WIDE> {
  __device__ __forceinline__ float2 tail(float2 z, float2* e) const {
    constexpr float p = NormalTail<WIDE>::p;
    const float2 t = make_float2(rcp_approx(fmaf(fabsf(z.x), p, 1.0f)), rcp_approx(fmaf(fabsf(z.y), p, 1.0f)));
    const float2 w = fmul2(fmul2(z, this->a), z);
    *e = make_float2(ex2_approx(w.x), ex2_approx(w.y));
    return fmul2(this->g(t), fmul2(t, *e));
  }
  // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
  __device__ __forceinline__ float2 value(float2 z) const {
    float2 e;
    const float2 h = tail(z, &e);
    return make_float2(fmaf(-fabsf(z.x), h.x, fmaxf(z.x, 0.f)), fmaf(-fabsf(z.y), h.y, fmaxf(z.y, 0.f)));
  }
  // Phi(z) + z phi(z)
  __device__ __forceinline__ float2 slope(float2 z) const {
    float2 e;
    const float2 h = tail(z, &e);
    const float2 ze = fmul2(z, e);
    return make_float2(fmaf(0.3989422804014327f, ze.x, z.x < 0.f ? h.x : 1.0f - h.x),
                       fmaf(0.3989422804014327f, ze.y, z.y < 0.f ? h.y : 1.0f - h.y));
  }
};

// Tanh form: z s with s = sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3).
template <bool WIDE>
struct Gelu<2, WIDE> {
  static constexpr float k = 0.7978845608028654f, kl = -2.0f * k * 1.4426950408889634f;
  float2 one = held(1.0f), k1 = held(kl), k3 = held(0.044715f * kl);
  __device__ __forceinline__ float2 gate(float2 z, float2 z2) const {
    const float2 w = fmul2(z, ffma2(z2, k3, k1));
    const float2 d = fadd2(make_float2(ex2_approx(w.x), ex2_approx(w.y)), one);
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
  }
  __device__ __forceinline__ float2 value(float2 z) const { return fmul2(z, gate(z, fmul2(z, z))); }
  // s + z s (1 - s) 2 u'(z)
  __device__ __forceinline__ float2 slope(float2 z) const {
    const float2 z2 = fmul2(z, z), s = gate(z, z2);
    const float2 zs = fmul2(z, s);
    return make_float2(fmaf(fmaf(-zs.x, s.x, zs.x), fmaf(6.0f * 0.044715f * k, z2.x, 2.0f * k), s.x),
                       fmaf(fmaf(-zs.y, s.y, zs.y), fmaf(6.0f * 0.044715f * k, z2.y, 2.0f * k), s.y));
  }
};

// fn(std::integral_constant<int, act>()), so that the choice is made once a row.
template <typename F>
__device__ __forceinline__ void by_act(int act, F&& fn) {
  if (act == 0)
    fn(std::integral_constant<int, 0>());
  else if (act == 1)
    fn(std::integral_constant<int, 1>());
  else
    fn(std::integral_constant<int, 2>());
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

// Chunks a thread is given at a time: its 1 to 4 steps cover a row with at most the
// last step's chunks past the end.
template <typename X>
__host__ __device__ constexpr int chunk_step() {
  return sizeof(X) == 4 ? 2 : 1;
}

// G threads a row, each with NCH chunks of V elements; a group takes ROWS rows at
// once (two where there are rows enough: a warp with one 1 KB row in flight reaches
// 4.4 TB/s of the 6.5).  Blocks an SM, where the compiler's own choice of registers is
// the worse one: two rows fit four blocks (with three 51199 x 512 fp16 takes 22 us for
// 20), and fp32 rows of 513 to 768 columns are faster with the registers of three, gamma
// and beta on their way early (7992 x 768 fp32 10.0 us for 10.8; 0 leaves it the choice).
template <typename X, int V, int NCH, int G, int ROWS>
constexpr int kFwdBlocks = ROWS == 2 ? 4 : sizeof(X) == 4 && V == 4 && NCH == 6 && G == 32 ? 3 : 0;

template <typename X, typename Y, int V, int NCH, int G, int ROWS>
__global__ void __launch_bounds__(kLnThreads, kFwdBlocks<X, V, NCH, G, ROWS>)
layernorm_fwd_kernel(const X* __restrict__ x, int64_t x_ld, Y* __restrict__ y, int64_t y_ld, int64_t rows, int cols,
                     const float* __restrict__ gamma, const float* __restrict__ beta, float eps, int act,
                     float* __restrict__ mean_out, float* __restrict__ rstd_out) {
  __shared__ float red[kLnThreads / 32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int NP = NCH * V / 2;
  const int lane = threadIdx.x % G;
  const int64_t row = (static_cast<int64_t>(blockIdx.x) * (kLnThreads / G) + threadIdx.x / G) * ROWS;
  pdl_wait();
  if (row >= rows) return;  // whole groups
  const int here = ROWS == 1 || row + 1 < rows ? ROWS : 1;
  float2 v[ROWS][NP];
  float mean[ROWS], rstd[ROWS];
  {
    Vec<X, V> raw[ROWS][NCH];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)  // (past the last row: the last row again, not written)
      load_row<X, V, NCH, G>(x + (row + min(k, here - 1)) * x_ld, lane, cols, raw[k]);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) widen<X, V, NCH>(raw[k], v[k]);
  }
  const float inv = 1.0f / cols;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    float2 s = v[k][0];
#pragma unroll
    for (int i = 1; i < NP; ++i) s = fadd2(s, v[k][i]);
    mean[k] = s.x + s.y;
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) mean[k] = group_sum<G>(mean[k], red) * inv;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    float2 q = both(0.f);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      v[k][i] = fadd2(v[k][i], both(-mean[k]));
      // columns past the end, which can only be in the last chunks (see by_chunks)
      const int e = 2 * i;
      if (V == 1 || e / V >= NCH - chunk_step<X>()) {
        if ((lane + G * (e / V)) * V >= cols) v[k][i].x = 0.f;
        if ((lane + G * ((e + 1) / V)) * V >= cols) v[k][i].y = 0.f;
      }
      q = ffma2(v[k][i], v[k][i], q);
    }
    rstd[k] = q.x + q.y;
  }
#pragma unroll
  for (int k = 0; k < ROWS; ++k) rstd[k] = rsqrtf(group_sum<G>(rstd[k], red) * inv + eps);
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (lane == 0 && k < here) {
      mean_out[row + k] = mean[k];
      rstd_out[row + k] = rstd[k];
    }
  }
  by_act(act, [&](auto a) {
    const Gelu<decltype(a)::value, sizeof(Y) == 4> gelu;
#pragma unroll
    for (int e = 0; e < 2 * NP; e += 4) {
      const float4 g = load4<V, G>(gamma, lane, cols, e), b = load4<V, G>(beta, lane, cols, e);
#pragma unroll
      for (int k = 0; k < ROWS; ++k) {
        const float2 r = both(rstd[k]);
        v[k][e / 2] = gelu.value(ffma2(fmul2(v[k][e / 2], r), make_float2(g.x, g.y), make_float2(b.x, b.y)));
        v[k][e / 2 + 1] = gelu.value(ffma2(fmul2(v[k][e / 2 + 1], r), make_float2(g.z, g.w), make_float2(b.z, b.w)));
      }
    }
  });
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if (k < here) store_row<Y, V, NCH, G>(y + (row + k) * y_ld, lane, cols, v[k]);
}

// Rows on their way per thread in the backward pass (see its ring).
template <typename X, int V, int NCH>
__host__ __device__ constexpr int bwd_stages() {
  return V == 1 ? 0 : (sizeof(X) == 2 && NCH * V <= 16 ? 3 : 2);
}
template <typename X, typename Y, int V, int NCH>
__host__ __device__ constexpr int bwd_stage_bytes(bool res) {
  return kLnThreads * NCH * V * static_cast<int>((res ? 2 : 1) * sizeof(X) + sizeof(Y));
}

// Persistent blocks: each thread keeps its columns' dgamma and dbeta over all
// the rows it sees; the block adds its groups' sums in order and leaves one
// partial per block, which layernorm_affine_kernel adds up in block order.  The
// next two or three rows are on their way to a ring in shared memory, every
// thread copying what it will read (in registers there is room for one, and 16
// warps with one row in flight each left HBM at half its rate).
template <typename X, typename Y, int V, int NCH, int G>
__global__ void __launch_bounds__(kLnThreads, NCH * V <= 16 ? 2 : 1)
layernorm_bwd_kernel(const Y* __restrict__ dy, int64_t dy_ld, const X* __restrict__ x, int64_t x_ld, int64_t rows,
                     int cols, const float* __restrict__ gamma, const float* __restrict__ beta,
                     const float* __restrict__ mean, const float* __restrict__ rstd, int act, const X* dres,
                     int64_t dres_ld, X* dx, int64_t dx_ld, float* __restrict__ partial,
                     float* __restrict__ dgamma, float* __restrict__ dbeta) {
  extern __shared__ __align__(16) uint8_t ring[];  // [stages]{x, dy, dres}; at the end [groups][2][cols] sums
  __shared__ float red[kLnThreads / 32];
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int kGroups = kLnThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  constexpr int NP = NCH * V / 2;
  float2 dg[NP], db[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) dg[i] = db[i] = both(0.f);
  const float inv = 1.0f / cols;
  constexpr int kStages = bwd_stages<X, V, NCH>();
  const int stage_bytes = bwd_stage_bytes<X, Y, V, NCH>(dres != nullptr);
  constexpr int kXBytes = kLnThreads * NCH * V * static_cast<int>(sizeof(X));
  constexpr int kYBytes = kLnThreads * NCH * V * static_cast<int>(sizeof(Y));
  auto slot_x = [&](int st) { return reinterpret_cast<Vec<X, V>*>(ring + st * stage_bytes) + threadIdx.x; };
  auto slot_y = [&](int st) { return reinterpret_cast<Vec<Y, V>*>(ring + st * stage_bytes + kXBytes) + threadIdx.x; };
  auto slot_r = [&](int st) {
    return reinterpret_cast<Vec<X, V>*>(ring + st * stage_bytes + kXBytes + kYBytes) + threadIdx.x;
  };
  auto fetch = [&](int64_t row, int st) {
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int c = (lane + G * i) * V;
        if (c < cols) {
          copy_async<V * sizeof(X)>(slot_x(st) + i * kLnThreads, x + row * x_ld + c);
          copy_async<V * sizeof(Y)>(slot_y(st) + i * kLnThreads, dy + row * dy_ld + c);
          if (dres) copy_async<V * sizeof(X)>(slot_r(st) + i * kLnThreads, dres + row * dres_ld + c);
        }
      }
    }
    copy_commit();  // a group per row, an empty one past the end
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kGroups + group;
  pdl_wait();
  if (kStages > 0) {
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(row + i * step, i);
  }
  int st = 0;
  float mn = row < rows ? mean[row] : 0.f, rn = row < rows ? rstd[row] : 0.f;
  for (; row < rows; row += step) {
    const float r = rn, m = mn;
    if (row + step < rows) {
      mn = mean[row + step];
      rn = rstd[row + step];
    }
    float2 xh[NP], w[NP], res[NP];
    if (kStages > 0) {
      copy_wait<kStages == 0 ? 0 : kStages - 1>();
      read_ring<X, V, NCH, G>(slot_x(st), lane, cols, xh);
      read_ring<Y, V, NCH, G>(slot_y(st), lane, cols, w);
      // (dres is read when it is needed; its stage is refilled after that)
      if (!dres) fetch(row + kStages * step, st);
    } else {
      Vec<X, V> xv[NCH];
      Vec<Y, V> yv[NCH];
      load_row<X, V, NCH, G>(x + row * x_ld, lane, cols, xv);
      load_row<Y, V, NCH, G>(dy + row * dy_ld, lane, cols, yv);
      widen<X, V, NCH>(xv, xh);
      widen<Y, V, NCH>(yv, w);
    }
    float2 s1 = both(0.f), s2 = both(0.f);
    // (columns past the end: dy is 0, so they add nothing)
    by_act(act, [&](auto a) {
      constexpr int ACT = decltype(a)::value;
      const Gelu<ACT, sizeof(X) == 4> gelu;  // (dx is X)
#pragma unroll
      for (int e = 0; e < 2 * NP; e += 4) {
        const float4 g4 = load4<V, G>(gamma, lane, cols, e);
        float4 b4 = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ACT != 0) b4 = load4<V, G>(beta, lane, cols, e);
#pragma unroll
        for (int i = e / 2; i < e / 2 + 2; ++i) {
          const float2 g = i & 1 ? make_float2(g4.z, g4.w) : make_float2(g4.x, g4.y);
          const float2 b = i & 1 ? make_float2(b4.z, b4.w) : make_float2(b4.x, b4.y);
          xh[i] = fmul2(fadd2(xh[i], both(-m)), both(r));
          if (ACT != 0) w[i] = fmul2(w[i], gelu.slope(ffma2(xh[i], g, b)));
          dg[i] = ffma2(w[i], xh[i], dg[i]);
          db[i] = fadd2(db[i], w[i]);
          w[i] = fmul2(w[i], g);
          s1 = fadd2(s1, w[i]);
          s2 = ffma2(w[i], xh[i], s2);
        }
      }
    });
    const float c1 = group_sum<G>(s1.x + s1.y, red) * inv;
    const float c2 = group_sum<G>(s2.x + s2.y, red) * inv;
    if (dres) {
      if (kStages > 0) {
        read_ring<X, V, NCH, G>(slot_r(st), lane, cols, res);
        fetch(row + kStages * step, st);
      } else {
        Vec<X, V> rv[NCH];
        load_row<X, V, NCH, G>(dres + row * dres_ld, lane, cols, rv);
        widen<X, V, NCH>(rv, res);
      }
#pragma unroll
      for (int i = 0; i < NP; ++i)
        w[i] = ffma2(both(r), ffma2(xh[i], both(-c2), fadd2(w[i], both(-c1))), res[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NP; ++i) w[i] = fmul2(both(r), ffma2(xh[i], both(-c2), fadd2(w[i], both(-c1))));
    }
    st = st + 1 == kStages ? 0 : st + 1;
    store_row<X, V, NCH, G>(dx + row * dx_ld, lane, cols, w);
  }
  // The block's sums: to `partial`, or, when the grid is one cluster (dgamma given),
  // in shared memory for its blocks to add up.
  const bool cluster = dgamma != nullptr;
  float* acc = reinterpret_cast<float*>(ring);
  float* mine = cluster ? acc : partial + static_cast<int64_t>(blockIdx.x) * 2 * cols;
  float* sums = kGroups > 1 ? acc + group * 2 * cols : mine;
  __syncthreads();  // every group is done with the ring
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = (lane + G * i) * V;
    if (c < cols) {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int e = i * V + k;
        sums[c + k] = e & 1 ? dg[e / 2].y : dg[e / 2].x;
        sums[cols + c + k] = e & 1 ? db[e / 2].y : db[e / 2].x;
      }
    }
  }
  if (kGroups > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * cols; c += kLnThreads) {
      float v = acc[c];
#pragma unroll
      for (int i = 1; i < kGroups; ++i) v += acc[i * 2 * cols + c];
      mine[c] = v;
    }
  }
  if (cluster) {
    cluster_sync();
    const int blocks = static_cast<int>(gridDim.x);
    for (int c = static_cast<int>(blockIdx.x) * kLnThreads + threadIdx.x; c < 2 * cols; c += blocks * kLnThreads) {
      float v = 0.f;
      for (int i = 0; i < blocks; ++i) v += ld_dsmem(mapa_shared(smem_u32(acc + c), i));
      (c < cols ? dgamma + c : dbeta + (c - cols))[0] = v;
    }
    cluster_sync();  // no block's shared memory goes before the others have read it
  }
}

// dgamma and dbeta: the blocks' partials added in a fixed order.  A block takes 8
// columns of the 2 cols with 64 threads each, so that all of a thread's loads (5
// of 296 partials) are in flight at once; 32 columns to a block with 16 warps took
// 7.3 us for 1024 columns where this takes 5.5 (each alone, with cold caches).
constexpr int kAffineCols = 8, kAffineThreads = 512;
__global__ void __launch_bounds__(kAffineThreads)
layernorm_affine_kernel(const float* __restrict__ partial, int blocks, int cols, float* __restrict__ dgamma,
                        float* __restrict__ dbeta) {
  __shared__ float red[kAffineThreads / 32][kAffineCols];
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int col = threadIdx.x % kAffineCols;
  const int c = blockIdx.x * kAffineCols + col;
  pdl_wait();
  float s = 0.f;
  if (c < 2 * cols) {
#pragma unroll 8
    for (int i = threadIdx.x / kAffineCols; i < blocks; i += kAffineThreads / kAffineCols)
      s += partial[static_cast<int64_t>(i) * 2 * cols + c];
  }
#pragma unroll
  for (int o = kAffineCols; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 < kAffineCols) red[threadIdx.x / 32][col] = s;
  __syncthreads();
  if (threadIdx.x < kAffineCols && c < 2 * cols) {
    s = red[0][col];
#pragma unroll
    for (int i = 1; i < kAffineThreads / 32; ++i) s += red[i][col];
    (c < cols ? dgamma + c : dbeta + (c - cols))[0] = s;
  }
}

// Calls fn with the compile-time shape for this row: vector accesses when the
// width, every stride and every pointer allow 16-byte chunks of X (and the same
// number of elements of Y and fp32), single elements otherwise.
template <typename X, int G, typename F>
cudaError_t by_chunks(bool vec, int cols, F&& fn) {
  constexpr int V = 16 / sizeof(X);
  constexpr int kStep = chunk_step<X>();
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

// Blocks of the backward pass: what is resident at once (see its launch bounds).
// Few rows, at most one to a group: one cluster of up to 8 blocks does it all in one
// launch, adding its blocks' sums through distributed shared memory (49 x 768: 5.4 us
// on the GPU against 4.9 in two launches, of which each costs the host 2.7; at 256
// rows 8.8 against 5.5).
constexpr int kLnCluster = 8;
bool bwd_in_cluster(int64_t rows, int cols) {
  return rows <= kLnCluster * (cols <= kWarpCols ? kLnThreads / 32 : 1);
}

int bwd_blocks(int64_t rows, int cols) {
  const int per = cols <= kWarpCols ? kLnThreads / 32 : 1;
  const int64_t most = cols <= kWarpCols / 2 ? 2 * kNumSMs : kNumSMs;
  const int64_t want = (rows + per - 1) / per;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(want, bwd_in_cluster(rows, cols) ? kLnCluster : most)));
}

template <typename X, typename Y, int V, int NCH, int G>
cudaError_t fwd_launch(const LnTrain& s, const void* xp, void* yp, float eps, float* mean, float* rstd,
                       cudaStream_t st) {
  constexpr int kPer = kLnThreads / G;
  // Two 16-bit rows of up to 512 columns to a warp once a row each fills the GPU
  // twice (7984 x 512: 4.3 us, one each 5.2).
  constexpr int kRows = G == 32 && V == 8 && NCH <= 2 ? 2 : 1;
  const bool more = kRows == 2 && s.rows >= 2 * kPer * kNumSMs;
  const int64_t per = more ? kRows * kPer : kPer;
  return launch_pdl(more ? layernorm_fwd_kernel<X, Y, V, NCH, G, kRows> : layernorm_fwd_kernel<X, Y, V, NCH, G, 1>,
                    dim3(static_cast<unsigned>((s.rows + per - 1) / per)), dim3(kLnThreads), 0, st,
                    static_cast<const X*>(xp), s.x_ld, static_cast<Y*>(yp), s.y_ld, s.rows, s.cols, s.gamma, s.beta,
                    eps, s.act, mean, rstd);
}

template <typename X, typename Y, int G>
cudaError_t fwd(const LnTrain& s, const void* xp, void* yp, float eps, float* mean, float* rstd, cudaStream_t st) {
  constexpr int V = 16 / sizeof(X);
  const bool vec = s.cols % V == 0 && s.x_ld % V == 0 && s.y_ld % V == 0 && aligned(xp, 16) &&
                   aligned(yp, V * sizeof(Y)) && aligned(s.gamma, 16) && aligned(s.beta, 16);
  return by_chunks<X, G>(vec, s.cols, [&](auto v, auto nch) {
    return fwd_launch<X, Y, decltype(v)::value, decltype(nch)::value, G>(s, xp, yp, eps, mean, rstd, st);
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
  float* dgamma;  // null: sums to partial
  float* dbeta;
};

template <typename X, typename Y, int G>
cudaError_t bwd(const LnTrain& s, const BwdPtrs& p, cudaStream_t st) {
  constexpr int V = 16 / sizeof(X);
  const bool vec = s.cols % V == 0 && s.x_ld % V == 0 && s.y_ld % V == 0 && p.dx_ld % V == 0 &&
                   (!p.dres || (p.dres_ld % V == 0 && aligned(p.dres, 16))) && aligned(p.x, 16) && aligned(p.dx, 16) &&
                   aligned(p.dy, V * sizeof(Y)) && aligned(s.gamma, 16) && aligned(s.beta, 16);
  const size_t sums = (p.dgamma || G == 32 ? kLnThreads / G : 0) * 2 * static_cast<size_t>(s.cols) * sizeof(float);
  return by_chunks<X, G>(vec, s.cols, [&](auto v, auto nch) {
    constexpr int kV = decltype(v)::value, kN = decltype(nch)::value;
    const size_t smem = std::max(
        sums, static_cast<size_t>(bwd_stages<X, kV, kN>()) * bwd_stage_bytes<X, Y, kV, kN>(p.dres != nullptr));
    auto kernel = layernorm_bwd_kernel<X, Y, kV, kN, G>;
    if (smem > 47 * 1024) {  // with the static part, more than the 48 KB that need no asking
      const cudaError_t r =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
      if (r != cudaSuccess) return r;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(bwd_blocks(s.rows, s.cols));
    cfg.blockDim = dim3(kLnThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {cfg.gridDim.x, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = p.dgamma ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<const Y*>(p.dy), s.y_ld, static_cast<const X*>(p.x), s.x_ld,
                              s.rows, s.cols, s.gamma, s.beta, p.mean, p.rstd, s.act, static_cast<const X*>(p.dres),
                              p.dres_ld, static_cast<X*>(p.dx), p.dx_ld, p.partial, p.dgamma, p.dbeta);
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
  if (bwd_in_cluster(rows, cols)) return 0;
  return static_cast<size_t>(bwd_blocks(rows, cols)) * 2 * cols * sizeof(float);
}

cudaError_t launch_layernorm_bwd(const LnTrain& s, const void* dy, const void* x, const float* mean,
                                 const float* rstd, const void* dres, int64_t dres_ld, void* dx, int64_t dx_ld,
                                 float* dgamma, float* dbeta, void* ws, cudaStream_t st) {
  const bool cluster = bwd_in_cluster(s.rows, s.cols);
  const BwdPtrs p = {dy,    x,     mean, rstd, dres, dres_ld, dx, dx_ld, static_cast<float*>(ws), cluster ? dgamma : nullptr,
                     cluster ? dbeta : nullptr};
  const cudaError_t r = by_types(s.x_type, s.y_type, [&](auto xt, auto yt) {
    using X = decltype(xt);
    using Y = decltype(yt);
    return s.cols <= kWarpCols ? bwd<X, Y, 32>(s, p, st) : bwd<X, Y, kLnThreads>(s, p, st);
  });
  if (r != cudaSuccess || cluster) return r;
  return launch_pdl(layernorm_affine_kernel, dim3((2 * s.cols + kAffineCols - 1) / kAffineCols),
                    dim3(kAffineThreads), 0, st, p.partial,
                    bwd_blocks(s.rows, s.cols), s.cols, dgamma, dbeta);
}

}  // namespace w2v
