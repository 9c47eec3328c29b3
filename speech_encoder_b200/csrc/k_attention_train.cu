// Attention for training, head dim 64, scale 1/8, fp16 or bf16: the forward
// pass that leaves each row's log-sum-exp, and the backward pass that recomputes
// the probabilities from it.  Clips of a padded batch have lengths of their own.
//
// All products run on tcgen05 with fp32 accumulators in tensor memory.  The
// streamed operands (K and V, or Q and dO) come by TMA as 64-row tiles of
// 128-byte rows, 128-byte swizzled, and each tile serves two products: with its
// rows as the N dimension (K-major B: scores, dP) and with its rows as the
// reduction dimension (MN-major B: P V, P^T dO, dS K, dS^T Q), so nothing is
// ever transposed in memory.
//
// Rows past a clip's frames may hold anything.  As rows of an A operand they
// only reach accumulator rows that are not used; as rows of a streamed tile they
// would reach everything (0 * NaN), so the warp that issues the products first
// overwrites those rows of the clip's last tile with zeros in shared memory.
#include "ptx.cuh"
#include "w2v_internal.h"

namespace w2v {
namespace {

constexpr int kHd = 64;             // head dim
constexpr int kSub = 64;            // rows of a streamed tile
constexpr int kTileBytes = kSub * kHd * 2;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kC2 = 0.125f * kLog2e;  // scores to log2 units

// kind::f16 instruction descriptor with an fp32 accumulator: A and B both fp16
// or both bf16, A K-major (or in tensor memory), B K-major or MN-major.
template <bool BF16>
__device__ __forceinline__ constexpr uint32_t idesc_train(int M, int N, bool b_mn) {
  return (1u << 4) | ((BF16 ? 1u : 0u) << 7) | ((BF16 ? 1u : 0u) << 10) | ((b_mn ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// Two fp32 values rounded to the operand type, the first in the low half.
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if (BF16)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if (BF16) return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// One lane of the (converged) warp.  With the whole warp around the loop and the
// issue behind this predicate, addresses and descriptors stay in uniform
// registers; behind `lane == 0` each product took about 90 cycles to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// A value that is the same in every lane, in a form that the compiler knows to be.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

__device__ __forceinline__ int clip_frames(const int32_t* frames, int b, int T) {
  if (!frames) return T;
  const int n = frames[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

// Zeros rows [valid, 64) of a 64-row tile (one warp).  Zero chunks do not care
// about the swizzle.
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int valid, int lane) {
  for (int i = valid * 8 + lane; i < kSub * 8; i += 32)
    *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
}

// One thread's 32 columns of an accumulator row, scaled and rounded; zeros where
// the row is not live (the accumulator may then hold anything).
template <bool BF16>
__device__ __forceinline__ void store_row_part(uint32_t taddr, uint16_t* dst, float scale, bool write, bool live) {
  float v[32];
  tmem_ld32(taddr, v);
  if (!write) return;
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live)
      u = make_uint4(pack2<BF16>(v[i] * scale, v[i + 1] * scale), pack2<BF16>(v[i + 2] * scale, v[i + 3] * scale),
                     pack2<BF16>(v[i + 4] * scale, v[i + 5] * scale), pack2<BF16>(v[i + 6] * scale, v[i + 7] * scale));
    *reinterpret_cast<uint4*>(dst + i) = u;
  }
}

// -------------------------------------------------------------------- forward
// One CTA per (128-query tile, clip and head): warps 0-3 softmax, one thread
// per query row; warp 4 TMA; warp 5 tensor memory and products.  Within a CTA
// the steps of a 64-key tile (scores, softmax, P V) follow one another; 128
// tensor-memory columns and 50 KB of shared memory let four CTAs share an SM
// and fill each other's gaps.
struct FwdSmem {
  static constexpr int kStages = 2;
  static constexpr int Q = 0;
  static constexpr int KV = 2 * kTileBytes;  // [stages]{K, V}
  static constexpr int BAR = KV + kStages * 2 * kTileBytes;
  static constexpr int TOTAL = BAR + 128 + 1024;
};
constexpr int kFwdThreads = 192;

template <bool BF16>
__global__ void __launch_bounds__(kFwdThreads, 4)
attention_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const int32_t* __restrict__ frames, int T, int H,
                     int tiles, uint16_t* __restrict__ out, int64_t out_ld, int64_t out_bs, float* __restrict__ lse,
                     int* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + FwdSmem::BAR);
  uint64_t* q_full = bars;
  uint64_t* s_full = bars + 1;
  uint64_t* p_full = bars + 2;
  uint64_t* pv_done = bars + 3;
  uint64_t* kv_full = bars + 4;
  uint64_t* kv_empty = bars + 4 + FwdSmem::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 4 + 2 * FwdSmem::kStages);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int qt = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int b = bh / H, h = bh % H;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(s_full, 1);
    mbar_init(p_full, 4);
    mbar_init(pv_done, 1);
    for (int i = 0; i < FwdSmem::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    fence_mbar_init();
    pdl_launch_dependents();
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, 128);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t tS = tmem, tO = tmem + 64;
  pdl_wait();
  const int len = clip_frames(frames, b, T);
  const int nkv = qt * 128 < len ? (len + kSub - 1) / kSub : 0;  // no key tile for rows past the clip

  if (warp == 4) {
    if (lane == 0 && nkv > 0) {
      mbar_arrive_expect_tx(q_full, 2 * kTileBytes);
      tma_load_3d(smem + FwdSmem::Q, &tmQ, q_full, h * kHd, qt * 128, b);
      tma_load_3d(smem + FwdSmem::Q + kTileBytes, &tmQ, q_full, h * kHd, qt * 128 + kSub, b);
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < nkv; ++j) {
        const int st = j % FwdSmem::kStages;
        if (j >= FwdSmem::kStages && !mbar_wait(&kv_empty[st], ((j / FwdSmem::kStages) & 1) ^ 1)) {
          atomicOr(err, kErrWaitProducer);
          ok = false;
          break;
        }
        uint8_t* dst = smem + FwdSmem::KV + st * 2 * kTileBytes;
        mbar_arrive_expect_tx(&kv_full[st], 2 * kTileBytes);
        tma_load_3d(dst, &tmK, &kv_full[st], h * kHd, j * kSub, b);
        tma_load_3d(dst + kTileBytes, &tmV, &kv_full[st], h * kHd, j * kSub, b);
        issued = j + 1;
      }
      if (!ok) {  // wait for the copies in flight before the CTA's shared memory goes
        mbar_wait(q_full, 0);
        for (int j = issued > FwdSmem::kStages ? issued - FwdSmem::kStages : 0; j < issued; ++j)
          mbar_wait(&kv_full[j % FwdSmem::kStages], (j / FwdSmem::kStages) & 1);
      }
    }
  } else if (warp == 5) {
    constexpr uint32_t idS = idesc_train<BF16>(128, kSub, false);
    constexpr uint32_t idO = idesc_train<BF16>(128, kHd, true);
    const uint64_t dQ = desc_sw128(smem_u32(smem + FwdSmem::Q));
    bool ok = nkv == 0 || mbar_wait(q_full, 0);
    for (int j = 0; j < nkv; ++j) {
      const int st = j % FwdSmem::kStages;
      uint8_t* kv = smem + FwdSmem::KV + st * 2 * kTileBytes;
      // P of the previous tile lies over the scores: its product must be done.
      ok = __all_sync(0xffffffffu, ok && mbar_wait(&kv_full[st], (j / FwdSmem::kStages) & 1) &&
                                       (j == 0 || mbar_wait(pv_done, (j - 1) & 1)));
      if (!ok) break;
      const int valid = len - j * kSub;
      if (valid < kSub) {
        zero_tail_rows(kv + kTileBytes, valid, lane);
        fence_proxy_async_smem();
      }
      __syncwarp();
      const uint64_t dK = desc_sw128(smem_u32(kv)), dV = desc_sw128(smem_u32(kv + kTileBytes));
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f16(tS, dQ + 2 * kk, dK + 2 * kk, idS, kk);
        umma_commit(s_full);
      }
      __syncwarp();
      ok = __all_sync(0xffffffffu, mbar_wait(p_full, j & 1));
      if (!ok) break;
      tc_fence_after();
      if (elect_one()) {
        // 16 keys a step: 8 packed columns of P, 16 rows (2048 bytes) of V.
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tO, tS + 8 * kk, dV + static_cast<uint64_t>(128 * kk), idO, (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&kv_empty[st]);
        umma_commit(pv_done);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(err, kErrWaitMma);
  } else {
    const int r = warp * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    float m_ref = -INFINITY, l = 0.f;  // reference maximum (log2 units), sum of exponentials
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full, j & 1));
      if (ok) {
        tc_fence_after();
        const int valid = len - j * kSub;
        float s[32];
        float mx = -INFINITY;
#pragma unroll
        for (int c0 = 0; c0 < kSub; c0 += 32) {
          tmem_ld32(tS + lane_base + c0, s);
          if (valid < kSub) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c0 + i >= valid) s[i] = -INFINITY;
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) mx = fmax3(mx, s[i], s[i + 1]);
        }
        // The reference moves only when the maximum exceeds it by 2^8, so the
        // accumulator is rarely rescaled and P stays <= 256.
        const bool move = mx * kC2 > m_ref + 8.0f;
        if (__any_sync(0xffffffffu, move)) {
          const float m_new = move ? mx * kC2 : m_ref;
          if (j > 0) {
            const float alpha = ex2_approx(m_ref - m_new);
            l *= alpha;
            float o[16];
#pragma unroll
            for (int c0 = 0; c0 < kHd; c0 += 16) {
              tmem_ld16(tO + lane_base + c0, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tmem_st16(tO + lane_base + c0, o);
            }
          }
          m_ref = m_new;
        }
        // P of each half, packed, goes over score columns that were read already:
        // 0..15, then 16..31.
#pragma unroll
        for (int c0 = 0; c0 < kSub; c0 += 32) {
          tmem_ld32(tS + lane_base + c0, s);
          if (valid < kSub) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c0 + i >= valid) s[i] = -INFINITY;
          }
          uint32_t pk[16];
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const float2 x = ffma2(make_float2(s[i], s[i + 1]), make_float2(kC2, kC2), make_float2(-m_ref, -m_ref));
            const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
            sum = fadd2(sum, p);
            pk[i / 2] = pack2<BF16>(p.x, p.y);
          }
          l += sum.x + sum.y;
          tmem_st16_u32(tS + lane_base + c0 / 2, pk);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
    }
    if (nkv > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (nkv - 1) & 1));
    const int t = qt * 128 + r;
    if (ok) {
      tc_fence_after();
      const bool live = t < len;
      const float inv = live ? 1.0f / l : 0.f;
      uint16_t* dst = out + b * out_bs + t * out_ld + h * kHd;
#pragma unroll
      for (int c0 = 0; c0 < kHd; c0 += 32) store_row_part<BF16>(tO + lane_base + c0, dst + c0, inv, t < T, live);
      if (t < T) lse[static_cast<int64_t>(bh) * T + t] = live ? m_ref * kLn2 + logf(l) : -INFINITY;
    } else if (lane == 0) {
      atomicOr(err, kErrWaitSoftmax);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// -------------------------------------------------- backward: row statistics
// Per (clip, head, frame), padded to a multiple of 128 frames:
//   neg_l = -lse log2(e), -infinity where there is no probability, and
//   neg_d = -rowsum(dout o out), 0 there;
// in fp16 also, per 128 frames, the largest |dout row|^2 and |v row|^2.
// Eight lanes a row, 16 bytes each.
template <bool BF16>
__global__ void __launch_bounds__(256)
attention_bwd_rows_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ out, int64_t out_ld,
                          int64_t out_bs, const uint16_t* __restrict__ v, int64_t v_ld, int64_t v_bs,
                          const float* __restrict__ lse, const int32_t* __restrict__ frames, int T, int H, int tiles,
                          float* __restrict__ neg_l, float* __restrict__ neg_d, float2* __restrict__ peak) {
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int b = bh / H, h = bh % H;
  const int part = threadIdx.x & 7;
  pdl_wait();
  const int len = clip_frames(frames, b, T);
  float top_do = 0.f, top_v = 0.f;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int t = tile * 128 + it * 32 + (threadIdx.x >> 3);
    float d = 0.f, ndo = 0.f, nv = 0.f;
    if (t < len) {
      const int64_t at = b * out_bs + t * out_ld + h * kHd + part * 8;
      const uint4 a = *reinterpret_cast<const uint4*>(dout + at), o = *reinterpret_cast<const uint4*>(out + at);
      const uint32_t au[4] = {a.x, a.y, a.z, a.w}, ou[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = unpack2<BF16>(au[i]), y = unpack2<BF16>(ou[i]);
        d = fmaf(x.x, y.x, fmaf(x.y, y.y, d));
        if (!BF16) ndo = fmaf(x.x, x.x, fmaf(x.y, x.y, ndo));
      }
      if (!BF16) {
        const uint4 w = *reinterpret_cast<const uint4*>(v + b * v_bs + t * v_ld + h * kHd + part * 8);
        const uint32_t wu[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<BF16>(wu[i]);
          nv = fmaf(x.x, x.x, fmaf(x.y, x.y, nv));
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      d += __shfl_xor_sync(0xffffffffu, d, o);
      if (!BF16) {
        ndo += __shfl_xor_sync(0xffffffffu, ndo, o);
        nv += __shfl_xor_sync(0xffffffffu, nv, o);
      }
    }
    if (!BF16) {
      top_do = fmaxf(top_do, ndo);
      top_v = fmaxf(top_v, nv);
    }
    if (part == 0) {
      const int64_t at = static_cast<int64_t>(bh) * tiles * 128 + t;
      const float l = t < len ? lse[static_cast<int64_t>(bh) * T + t] : -INFINITY;
      neg_l[at] = l == -INFINITY ? -INFINITY : -l * kLog2e;
      neg_d[at] = t < len ? -d : 0.f;
    }
  }
  if (!BF16) {
    __shared__ float2 red[8];
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
      top_do = fmaxf(top_do, __shfl_xor_sync(0xffffffffu, top_do, o));
      top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, o));
    }
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(top_do, top_v);
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) {
        top_do = fmaxf(top_do, red[i].x);
        top_v = fmaxf(top_v, red[i].y);
      }
      peak[static_cast<int64_t>(bh) * tiles + tile] = make_float2(top_do, top_v);
    }
  }
}

// Scale of dS in fp16, a power of two: |dS_ij| <= P_ij |dout_i| |v_j - out_i|
// <= 2 max|dout| max|v| (out_i is a mean of v rows), so with that bound brought
// just under 2^15 no entry overflows and the smallest keep what precision fp16
// can give them.  Every thread of the warp gets the same value.
__device__ __forceinline__ float ds_scale(const float2* peak, int tiles, int lane) {
  float top_do = 0.f, top_v = 0.f;
  for (int i = lane; i < tiles; i += 32) {
    const float2 p = peak[i];
    top_do = fmaxf(top_do, p.x);
    top_v = fmaxf(top_v, p.y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    top_do = fmaxf(top_do, __shfl_xor_sync(0xffffffffu, top_do, o));
    top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, o));
  }
  const float bound = 2.0f * sqrtf(top_do) * sqrtf(top_v);
  if (!(bound > 0.f) || !(bound < INFINITY)) return 1.0f;
  const int e = max(-100, min(100, 14 - ilogbf(bound)));
  return scalbnf(1.0f, e);
}

// ------------------------------------------------------------------- backward
// Two kinds of CTA in one launch, with the same inner step.  A CTA holds 128
// rows of a pair of operands (A1, A2) and streams 64-row tiles of the other
// pair (B1, B2); per tile
//   S = A1 B1^T, dP = A2 B2^T             (M = 128, N = 64, K = 64)
//   P = 2^(S c + neg_l), dS = P o (dP + neg_d)
// A key CTA holds (K, V) and streams (Q, dO); its S, P and dS are transposed
// (row = key), the statistics belong to columns, and P and dS, rounded to the
// operand type in tensor memory over S and dP, are the A operands of
//   dV += P dO, dK += dS Q                 (M = 128, N = 64, K = 64 queries).
// A query CTA holds (Q, dO), streams (K, V), has one row's statistics per
// thread, and needs only dQ += dS K.  S and dP are computed twice, which costs
// 7 products instead of the 5 of a single pass, but each gradient has one owner
// that sums it in a fixed order: no atomics and no fp32 partial sums in memory.
//
// Warps 0-7: one TMEM lane quarter and 32 of the 64 columns each; warp 8 TMA;
// warp 9 tensor memory and products.  256 tensor-memory columns and 99 KB of
// shared memory: two CTAs per SM fill each other's gaps.
struct BwdSmem {
  static constexpr int kStages = 4;
  static constexpr int A = 0;                      // key CTA: K, V (128 rows each)
  static constexpr int B = 4 * kTileBytes;         // [stages]{B1, B2}
  static constexpr int STAT = B + kStages * 2 * kTileBytes;  // [stages]{neg_l[64], neg_d[64]}
  static constexpr int BAR = STAT + kStages * 512;
  static constexpr int TOTAL = BAR + 256 + 1024;
};
constexpr int kBwdThreads = 320;

struct BwdArgs {
  const uint16_t* q;
  const uint16_t* dout;
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  int64_t qkv_ld, qkv_bs, out_ld, out_bs, grad_ld, grad_bs;
  const int32_t* frames;
  const float* neg_l;
  const float* neg_d;
  const float2* peak;
  int T, H, tiles, bh;
  int* err;
};

template <bool BF16, bool KEYS>
__device__ __forceinline__ void bwd_body(const CUtensorMap& tmA1, const CUtensorMap& tmA2, const CUtensorMap& tmB1,
                                         const CUtensorMap& tmB2, const BwdArgs& a, int tile, int bh) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BwdSmem::BAR);
  uint64_t* a_full = bars;
  uint64_t* s_full = bars + 1;
  uint64_t* dp_full = bars + 2;
  uint64_t* p_full = bars + 3;
  uint64_t* ds_full = bars + 4;
  uint64_t* v_done = bars + 5;
  uint64_t* acc_done = bars + 6;
  uint64_t* b_full = bars + 7;
  uint64_t* b_empty = bars + 7 + BwdSmem::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 7 + 2 * BwdSmem::kStages);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int b = bh / a.H, h = bh % a.H;

  if (threadIdx.x == 0) {
    mbar_init(a_full, KEYS ? 1 : 8);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_full, 8);
    mbar_init(ds_full, 8);
    mbar_init(v_done, 1);
    mbar_init(acc_done, 1);
    for (int i = 0; i < BwdSmem::kStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    fence_mbar_init();
    pdl_launch_dependents();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  // Key CTA: dV | dK | S, P | dP, dS.  Query CTA: Q, dO (packed) | dQ | S | dP, dS.
  const uint32_t tAcc1 = tmem, tAcc2 = tmem + 64, tS = tmem + 128, tD = tmem + 192;
  const uint32_t tA1 = tmem, tA2 = tmem + 32;
  pdl_wait();
  const int len = clip_frames(a.frames, b, a.T);
  const int n_sub = tile * 128 < len ? (len + kSub - 1) / kSub : 0;

  if (warp == 8) {
    if (lane == 0 && n_sub > 0) {
      if (KEYS) {
        mbar_arrive_expect_tx(a_full, 4 * kTileBytes);
        for (int i = 0; i < 2; ++i) {
          tma_load_3d(smem + BwdSmem::A + i * kTileBytes, &tmA1, a_full, h * kHd, tile * 128 + i * kSub, b);
          tma_load_3d(smem + BwdSmem::A + (2 + i) * kTileBytes, &tmA2, a_full, h * kHd, tile * 128 + i * kSub, b);
        }
      }
      const float* nl = a.neg_l + static_cast<int64_t>(bh) * a.tiles * 128;
      const float* nd = a.neg_d + static_cast<int64_t>(bh) * a.tiles * 128;
      int issued = 0;
      bool ok = true;
      for (int j = 0; j < n_sub; ++j) {
        const int st = j % BwdSmem::kStages;
        if (j >= BwdSmem::kStages && !mbar_wait(&b_empty[st], ((j / BwdSmem::kStages) & 1) ^ 1)) {
          atomicOr(a.err, kErrWaitProducer);
          ok = false;
          break;
        }
        uint8_t* dst = smem + BwdSmem::B + st * 2 * kTileBytes;
        mbar_arrive_expect_tx(&b_full[st], 2 * kTileBytes + (KEYS ? 512 : 0));
        tma_load_3d(dst, &tmB1, &b_full[st], h * kHd, j * kSub, b);
        tma_load_3d(dst + kTileBytes, &tmB2, &b_full[st], h * kHd, j * kSub, b);
        if (KEYS) {
          bulk_load(smem + BwdSmem::STAT + st * 512, nl + j * kSub, 256, &b_full[st]);
          bulk_load(smem + BwdSmem::STAT + st * 512 + 256, nd + j * kSub, 256, &b_full[st]);
        }
        issued = j + 1;
      }
      if (!ok) {  // wait for the copies in flight before the CTA's shared memory goes
        if (KEYS) mbar_wait(a_full, 0);
        for (int j = issued > BwdSmem::kStages ? issued - BwdSmem::kStages : 0; j < issued; ++j)
          mbar_wait(&b_full[j % BwdSmem::kStages], (j / BwdSmem::kStages) & 1);
      }
    }
  } else if (warp == 9) {
    constexpr uint32_t idS = idesc_train<BF16>(128, kSub, false);
    constexpr uint32_t idG = idesc_train<BF16>(128, kHd, true);
    const uint64_t dA1 = desc_sw128(smem_u32(smem + BwdSmem::A));
    const uint64_t dA2 = desc_sw128(smem_u32(smem + BwdSmem::A + 2 * kTileBytes));
    const uint64_t dB = desc_sw128(smem_u32(smem + BwdSmem::B));
    auto tile_b1 = [&](int j) { return dB + static_cast<uint64_t>((j % BwdSmem::kStages) * (2 * kTileBytes >> 4)); };
    auto tile_b2 = [&](int j) { return tile_b1(j) + (kTileBytes >> 4); };
    auto wait_tile = [&](int j) {
      const int st = j % BwdSmem::kStages;
      const bool there = __all_sync(0xffffffffu, mbar_wait(&b_full[st], (j / BwdSmem::kStages) & 1));
      const int valid = len - j * kSub;
      if (there && valid < kSub) {
        uint8_t* bt = smem + BwdSmem::B + st * 2 * kTileBytes;
        zero_tail_rows(bt, valid, lane);
        zero_tail_rows(bt + kTileBytes, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      return there;
    };
    auto scores = [&](uint32_t d, uint64_t da, uint32_t ta, uint64_t db, uint64_t* bar) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (KEYS)
            umma_f16(d, da + 2 * kk, db + 2 * kk, idS, kk);
          else
            umma_f16_ts(d, ta + 8 * kk, db + 2 * kk, idS, kk);
        }
        umma_commit(bar);
      }
      __syncwarp();
    };
    // P and dS: columns 32 w .. 32 w + 31 packed at columns 32 w .. 32 w + 15, so
    // the four 16-row steps start at 0, 8, 32 and 40; each is 16 rows (2048 bytes)
    // of the streamed tile.
    auto accumulate = [&](uint32_t d, uint32_t ta, uint64_t db, int j, uint64_t* bar, uint64_t* empty) {
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(d, ta + 32 * (kk >> 1) + 8 * (kk & 1), db + static_cast<uint64_t>(128 * kk), idG,
                      (j > 0 || kk > 0) ? 1u : 0u);
        if (empty) umma_commit(empty);
        umma_commit(bar);
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t* bar, int j) { return __all_sync(0xffffffffu, mbar_wait(bar, j & 1)); };
    bool ok = n_sub == 0 || (__all_sync(0xffffffffu, mbar_wait(a_full, 0)) && wait_tile(0));
    if (ok && n_sub > 0) {
      scores(tS, dA1, tA1, tile_b1(0), s_full);
      scores(tD, dA2, tA2, tile_b2(0), dp_full);
    }
    // The next tile's scores run while the warps form this tile's dS, and its dP
    // while they form the next P, each as soon as its columns are free: those of S
    // once P's product is done (key CTA) or S has been read (query CTA), those of
    // dP once dS's product is done.
    for (int j = 0; ok && j < n_sub; ++j) {
      const bool more = j + 1 < n_sub;
      if (!(ok = wait(p_full, j))) break;
      if (KEYS) accumulate(tAcc1, tS, tile_b2(j), j, v_done, nullptr);
      if (more) {
        if (!(ok = wait_tile(j + 1) && (!KEYS || wait(v_done, j)))) break;
        scores(tS, dA1, tA1, tile_b1(j + 1), s_full);
      }
      if (!(ok = wait(ds_full, j))) break;
      accumulate(tAcc2, tD, tile_b1(j), j, acc_done, &b_empty[j % BwdSmem::kStages]);
      if (more) {
        if (!(ok = wait(acc_done, j))) break;
        scores(tD, dA2, tA2, tile_b2(j + 1), dp_full);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, kErrWaitMma);
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const int t = tile * 128 + quarter * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    const int64_t stat_row = static_cast<int64_t>(bh) * a.tiles * 128;
    const float scale = BF16 ? 1.0f : ds_scale(a.peak + static_cast<int64_t>(bh) * a.tiles, a.tiles, lane);
    float row_l = 0.f, row_d = 0.f;
    if (!KEYS) {
      // Packed rows of Q (half 0) or dO (half 1) into tensor memory; zeros past the clip.
      const uint16_t* src = half == 0 ? a.q + b * a.qkv_bs + t * a.qkv_ld : a.dout + b * a.out_bs + t * a.out_ld;
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; i += 4) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (t < len) u = *reinterpret_cast<const uint4*>(src + h * kHd + 2 * i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
      const uint32_t dst = (half == 0 ? tA1 : tA2) + lane_base;
      tmem_st16_u32(dst, *reinterpret_cast<const uint32_t(*)[16]>(w));
      tmem_st16_u32(dst + 16, *reinterpret_cast<const uint32_t(*)[16]>(w + 16));
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(a_full);
      row_l = a.neg_l[stat_row + t];
      row_d = a.neg_d[stat_row + t];
    }
    bool ok = true;
    for (int j = 0; j < n_sub; ++j) {
      const float* st_l = reinterpret_cast<const float*>(smem + BwdSmem::STAT + (j % BwdSmem::kStages) * 512) + half * 32;
      const float* st_d = st_l + 64;
      const int valid = len - j * kSub - half * 32;
      float s[32];
      uint32_t pk[16];
      // (KEYS: the statistics came with the streamed tile, whose arrival only the
      // product warp has seen)
      if (ok)
        ok = __all_sync(0xffffffffu, mbar_wait(s_full, j & 1) &&
                                         (!KEYS || mbar_wait(&b_full[j % BwdSmem::kStages], (j / BwdSmem::kStages) & 1)));
      if (ok) {
        tc_fence_after();
        tmem_ld32(tS + lane_base + half * 32, s);
      }
      if (!KEYS) {  // S has been read: its columns are free for the next tile's
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (ok) {
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 l4 = make_float4(row_l, row_l, row_l, row_l);
          if (KEYS) l4 = *reinterpret_cast<const float4*>(st_l + i);
          const float2 x0 = ffma2(make_float2(s[i], s[i + 1]), make_float2(kC2, kC2), make_float2(l4.x, l4.y));
          const float2 x1 = ffma2(make_float2(s[i + 2], s[i + 3]), make_float2(kC2, kC2), make_float2(l4.z, l4.w));
          s[i] = ex2_approx(x0.x);
          s[i + 1] = ex2_approx(x0.y);
          s[i + 2] = ex2_approx(x1.x);
          s[i + 3] = ex2_approx(x1.y);
        }
        // Keys past the clip: their scores are 0, not -infinity, and 2^neg_l may overflow.
        if (!KEYS && valid < 32) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i >= valid) s[i] = 0.f;
        }
        if (KEYS) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) pk[i / 2] = pack2<BF16>(s[i], s[i + 1]);
          tmem_st16_u32(tS + lane_base + half * 32, pk);
        }
      }
      if (KEYS) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1));
      if (ok) {
        tc_fence_after();
        float dp[32];
        tmem_ld32(tD + lane_base + half * 32, dp);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float4 d4 = make_float4(row_d, row_d, row_d, row_d);
          if (KEYS) d4 = *reinterpret_cast<const float4*>(st_d + i);
          float2 g0 = fmul2(fadd2(make_float2(dp[i], dp[i + 1]), make_float2(d4.x, d4.y)), make_float2(s[i], s[i + 1]));
          float2 g1 =
              fmul2(fadd2(make_float2(dp[i + 2], dp[i + 3]), make_float2(d4.z, d4.w)), make_float2(s[i + 2], s[i + 3]));
          if (!BF16) {
            g0 = fmul2(g0, make_float2(scale, scale));
            g1 = fmul2(g1, make_float2(scale, scale));
          }
          pk[i / 2] = pack2<BF16>(g0.x, g0.y);
          pk[i / 2 + 1] = pack2<BF16>(g1.x, g1.y);
        }
        // A single frame has P = 1 and no gradient through the softmax: dP and
        // rowsum(dO o O) are the same number there, summed in two orders.
        if (len == 1) {
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = 0u;
        }
        tmem_st16_u32(tD + lane_base + half * 32, pk);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (n_sub > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(acc_done, (n_sub - 1) & 1));
    if (ok) {
      tc_fence_after();
      const bool write = t < a.T, live = t < len;
      const int64_t at = b * a.grad_bs + t * a.grad_ld + h * kHd + half * 32;
      const float back = 0.125f / scale;
      store_row_part<BF16>(tAcc2 + lane_base + half * 32, (KEYS ? a.dk : a.dq) + at, back, write, live);
      if (KEYS) store_row_part<BF16>(tAcc1 + lane_base + half * 32, a.dv + at, 1.0f, write, live);
    } else if (lane == 0) {
      atomicOr(a.err, kErrWaitSoftmax);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kBwdThreads, 2)
attention_bwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDo,
                     const __grid_constant__ BwdArgs a) {
  const int units = a.tiles * a.bh;
  const int u = blockIdx.x < units ? blockIdx.x : blockIdx.x - units;
  if (blockIdx.x < units)
    bwd_body<BF16, true>(tmK, tmV, tmQ, tmDo, a, u % a.tiles, u / a.tiles);
  else
    bwd_body<BF16, false>(tmQ, tmDo, tmK, tmV, a, u % a.tiles, u / a.tiles);
}

// [batch][T][H][64] operand as {H * 64, T, batch}, 64-row boxes of one head.
cudaError_t map_rows(CUtensorMap* m, const void* p, int64_t ld, int64_t bs, const AttnTrain& s) {
  const uint64_t dims[3] = {static_cast<uint64_t>(s.H) * kHd, static_cast<uint64_t>(s.T),
                            static_cast<uint64_t>(s.batch)};
  const uint64_t strides[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(bs) * 2};
  const uint32_t box[3] = {kHd, kSub, 1};
  return make_tmap_f16(m, p, 3, dims, strides, box, true);
}

}  // namespace

cudaError_t launch_attention_fwd(const AttnTrain& s, const void* q, const void* k, const void* v, void* out,
                                 float* lse, int* err, cudaStream_t st) {
  CUtensorMap tq, tk, tv;
  cudaError_t r;
  if ((r = map_rows(&tq, q, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  if ((r = map_rows(&tk, k, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  if ((r = map_rows(&tv, v, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  auto kernel = s.bf16 ? attention_fwd_kernel<true> : attention_fwd_kernel<false>;
  if ((r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FwdSmem::TOTAL)) != cudaSuccess)
    return r;
  const int tiles = (s.T + 127) / 128;
  return launch_pdl(kernel, dim3(tiles * s.batch * s.H), dim3(kFwdThreads), FwdSmem::TOTAL, st, tq, tk, tv, s.frames,
                    s.T, s.H, tiles, static_cast<uint16_t*>(out), s.out_ld, s.out_bs, lse, err);
}

size_t attention_bwd_ws_bytes(int batch, int T, int H) {
  const size_t tiles = (static_cast<size_t>(T) + 127) / 128, bh = static_cast<size_t>(batch) * H;
  return bh * tiles * (128 * 2 * sizeof(float) + sizeof(float2));
}

cudaError_t launch_attention_bwd(const AttnTrain& s, const void* dout, const void* q, const void* k, const void* v,
                                 const void* out, const float* lse, void* dq, void* dk, void* dv, void* ws, int* err,
                                 cudaStream_t st) {
  CUtensorMap tq, tk, tv, td;
  cudaError_t r;
  if ((r = map_rows(&tq, q, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  if ((r = map_rows(&tk, k, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  if ((r = map_rows(&tv, v, s.qkv_ld, s.qkv_bs, s)) != cudaSuccess) return r;
  if ((r = map_rows(&td, dout, s.out_ld, s.out_bs, s)) != cudaSuccess) return r;
  const int tiles = (s.T + 127) / 128, bh = s.batch * s.H;
  const int64_t rows = static_cast<int64_t>(bh) * tiles * 128;
  float* neg_l = static_cast<float*>(ws);
  float* neg_d = neg_l + rows;
  float2* peak = reinterpret_cast<float2*>(neg_d + rows);
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  r = launch_pdl(s.bf16 ? attention_bwd_rows_kernel<true> : attention_bwd_rows_kernel<false>, dim3(tiles * bh),
                 dim3(256), 0, st, u16(dout), u16(out), s.out_ld, s.out_bs, u16(v), s.qkv_ld, s.qkv_bs, lse, s.frames,
                 s.T, s.H, tiles, neg_l, neg_d, peak);
  if (r != cudaSuccess) return r;
  BwdArgs a;
  a.q = u16(q);
  a.dout = u16(dout);
  a.dq = static_cast<uint16_t*>(dq);
  a.dk = static_cast<uint16_t*>(dk);
  a.dv = static_cast<uint16_t*>(dv);
  a.qkv_ld = s.qkv_ld; a.qkv_bs = s.qkv_bs;
  a.out_ld = s.out_ld; a.out_bs = s.out_bs;
  a.grad_ld = s.grad_ld; a.grad_bs = s.grad_bs;
  a.frames = s.frames;
  a.neg_l = neg_l;
  a.neg_d = neg_d;
  a.peak = peak;
  a.T = s.T; a.H = s.H; a.tiles = tiles; a.bh = bh;
  a.err = err;
  auto kernel = s.bf16 ? attention_bwd_kernel<true> : attention_bwd_kernel<false>;
  if ((r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BwdSmem::TOTAL)) != cudaSuccess)
    return r;
  return launch_pdl(kernel, dim3(2 * tiles * bh), dim3(kBwdThreads), BwdSmem::TOTAL, st, tq, tk, tv, td, a);
}

}  // namespace w2v
