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
constexpr float kLowest = -3.402823466e38f;  // the lowest fp32: below every finite score in log2 units

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

// The work unit of a CTA: 128 rows of one clip and head.  Unit u of a ragged batch
// is the u-th in the order longest clip first (ties by index), heads, tiles, of the
// tiles that hold frames; after those, in the same order, the tiles of padded rows
// alone.  CTAs start in grid order, so the last to start are short ones, and those
// with nothing but zeros to write do not hold places among the others (they did,
// and left half of the places empty for a third of a batch of 8 clips).  For
// batches of up to 64 clips, whose lengths a warp can hold and compare; larger ones
// are taken as they come.  All lanes of the warp take part and get the same answer.
struct Unit {
  int b, h, tile, len;
};
constexpr int kRankedBatch = 64;

// How many of all `units` have frames (all, for a batch that is taken as it comes).
__device__ __forceinline__ int live_units(const int32_t* frames, int batch, int T, int H, int units, int lane) {
  if (batch > kRankedBatch) return units;
  int m = lane < batch ? (clip_frames(frames, lane, T) + 127) / 128 : 0;
  if (lane + 32 < batch) m += (clip_frames(frames, lane + 32, T) + 127) / 128;
  return static_cast<int>(__reduce_add_sync(0xffffffffu, m)) * H;
}

__device__ __forceinline__ Unit find_unit(const int32_t* frames, int batch, int T, int H, int tiles, int u, int lane) {
  Unit r;
  if (!frames || batch > kRankedBatch) {
    r.tile = u % tiles;
    r.h = u / tiles % H;
    r.b = u / tiles / H;
    r.len = frames ? clip_frames(frames, r.b, T) : T;
    return r;
  }
  const int n0 = lane < batch ? clip_frames(frames, lane, T) : -1;
  const int n1 = lane + 32 < batch ? clip_frames(frames, lane + 32, T) : -1;
  int before0 = 0, before1 = 0, all = 0;  // tiles with frames of the clips before this lane's two; of all clips
  for (int o = 0; o < batch; ++o) {
    const int n = __shfl_sync(0xffffffffu, o < 32 ? n0 : n1, o & 31), m = (n + 127) / 128;
    if (n > n0 || (n == n0 && o < lane)) before0 += m;
    if (n > n1 || (n == n1 && o < lane + 32)) before1 += m;
    all += m;
  }
  const bool live = u < all * H;
  const int at = live ? u : u - all * H;
  // (counts of padded tiles likewise: all tiles less those with frames, clips in index order)
  if (!live) {
    before0 = before1 = 0;
    for (int o = 0; o < batch; ++o) {
      const int n = __shfl_sync(0xffffffffu, o < 32 ? n0 : n1, o & 31), m = tiles - (n + 127) / 128;
      if (o < lane) before0 += m;
      if (o < lane + 32) before1 += m;
    }
  }
  const int m0 = n0 < 0 ? 0 : (live ? (n0 + 127) / 128 : tiles - (n0 + 127) / 128);
  const int m1 = n1 < 0 ? 0 : (live ? (n1 + 127) / 128 : tiles - (n1 + 127) / 128);
  const bool mine0 = at >= before0 * H && at < (before0 + m0) * H;
  const bool mine1 = at >= before1 * H && at < (before1 + m1) * H;
  const int src = __ffs(__ballot_sync(0xffffffffu, mine0 || mine1)) - 1;
  const int m = __shfl_sync(0xffffffffu, mine1 ? m1 : m0, src);
  const int in = at - __shfl_sync(0xffffffffu, mine1 ? before1 : before0, src) * H;
  r.b = __shfl_sync(0xffffffffu, mine1 ? lane + 32 : lane, src);
  r.len = __shfl_sync(0xffffffffu, mine1 ? n1 : n0, src);
  r.h = in / m;
  r.tile = in % m + (live ? 0 : tiles - m);
  return r;
}

// 2^x of a pair on the FMA and ALU pipes, for a share of the forward pass's
// exponentials: its softmax warps are bound by the exponent unit (16 a clock per SM)
// and by issue about equally, and the share's optimum is flat (2 x 2999 frames x 16
// heads: none 118 us, a quarter of the pairs 115, half 124).  The backward pass,
// which has more else to do, is fastest with none.  x = j + f with j the
// nearest integer (adding 1.5 * 2^23 leaves j in the low mantissa bits), 2^f by the
// polynomial of degree 4 with the smallest largest relative error on [-1/2, 1/2]
// (2.7e-6, found by linear programming over a fine grid), j added to the
// exponent.  x is clamped below at -126, and so is NaN: rows with a score that is
// not finite are found by their maximum (see the forward kernel).
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  constexpr float kMagic = 12582912.0f;
  x = make_float2(fmaxf(x.x, -126.0f), fmaxf(x.y, -126.0f));
  const float2 t = fadd2(x, make_float2(kMagic, kMagic));
  const float2 j = fadd2(t, make_float2(-kMagic, -kMagic));
  const float2 f = ffma2(j, make_float2(-1.0f, -1.0f), x);
  float2 p = ffma2(f, make_float2(0.009567738510668278f, 0.009567738510668278f),
                   make_float2(0.05591749772429466f, 0.05591749772429466f));
  p = ffma2(p, f, make_float2(0.24024811387062073f, 0.24024811387062073f));
  p = ffma2(p, f, make_float2(0.6931219100952148f, 0.6931219100952148f));
  p = ffma2(p, f, make_float2(0.9999992251396179f, 0.9999992251396179f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

__device__ __forceinline__ float2 exp2_unit(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }

// Zeros over the 64 columns of one head in rows [from, to).
__device__ __forceinline__ void zero_rows(uint16_t* p, int64_t ld, int from, int to) {
  for (int i = threadIdx.x; i < (to - from) * 8; i += blockDim.x)
    *reinterpret_cast<uint4*>(p + (from + (i >> 3)) * ld + (i & 7) * 8) = make_uint4(0, 0, 0, 0);
}

// Zeros rows [valid, 64) of a 64-row tile (one warp).  Zero chunks do not care
// about the swizzle.
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int valid, int lane) {
  for (int i = valid * 8 + lane; i < kSub * 8; i += 32)
    *reinterpret_cast<uint4*>(tile + i * 16) = make_uint4(0, 0, 0, 0);
}

// Offset of 16-byte chunk c of row r in a tile of 128-byte rows, 128-byte swizzled.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// One thread's 32 columns of an accumulator row, scaled and rounded, into a staged
// tile of 128 rows (chunks c0 .. c0 + 3); zeros where the row is not live (the
// accumulator may then hold anything).
template <bool BF16>
__device__ __forceinline__ void stage_row_part(uint32_t taddr, uint8_t* tile, int r, int c0, float scale, bool live) {
  float v[32];
  tmem_ld32(taddr, v);
#pragma unroll
  for (int i = 0; i < 32; i += 8) {
    uint4 u = make_uint4(0, 0, 0, 0);
    if (live)
      u = make_uint4(pack2<BF16>(v[i] * scale, v[i + 1] * scale), pack2<BF16>(v[i + 2] * scale, v[i + 3] * scale),
                     pack2<BF16>(v[i + 4] * scale, v[i + 5] * scale), pack2<BF16>(v[i + 6] * scale, v[i + 7] * scale));
    *reinterpret_cast<uint4*>(tile + swizzled(r, c0 + i / 8)) = u;
  }
}

// The same of acc1 - w acc2.
template <bool BF16>
__device__ __forceinline__ void stage_row_difference(uint32_t acc1, uint32_t acc2, uint8_t* tile, int r, int c0,
                                                     float scale, float w, bool live) {
#pragma unroll
  for (int half = 0; half < 32; half += 16) {
    float v[16], x[16];
    tmem_ld16(acc1 + half, v);
    tmem_ld16(acc2 + half, x);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = scale * fmaf(-w, x[i], v[i]);
#pragma unroll
    for (int i = 0; i < 16; i += 8) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (live)
        u = make_uint4(pack2<BF16>(v[i], v[i + 1]), pack2<BF16>(v[i + 2], v[i + 3]), pack2<BF16>(v[i + 4], v[i + 5]),
                       pack2<BF16>(v[i + 6], v[i + 7]));
      *reinterpret_cast<uint4*>(tile + swizzled(r, c0 + (half + i) / 8)) = u;
    }
  }
}

// A staged tile to rows [0, rows) of one head, eight threads a row (a thread per
// row, straight from its registers, writes 32 lines an instruction and took 2.3 us
// for two tiles where this takes 1.5).
__device__ __forceinline__ void store_tile(const uint8_t* tile, uint16_t* dst, int64_t ld, int rows, int tid,
                                           int threads) {
  for (int i = tid; i < rows * 8; i += threads)
    *reinterpret_cast<uint4*>(dst + (i >> 3) * ld + (i & 7) * 8) =
        *reinterpret_cast<const uint4*>(tile + swizzled(i >> 3, i & 7));
}

// -------------------------------------------------------------------- forward
// One CTA per (128-query tile, clip and head): warps 0-3 softmax, one thread per
// query row; warp 4 TMA; warp 5 tensor memory and products.  Three score buffers of
// 64 keys in turn: the scores of tile j + 2 are issued once P V of tile j - 1, which
// had their buffer, is done, so the softmax warps go from tile to tile without
// waiting for a product.  P, packed, overwrites the columns that its thread has
// read; the accumulator is touched only when a row's reference maximum moves, after
// the previous P V.  256 tensor-memory columns and 82 KB of shared memory: two CTAs
// an SM (four with one score buffer each took 134 us for 2 x 2999 frames x 16 heads
// where this takes 115).
struct FwdSmem {
  static constexpr int kStages = 4;
  static constexpr int Q = 0;
  static constexpr int KV = 2 * kTileBytes;  // [stages]{K, V}
  static constexpr int BAR = KV + kStages * 2 * kTileBytes;
  static constexpr int TOTAL = BAR + 256 + 1024;
};
constexpr int kFwdThreads = 192;

template <bool BF16>
__global__ void __launch_bounds__(kFwdThreads, 2)
attention_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const int32_t* __restrict__ frames, int T, int H,
                     int batch, int tiles, uint16_t* __restrict__ out, int64_t out_ld, int64_t out_bs,
                     float* __restrict__ lse, int* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + FwdSmem::BAR);
  uint64_t* q_full = bars;
  uint64_t* s_full = bars + 1;   // [3], by score buffer
  uint64_t* p_full = bars + 4;   // [3]
  uint64_t* pv_done = bars + 7;  // [2], by parity of the tile
  uint64_t* kv_full = bars + 9;
  uint64_t* kv_empty = bars + 9 + FwdSmem::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 9 + 2 * FwdSmem::kStages);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  // Before tensor memory is asked for: a CTA that held columns while it waited for
  // the kernel before could keep them from a CTA of that kernel.  For the same
  // reason the next kernel may start only once this one's columns are taken.
  pdl_wait();
  const Unit unit = find_unit(frames, batch, T, H, tiles, blockIdx.x, lane);
  const int b = unit.b, h = unit.h, qt = unit.tile, len = unit.len;
  const int64_t bh = static_cast<int64_t>(b) * H + h;
  const int nkv = (len + kSub - 1) / kSub;
  if (qt * 128 >= len) {  // rows past the clip
    const int to = min(T, qt * 128 + 128);
    zero_rows(out + b * out_bs + h * kHd, out_ld, qt * 128, to);
    for (int t = qt * 128 + threadIdx.x; t < to; t += kFwdThreads) lse[bh * T + t] = -INFINITY;
    return;
  }

  auto load_tile = [&](int j) {
    const int st = j % FwdSmem::kStages;
    uint8_t* dst = smem + FwdSmem::KV + st * 2 * kTileBytes;
    mbar_arrive_expect_tx(&kv_full[st], 2 * kTileBytes);
    tma_load_3d(dst, &tmK, &kv_full[st], h * kHd, j * kSub, b);
    tma_load_3d(dst + kTileBytes, &tmV, &kv_full[st], h * kHd, j * kSub, b);
  };
  // The copying thread sets up the barriers and starts the first copies before the
  // others have the tensor memory.
  if (threadIdx.x == 4 * 32) {
    mbar_init(q_full, 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    for (int i = 0; i < FwdSmem::kStages; ++i) {
      mbar_init(&kv_full[i], 1);
      mbar_init(&kv_empty[i], 1);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(q_full, 2 * kTileBytes);
    tma_load_3d(smem + FwdSmem::Q, &tmQ, q_full, h * kHd, qt * 128, b);
    tma_load_3d(smem + FwdSmem::Q + kTileBytes, &tmQ, q_full, h * kHd, qt * 128 + kSub, b);
    for (int j = 0; j < min(nkv, FwdSmem::kStages); ++j) load_tile(j);
  }
  if (warp == 5) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  const uint32_t tS = tmem, tO = tmem + 192;  // scores at 0, 64, 128
  if (threadIdx.x == 0) pdl_launch_dependents();

  if (warp == 4) {
    if (lane == 0) {
      for (int j = FwdSmem::kStages; j < nkv; ++j) {
        if (!mbar_wait(&kv_empty[j % FwdSmem::kStages], ((j / FwdSmem::kStages) & 1) ^ 1)) {
          atomicOr(err, kErrWaitProducer);
          // wait for the copies in flight before the CTA's shared memory goes
          mbar_wait(q_full, 0);
          for (int i = j - FwdSmem::kStages; i < j; ++i)
            mbar_wait(&kv_full[i % FwdSmem::kStages], (i / FwdSmem::kStages) & 1);
          break;
        }
        load_tile(j);
      }
    }
  } else if (warp == 5) {
    constexpr uint32_t idS = idesc_train<BF16>(128, kSub, false);
    constexpr uint32_t idO = idesc_train<BF16>(128, kHd, true);
    const uint64_t dQ = desc_sw128(smem_u32(smem + FwdSmem::Q));
    const uint64_t dKV = desc_sw128(smem_u32(smem + FwdSmem::KV));
    auto tile_k = [&](int j) { return dKV + static_cast<uint64_t>((j % FwdSmem::kStages) * (2 * kTileBytes >> 4)); };
    auto scores = [&](int j) {
      const int st = j % FwdSmem::kStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&kv_full[st], (j / FwdSmem::kStages) & 1))) return false;
      const int valid = len - j * kSub;
      if (valid < kSub) {
        zero_tail_rows(smem + FwdSmem::KV + st * 2 * kTileBytes + kTileBytes, valid, lane);
        fence_proxy_async_smem();
        __syncwarp();
      }
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f16(tS + 64 * (j % 3), dQ + 2 * kk, tile_k(j) + 2 * kk, idS, kk);
        umma_commit(&s_full[j % 3]);
      }
      __syncwarp();
      return true;
    };
    bool ok = __all_sync(0xffffffffu, mbar_wait(q_full, 0)) && scores(0) && (nkv < 2 || scores(1));
    for (int j = 0; ok && j < nkv; ++j) {
      if (j + 2 < nkv) {
        if (j > 0) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1));
        if (!ok || !(ok = scores(j + 2))) break;
      }
      if (!(ok = __all_sync(0xffffffffu, mbar_wait(&p_full[j % 3], (j / 3) & 1)))) break;
      tc_fence_after();
      if (elect_one()) {
        // 16 keys a step: 8 packed columns of P, 16 rows (2048 bytes) of V.
        const uint64_t dV = tile_k(j) + (kTileBytes >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tO, tS + 64 * (j % 3) + 8 * kk, dV + static_cast<uint64_t>(128 * kk), idO,
                      (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(&pv_done[j & 1]);
        umma_commit(&kv_empty[j % FwdSmem::kStages]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) atomicOr(err, kErrWaitMma);
  } else {
    const int r = warp * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
    // Reference maximum (log2 units), sum of exponentials.  A row whose softmax is not
    // defined ends with a reference that is not finite or still the lowest, and gets
    // NaN: +infinity stands for a NaN or an infinite score, the lowest for a row without
    // a score above -infinity.  The probabilities do not show it by themselves: the
    // polynomial makes 2^-126 of NaN.
    float m_ref = kLowest, l = 0.f;
    bool ok = true;
    for (int j = 0; j < nkv; ++j) {
      const uint32_t cols = tS + 64 * (j % 3) + lane_base;
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&s_full[j % 3], (j / 3) & 1));
      if (ok) {
        tc_fence_after();
        const int valid = len - j * kSub;
        float s[kSub];
        tmem_ld32(cols, *reinterpret_cast<float(*)[32]>(s));
        tmem_ld32(cols + 32, *reinterpret_cast<float(*)[32]>(s + 32));
        if (valid < kSub) {
#pragma unroll
          for (int i = 0; i < kSub; ++i)
            if (i >= valid) s[i] = -INFINITY;
        }
        float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int i = 4; i < kSub; i += 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = i + 4 < kSub ? fmax3_nan(mx[k], s[i + k], s[i + 4 + k]) : fmax_nan(mx[k], s[i + k]);
        }
        mx[0] = fmax3_nan(mx[0], mx[1], fmax_nan(mx[2], mx[3]));
        // The reference moves only when the maximum exceeds it by 2^8, so the
        // accumulator is rarely rescaled and P stays <= 256; for NaN it moves to
        // +infinity, once.
        const bool move = !(mx[0] * kC2 <= m_ref + 8.0f) && m_ref < INFINITY;
        if (__any_sync(0xffffffffu, move)) {
          const float m_new = move ? fminf(mx[0] * kC2, INFINITY) : m_ref;  // (fminf drops a NaN)
          if (j > 0) {
            // (P V of tile j - 3 was done before these scores: the parity is the last one's)
            ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1));
            if (ok) {
              tc_fence_after();
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
          }
          m_ref = m_new;
        }
        uint32_t pk[kSub / 2];
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kSub; i += 2) {
          const float2 x = ffma2(make_float2(s[i], s[i + 1]), make_float2(kC2, kC2), make_float2(-m_ref, -m_ref));
          const float2 p = i % 8 == 0 ? exp2_poly(x) : exp2_unit(x);  // (a quarter, see exp2_poly)
          sum[(i >> 1) & 1] = fadd2(sum[(i >> 1) & 1], p);
          pk[i / 2] = pack2<BF16>(p.x, p.y);
        }
        sum[0] = fadd2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        // over the first half of the columns, which were read above
        tmem_st16_u32(cols, *reinterpret_cast<const uint32_t(*)[16]>(pk));
        tmem_st16_u32(cols + 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[j % 3]);
    }
    // The last two products in order: these scores say only that P V of tile
    // nkv - 4 is done, and a warp may be two tiles ahead of another, so the parity of
    // the last product's barrier alone could still be that of tile nkv - 5.
    if (ok && nkv > 1) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[nkv & 1], ((nkv - 2) >> 1) & 1));
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&pv_done[(nkv - 1) & 1], ((nkv - 1) >> 1) & 1));
    const int t = qt * 128 + r;
    if (ok) {
      tc_fence_after();
      const bool live = t < len;
      if (!(fabsf(m_ref) < -kLowest)) l = __int_as_float(0x7fffffff);
      const float inv = live ? 1.0f / l : 0.f;
#pragma unroll
      for (int c0 = 0; c0 < kHd; c0 += 32)  // over Q, which nothing reads any more
        stage_row_part<BF16>(tO + lane_base + c0, smem + FwdSmem::Q, r, c0 / 8, inv, live);
      if (t < T) lse[bh * T + t] = live ? m_ref * kLn2 + logf(l) : -INFINITY;
    } else if (lane == 0) {
      atomicOr(err, kErrWaitSoftmax);
    }
    named_barrier_sync(1, 128);
    store_tile(smem + FwdSmem::Q, out + b * out_bs + static_cast<int64_t>(qt) * 128 * out_ld + h * kHd, out_ld,
               min(128, T - qt * 128), threadIdx.x, 128);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// -------------------------------------------------- backward: row statistics
// The statistics of a row reach S and dP inside the products: 16 more channels on
// each side, a row's pieces against constants, make
//   S = q k^T - 8 lse,   dP = dout v^T - rowsum(dout o out)
// in the fp32 accumulator.  Without them every thread of a key CTA read two
// statistics per column from shared memory (16 wide loads and 16 additions per 32
// columns, a quarter of its time).  A value is split into three pieces of the
// operand type, hi + mid + lo, each the rounding of what is left.  In bf16 that is
// all of an fp32's 24 bits.  In fp16 it is too until a piece reaches the subnormal
// step, so the error is absolute: 2^-25 c for a constant c.  fp16's range is widened by
// groups of three channels with different constants, of which a value uses the first
// where value / c fits:
//   8 lse:  64 (up to 2^21), 2^15
//   rowsum: 2^-24 (up to 2^-10), 2^-14 (1), 2^-4 (2^10), 2^6 (2^20), 2^15
// From the second group on 2^-25 c is below 2^-28 of the value.  8 lse is off by at
// most 2^-19 in the first, whatever its size, and a probability by 2^-22 of itself,
// since lse is added to its exponent; a row sum by 2^-49, less than the smallest
// product of two fp16 values that dP is a sum of.  Past 65504 * 2^15 a value has no
// pieces: the row's gradients are not finite.
// Rows that carry nothing get lse = infinity, so that their probabilities are 0.
//
// Layout, per (clip, head): rows padded to a multiple of 128, in the unswizzled
// K-major core-matrix order [8 rows][2][8][16 bytes], so that any multiple of 8
// rows is one contiguous operand.
constexpr int kAugRow = 32;                       // bytes: 16 channels
constexpr uint32_t kAugLbo = 128, kAugSbo = 256;  // next 8 channels, next 8 rows

__device__ __forceinline__ int aug_offset(int row, int half) { return (row >> 3) * 256 + half * 128 + (row & 7) * 16; }

// The constants of channels 8 half .. 8 half + 7.
template <bool BF16>
__device__ __forceinline__ uint4 aug_constants(bool rowsum, int half) {
  if (BF16) return half ? make_uint4(0, 0, 0, 0) : make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
  // fp16 bits: 64 = 5400, 2^15 = 7800, 2^-24 = 0001, 2^-14 = 0400, 2^-4 = 2C00, 2^6 = 5400
  if (!rowsum) return half ? make_uint4(0, 0, 0, 0) : make_uint4(0x54005400u, 0x78005400u, 0x78007800u, 0);
  return half ? make_uint4(0x54002C00u, 0x54005400u, 0x78007800u, 0x00007800u)
              : make_uint4(0x00010001u, 0x04000001u, 0x04000400u, 0x2C002C00u);
}

// Channels 8 half .. 8 half + 7 of value v (v = -infinity: hi = -infinity).
template <bool BF16>
__device__ __forceinline__ uint4 aug_pieces(float v, bool rowsum, int half) {
  int group = 0;
  float x = v;
  if (!BF16) {
    const float m = fabsf(v);
    if (rowsum) {
      group = m <= 0x1p-10f ? 0 : m <= 1.0f ? 1 : m <= 0x1p10f ? 2 : m <= 0x1p20f ? 3 : 4;
      const float inv = group == 0 ? 0x1p24f : group == 1 ? 0x1p14f : group == 2 ? 0x1p4f : group == 3 ? 0x1p-6f : 0x1p-15f;
      x = v * inv;
    } else {
      group = m <= 0x1p21f || v == -INFINITY ? 0 : 1;
      x = v * (group == 0 ? 0x1p-6f : 0x1p-15f);
    }
  }
  float r[3];
  r[0] = unpack2<BF16>(pack2<BF16>(x, 0.f)).x;
  const float rest = v == -INFINITY ? 0.f : x - r[0];
  r[1] = unpack2<BF16>(pack2<BF16>(rest, 0.f)).x;
  r[2] = rest - r[1];
  float ch[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int piece = half * 8 + i - 3 * group;
    ch[i] = piece == 0 ? r[0] : piece == 1 ? r[1] : piece == 2 ? r[2] : 0.f;
  }
  return make_uint4(pack2<BF16>(ch[0], ch[1]), pack2<BF16>(ch[2], ch[3]), pack2<BF16>(ch[4], ch[5]),
                    pack2<BF16>(ch[6], ch[7]));
}

struct BwdOut {
  uint16_t* dq;
  uint16_t* dk;
  uint16_t* dv;
  int64_t ld, bs;
};

// In fp16 also, per 128 frames, the largest |dout row|^2 and |v row|^2.  Tiles of
// padded rows alone get their zero gradients here.
// Eight lanes a row, 16 bytes each.
template <bool BF16>
__global__ void __launch_bounds__(256)
attention_bwd_rows_kernel(const uint16_t* __restrict__ dout, const uint16_t* __restrict__ out, int64_t out_ld,
                          int64_t out_bs, const uint16_t* __restrict__ v, int64_t v_ld, int64_t v_bs,
                          const float* __restrict__ lse, const int32_t* __restrict__ frames, int T, int H, int tiles,
                          uint8_t* __restrict__ aug_l, uint8_t* __restrict__ aug_d, float2* __restrict__ peak,
                          const BwdOut g) {
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int tile = blockIdx.x % tiles, bh = blockIdx.x / tiles;
  const int b = bh / H, h = bh % H;
  const int part = threadIdx.x & 7;
  pdl_wait();
  const int len = clip_frames(frames, b, T);
  if (tile * 128 >= len) {  // rows past the clip: their gradients are written here, the rest is not asked for
    const int to = min(T, tile * 128 + 128);
    const int64_t at = b * g.bs + h * kHd;
    zero_rows(g.dq + at, g.ld, tile * 128, to);
    zero_rows(g.dk + at, g.ld, tile * 128, to);
    zero_rows(g.dv + at, g.ld, tile * 128, to);
    if (!BF16 && threadIdx.x == 0) peak[static_cast<int64_t>(bh) * tiles + tile] = make_float2(0.f, 0.f);
    return;
  }
  float top_do = 0.f, top_v = 0.f;
  // every load of the thread's four rows before any arithmetic
  uint4 ra[4], ro[4], rv[4];
  float rl[4];
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int t = tile * 128 + it * 32 + (threadIdx.x >> 3);
    ra[it] = ro[it] = rv[it] = make_uint4(0, 0, 0, 0);
    rl[it] = -INFINITY;
    if (t < len) {
      const int64_t at = b * out_bs + t * out_ld + h * kHd + part * 8;
      ra[it] = *reinterpret_cast<const uint4*>(dout + at);
      ro[it] = *reinterpret_cast<const uint4*>(out + at);
      if (!BF16) rv[it] = *reinterpret_cast<const uint4*>(v + b * v_bs + t * v_ld + h * kHd + part * 8);
      rl[it] = lse[static_cast<int64_t>(bh) * T + t];
    }
  }
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int t = tile * 128 + it * 32 + (threadIdx.x >> 3);
    float d = 0.f, ndo = 0.f, nv = 0.f;
    const uint32_t au[4] = {ra[it].x, ra[it].y, ra[it].z, ra[it].w}, ou[4] = {ro[it].x, ro[it].y, ro[it].z, ro[it].w};
    const uint32_t wu[4] = {rv[it].x, rv[it].y, rv[it].z, rv[it].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = unpack2<BF16>(au[i]), y = unpack2<BF16>(ou[i]), z = unpack2<BF16>(wu[i]);
      d = fmaf(x.x, y.x, fmaf(x.y, y.y, d));
      if (!BF16) {
        ndo = fmaf(x.x, x.x, fmaf(x.y, x.y, ndo));
        nv = fmaf(z.x, z.x, fmaf(z.y, z.y, nv));
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
    if (part < 4) {
      const bool rowsum = part >= 2;
      const float value = rowsum ? -d : (rl[it] == -INFINITY ? -INFINITY : -8.0f * rl[it]);
      uint8_t* dst = (rowsum ? aug_d : aug_l) + (static_cast<int64_t>(bh) * tiles + tile) * 128 * kAugRow;
      *reinterpret_cast<uint4*>(dst + aug_offset(it * 32 + (threadIdx.x >> 3), part & 1)) =
          aug_pieces<BF16>(value, rowsum, part & 1);
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

// Exponent of the scale of dS in fp16: |dS_ij| <= P_ij |dout_i| |v_j - out_i|
// <= 2 max|dout| max|v| (out_i is a mean of v rows), so with that bound brought
// just under 2^15 no entry overflows and the smallest keep what precision fp16
// can give them.  Every thread of the warp gets the same value.
__device__ __forceinline__ int ds_exponent(float top_do, float top_v) {
  const float bound = 2.0f * sqrtf(top_do) * sqrtf(top_v);
  if (!(bound > 0.f) || !(bound < INFINITY)) return 0;
  return max(-100, min(100, 14 - ilogbf(bound)));
}

__device__ __forceinline__ int ds_exponent(const float2* peak, int tiles, int lane) {
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
  return ds_exponent(top_do, top_v);
}

// ------------------------------------------------------------------- backward
// Sums over the warp of 16 values a lane: every two lanes get one value's, in order.
__device__ __forceinline__ float column_sums(float (&v)[16], int lane) {
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {
    const bool up = lane & (2 * n);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + n], 2 * n);
      v[i] = (up ? v[i + n] : v[i]) + other;
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 1);
}

// Two kinds of CTA in one launch, with the same inner step.  A CTA holds 128
// rows of a pair of operands (A1, A2) and streams 64-row tiles of the other
// pair (B1, B2), each with its 16 statistics channels; per tile
//   S = A1 B1^T, dP = A2 B2^T             (M = 128, N = 64, K = 64 + 16)
//   P = 2^(S c), dS = P o dP
// A key CTA holds (K, V) and streams (Q, dO); its S, P and dS are transposed
// (row = key) and, rounded to the operand type, the A operands of
//   dV += P dO, dK += dS Q                 (M = 128, N = 64, K = 64 queries).
// A query CTA holds (Q, dO), streams (K, V) and sums dQ += dS K and P K.  A row of dS
// sums to zero; what the rounded one sums to, r, is the error of rowsum(dO o out),
// which has the rounding of out, and the sum of its own entries' roundings, all nearly
// in proportion to P: so dQ - r (P K) is what it writes.  dq is then off by 1.31-1.36
// times one rounding of the exact result, and was by 1.53-1.66 without, at 49 to 2999
// frames; 2 x 2999 frames x 16 heads take 315 us for 288, 799 x 12 25.4 for 22.8.  dk has the error of
// the row sums of other CTAs' rows and stays at 1.44-1.6; in a clip of one tile of 64,
// where it can be many times that, both kinds of CTA see whole rows of P o dP and take
// their sum off first (49 x 12: 6.6 us for 5.9; dk 1.42 for 1.6).  S and dP
// are computed twice, which costs 8 products instead of the 5 of a single pass,
// but each gradient has one owner that sums it in a fixed order: no atomics and no
// fp32 partial sums in memory.
//
// Warps 0-7: one TMEM lane quarter and 32 of the 64 columns each; they pack dS and
// P together over the dP columns that they have read, so the S columns are free
// for the next tile as soon as they are read.  Warp 8: TMA; warp 9: tensor memory
// and products.  256 tensor-memory columns and 100 KB of shared memory: two CTAs
// per SM fill each other's gaps.
struct BwdSmem {
  static constexpr int kStages = 3;
  static constexpr int A = 0;                      // A1, A2 (128 rows each); at the end the gradients' tiles
  static constexpr int B = 4 * kTileBytes;         // [stages]{B1, B2}
  static constexpr int AugA = B + kStages * 2 * kTileBytes;  // {lse, rowsum} channels of A's 128 rows
  static constexpr int AugB = AugA + 2 * 128 * kAugRow;      // [stages]{lse, rowsum} of the streamed rows
  static constexpr int kAugTile = kSub * kAugRow;
  static constexpr int BAR = AugB + kStages * 2 * kAugTile;
  static constexpr int TOTAL = BAR + 256 + 1024;  // barriers and the TMEM address, then (at 192) 64 bytes of reductions
};
constexpr int kBwdThreads = 320;

struct BwdArgs {
  BwdOut g;
  const int32_t* frames;
  const uint8_t* aug_l;
  const uint8_t* aug_d;
  const float2* peak;
  int T, H, batch, tiles;
  int* err;
  // For T <= 128 a CTA makes the statistics of its clip itself (they are one tile's)
  // and no other kernel runs before this one (49 frames x 12 heads: one launch and
  // 2 us less); null otherwise.
  const uint16_t* dout;
  const uint16_t* out;
  const uint16_t* v;
  const float* lse;
  int64_t out_ld, out_bs, v_ld, v_bs;
};

// The statistics of one clip of at most 128 frames, as attention_bwd_rows_kernel
// makes them, straight into shared memory: two threads a row (warps 0-7).  Returns
// the exponent of dS's scale.
template <bool BF16, bool KEYS>
__device__ __forceinline__ int own_statistics(const BwdArgs& a, uint8_t* smem, int b, int h, int len) {
  float* red = reinterpret_cast<float*>(smem + BwdSmem::BAR + 192);  // [8 warps]{dout, v}
  const int row = threadIdx.x >> 1, part = threadIdx.x & 1;
  float top_do = 0.f, top_v = 0.f;
  if (threadIdx.x < 256) {
    float d = 0.f, l = -INFINITY;
    if (row < len) {
      const int64_t at = b * a.out_bs + row * a.out_ld + h * kHd + part * 32;
      const int64_t va = b * a.v_bs + row * a.v_ld + h * kHd + part * 32;
#pragma unroll
      for (int c = 0; c < 32; c += 8) {
        const uint4 x4 = *reinterpret_cast<const uint4*>(a.dout + at + c);
        const uint4 y4 = *reinterpret_cast<const uint4*>(a.out + at + c);
        uint4 z4 = make_uint4(0, 0, 0, 0);
        if (!BF16) z4 = *reinterpret_cast<const uint4*>(a.v + va + c);
        const uint32_t xu[4] = {x4.x, x4.y, x4.z, x4.w}, yu[4] = {y4.x, y4.y, y4.z, y4.w};
        const uint32_t zu[4] = {z4.x, z4.y, z4.z, z4.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<BF16>(xu[i]), y = unpack2<BF16>(yu[i]), z = unpack2<BF16>(zu[i]);
          d = fmaf(x.x, y.x, fmaf(x.y, y.y, d));
          if (!BF16) {
            top_do = fmaf(x.x, x.x, fmaf(x.y, x.y, top_do));
            top_v = fmaf(z.x, z.x, fmaf(z.y, z.y, top_v));
          }
        }
      }
      l = a.lse[(static_cast<int64_t>(b) * a.H + h) * a.T + row];
    }
    d += __shfl_xor_sync(0xffffffffu, d, 1);
    const float value = part ? -d : (l == -INFINITY ? -INFINITY : -8.0f * l);
    uint8_t* dst = KEYS ? smem + BwdSmem::AugB + (row >> 6) * 2 * BwdSmem::kAugTile + part * BwdSmem::kAugTile
                        : smem + BwdSmem::AugA + part * 128 * kAugRow;
    const int at = KEYS ? row & 63 : row;
#pragma unroll
    for (int half = 0; half < 2; ++half)
      *reinterpret_cast<uint4*>(dst + aug_offset(at, half)) = aug_pieces<BF16>(value, part, half);
    if (!BF16) {
      top_do += __shfl_xor_sync(0xffffffffu, top_do, 1);
      top_v += __shfl_xor_sync(0xffffffffu, top_v, 1);
#pragma unroll
      for (int o = 2; o < 32; o <<= 1) {
        top_do = fmaxf(top_do, __shfl_xor_sync(0xffffffffu, top_do, o));
        top_v = fmaxf(top_v, __shfl_xor_sync(0xffffffffu, top_v, o));
      }
      if ((threadIdx.x & 31) == 0) {
        red[threadIdx.x >> 4] = top_do;
        red[(threadIdx.x >> 4) + 1] = top_v;
      }
      named_barrier_sync(1, 256);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        top_do = fmaxf(top_do, red[2 * i]);
        top_v = fmaxf(top_v, red[2 * i + 1]);
      }
    }
  }
  return BF16 ? 0 : ds_exponent(top_do, top_v);
}

template <bool BF16, bool KEYS>
__device__ __forceinline__ void bwd_body(const CUtensorMap& tmA1, const CUtensorMap& tmA2, const CUtensorMap& tmB1,
                                         const CUtensorMap& tmB2, const BwdArgs& a, int u) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BwdSmem::BAR);
  uint64_t* a_full = bars;
  uint64_t* s_full = bars + 1;
  uint64_t* dp_full = bars + 2;
  uint64_t* s_read = bars + 3;
  uint64_t* ds_full = bars + 4;
  uint64_t* acc_done = bars + 5;
  uint64_t* b_full = bars + 6;
  uint64_t* b_empty = bars + 6 + BwdSmem::kStages;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 6 + 2 * BwdSmem::kStages);

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const Unit unit = find_unit(a.frames, a.batch, a.T, a.H, a.tiles, u, lane);
  const int b = unit.b, h = unit.h, tile = unit.tile, len = unit.len;
  const int64_t bh = static_cast<int64_t>(b) * a.H + h;
  const int n_sub = (len + kSub - 1) / kSub;
  if (tile * 128 >= len) {  // padded rows, in a batch that is taken as it comes or (own statistics) an empty clip
    if (a.dout) {
      const int64_t at = b * a.g.bs + h * kHd;
      zero_rows((KEYS ? a.g.dk : a.g.dq) + at, a.g.ld, 0, a.T);
      if (KEYS) zero_rows(a.g.dv + at, a.g.ld, 0, a.T);
    }
    return;
  }

  auto load_tile = [&](int j) {
    const int st = j % BwdSmem::kStages;
    uint8_t* dst = smem + BwdSmem::B + st * 2 * kTileBytes;
    mbar_arrive_expect_tx(&b_full[st], 2 * kTileBytes + (KEYS && !a.dout ? 2 * BwdSmem::kAugTile : 0));
    tma_load_3d(dst, &tmB1, &b_full[st], h * kHd, j * kSub, b);
    tma_load_3d(dst + kTileBytes, &tmB2, &b_full[st], h * kHd, j * kSub, b);
    if (KEYS && !a.dout) {
      uint8_t* aug = smem + BwdSmem::AugB + st * 2 * BwdSmem::kAugTile;
      const int64_t at = bh * a.tiles * 128 * kAugRow + j * BwdSmem::kAugTile;
      bulk_load(aug, a.aug_l + at, BwdSmem::kAugTile, &b_full[st]);
      bulk_load(aug + BwdSmem::kAugTile, a.aug_d + at, BwdSmem::kAugTile, &b_full[st]);
    }
  };
  // The copying thread sets up the barriers and starts the first copies before the
  // others have the tensor memory.
  if (threadIdx.x == 8 * 32) {
    mbar_init(a_full, 1);
    mbar_init(s_read, 8);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(ds_full, 8);
    mbar_init(acc_done, 1);
    for (int i = 0; i < BwdSmem::kStages; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    fence_mbar_init();
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(a_full, 4 * kTileBytes + (KEYS || a.dout ? 0 : 2 * 128 * kAugRow));
    for (int i = 0; i < 2; ++i) {
      tma_load_3d(smem + BwdSmem::A + i * kTileBytes, &tmA1, a_full, h * kHd, tile * 128 + i * kSub, b);
      tma_load_3d(smem + BwdSmem::A + (2 + i) * kTileBytes, &tmA2, a_full, h * kHd, tile * 128 + i * kSub, b);
    }
    if (!KEYS && !a.dout) {
      const int64_t at = (bh * a.tiles + tile) * 128 * kAugRow;
      bulk_load(smem + BwdSmem::AugA, a.aug_l + at, 128 * kAugRow, a_full);
      bulk_load(smem + BwdSmem::AugA + 128 * kAugRow, a.aug_d + at, 128 * kAugRow, a_full);
    }
    for (int j = 0; j < min(n_sub, BwdSmem::kStages); ++j) load_tile(j);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 256);
    tmem_relinquish();
  }
  // The constants that the other side's pieces meet: A's in a key CTA, one tile of
  // B's in a query CTA.
  for (int i = threadIdx.x; i < (KEYS ? 128 : kSub) * 4; i += kBwdThreads) {
    const int row = i >> 2, half = i & 1, rowsum = (i >> 1) & 1;
    uint8_t* dst = KEYS ? smem + BwdSmem::AugA + rowsum * 128 * kAugRow : smem + BwdSmem::AugB + rowsum * BwdSmem::kAugTile;
    *reinterpret_cast<uint4*>(dst + aug_offset(row, half)) = aug_constants<BF16>(rowsum, half);
  }
  int e = 0;  // of dS's scale (see below)
  if (a.dout) {
    e = own_statistics<BF16, KEYS>(a, smem, b, h, len);
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = uniform(*tmem_slot);
  // dV or P K | dK or dQ | S | dP, then dS and P
  const uint32_t tAcc1 = tmem, tAcc2 = tmem + 64, tS = tmem + 128, tD = tmem + 192;
  if (threadIdx.x == 0) pdl_launch_dependents();

  if (warp == 8) {
    if (lane == 0) {
      for (int j = BwdSmem::kStages; j < n_sub; ++j) {
        if (!mbar_wait(&b_empty[j % BwdSmem::kStages], ((j / BwdSmem::kStages) & 1) ^ 1)) {
          atomicOr(a.err, kErrWaitProducer);
          // wait for the copies in flight before the CTA's shared memory goes
          mbar_wait(a_full, 0);
          for (int i = j - BwdSmem::kStages; i < j; ++i)
            mbar_wait(&b_full[i % BwdSmem::kStages], (i / BwdSmem::kStages) & 1);
          break;
        }
        load_tile(j);
      }
    }
  } else if (warp == 9) {
    constexpr uint32_t idS = idesc_train<BF16>(128, kSub, false);
    constexpr uint32_t idG = idesc_train<BF16>(128, kHd, true);
    const uint64_t dA1 = desc_sw128(smem_u32(smem + BwdSmem::A));
    const uint64_t dA2 = desc_sw128(smem_u32(smem + BwdSmem::A + 2 * kTileBytes));
    const uint64_t dB = desc_sw128(smem_u32(smem + BwdSmem::B));
    const uint64_t dAugA = smem_desc(smem_u32(smem + BwdSmem::AugA), kAugLbo, kAugSbo, kSwizzleNone);
    const uint64_t dAugB = smem_desc(smem_u32(smem + BwdSmem::AugB), kAugLbo, kAugSbo, kSwizzleNone);
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
    // rowsum = 0: S of tile j, 1: dP
    auto scores = [&](int j, int rowsum) {
      tc_fence_after();
      if (elect_one()) {
        const uint32_t d = rowsum ? tD : tS;
        const uint64_t da = rowsum ? dA2 : dA1, db = rowsum ? tile_b2(j) : tile_b1(j);
        const int st = KEYS ? j % BwdSmem::kStages : 0;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f16(d, da + 2 * kk, db + 2 * kk, idS, kk);
        umma_f16(d, dAugA + static_cast<uint64_t>(rowsum * (128 * kAugRow >> 4)),
                 dAugB + static_cast<uint64_t>((2 * st + rowsum) * (BwdSmem::kAugTile >> 4)), idS, 1);
        umma_commit(rowsum ? dp_full : s_full);
      }
      __syncwarp();
    };
    // Products over the streamed rows, 16 (2048 bytes of the tile) a step.  Of
    // columns 32 w .. 32 w + 31 of dP, dS lies packed in the first 16 and P in the
    // others, so a product's steps start at 0, 8, 32 and 40 from its first.
    auto accumulate = [&](int j) {
      tc_fence_after();
      if (elect_one()) {
        const uint64_t db1 = tile_b1(j), db2 = tile_b2(j);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tAcc2, tD + 32 * (kk >> 1) + 8 * (kk & 1), db1 + static_cast<uint64_t>(128 * kk), idG,
                      (j > 0 || kk > 0) ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_f16_ts(tAcc1, tD + 16 + 32 * (kk >> 1) + 8 * (kk & 1),
                      (KEYS ? db2 : db1) + static_cast<uint64_t>(128 * kk), idG, (j > 0 || kk > 0) ? 1u : 0u);
        umma_commit(acc_done);
        umma_commit(&b_empty[j % BwdSmem::kStages]);
      }
      __syncwarp();
    };
    auto wait = [&](uint64_t* bar, int j) { return __all_sync(0xffffffffu, mbar_wait(bar, j & 1)); };
    bool ok = __all_sync(0xffffffffu, mbar_wait(a_full, 0)) && wait_tile(0);
    if (ok) {
      scores(0, 0);
      scores(0, 1);
    }
    // The next tile's scores run as soon as this tile's have been read, and its dP
    // once the products of this tile's dS and P, which lie over dP, are done: both
    // under the elementwise work.
    for (int j = 0; ok && j < n_sub; ++j) {
      const bool more = j + 1 < n_sub;
      if (more) {
        if (!(ok = wait(s_read, j) && wait_tile(j + 1))) break;
        scores(j + 1, 0);
      }
      if (!(ok = wait(ds_full, j))) break;
      accumulate(j);
      if (more) {
        if (!(ok = wait(acc_done, j))) break;
        scores(j + 1, 1);
      }
    }
    if (!ok && lane == 0) atomicOr(a.err, kErrWaitMma);
  } else {
    const int quarter = warp & 3, half = warp >> 2;
    const int row = quarter * 32 + lane, t = tile * 128 + row;
    const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
    // fp16: dS is scaled by 2^(up + down).  Up to 2^15 of it goes into P (which is
    // at most 1, and is as exact scaled as unscaled), and so into dV too; what
    // shrinks dS is a factor of its own.
    if (!BF16 && !a.dout) e = ds_exponent(a.peak + bh * a.tiles, a.tiles, lane);
    const int up = max(0, min(15, e)), down = min(0, e);
    const float unscale = exp2f(static_cast<float>(-up));
    const float shift = static_cast<float>(up), shrink = exp2f(static_cast<float>(down));
    float2 left = make_float2(0.f, 0.f);  // query CTA: the sum of the row's dS as rounded
    bool ok = true;
    for (int j = 0; j < n_sub; ++j) {
      const int valid = len - j * kSub - half * 32;
      float s[32];
      uint32_t pk[32];  // dS, then P
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(s_full, j & 1));
      if (ok) {
        tc_fence_after();
        tmem_ld32(tS + lane_base + half * 32, s);
      }
      tc_fence_before();  // S has been read: its columns are free for the next tile's
      __syncwarp();
      if (lane == 0) mbar_arrive(s_read);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 p =
            exp2_unit(ffma2(make_float2(s[i], s[i + 1]), make_float2(kC2, kC2), make_float2(shift, shift)));
        s[i] = p.x;
        s[i + 1] = p.y;
      }
      // Columns past the clip.  A query CTA's scores of such keys are -8 lse, not -infinity,
      // and may overflow; a key CTA's of such queries are -infinity, but NaN where the key
      // holds an infinity (times the zeros of the query), and NaN would reach dV and dK.
      if (valid < 32) {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i >= valid) s[i] = 0.f;
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(dp_full, j & 1));
      // A clip of one tile of 64 frames: what its rows of P o dP sum to is taken off dP
      // before dS is rounded (in a longer clip only dQ is put right, at the end).
      float* rest = reinterpret_cast<float*>(smem + BwdSmem::B + 2 * kTileBytes);  // (a stage that it does not use)
      float own_rest = 0.f;
      if (n_sub == 1) {
        if (ok) {
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < 32; c0 += 16) {
            float g[16];
            tmem_ld16(tD + lane_base + half * 32 + c0, g);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              g[i] = !KEYS || t < len ? g[i] * s[c0 + i] : 0.f;
              if (!KEYS) own_rest += g[i];
            }
            if (KEYS) {
              const float sum = column_sums(g, lane);
              if (quarter < 2) rest[quarter * 64 + half * 32 + c0 + (lane >> 1)] = sum * unscale;
            }
          }
          if (!KEYS) rest[half * 128 + row] = own_rest * unscale;
        }
        named_barrier_sync(1, 256);
        if (!KEYS) own_rest = rest[row] + rest[128 + row];
      }
      if (ok) {
        tc_fence_after();
#pragma unroll
        for (int c0 = 0; c0 < 32; c0 += 16) {
          float dp[16];
          tmem_ld16(tD + lane_base + half * 32 + c0, dp);
          if (n_sub == 1) {
#pragma unroll
            for (int i = 0; i < 16; ++i)
              dp[i] -= KEYS ? rest[half * 32 + c0 + i] + rest[64 + half * 32 + c0 + i] : own_rest;
          }
          if (!BF16 && down < 0) {
#pragma unroll
            for (int i = 0; i < 16; ++i) dp[i] *= shrink;
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float2 g = fmul2(make_float2(dp[i], dp[i + 1]), make_float2(s[c0 + i], s[c0 + i + 1]));
            pk[(c0 + i) / 2] = pack2<BF16>(g.x, g.y);
            if (!KEYS) left = fadd2(left, unpack2<BF16>(pk[(c0 + i) / 2]));
          }
        }
        tmem_st16_u32(tD + lane_base + half * 32, *reinterpret_cast<const uint32_t(*)[16]>(pk));
#pragma unroll
        for (int i = 0; i < 32; i += 2) pk[16 + i / 2] = pack2<BF16>(s[i], s[i + 1]);
        tmem_st16_u32(tD + lane_base + half * 32 + 16, *reinterpret_cast<const uint32_t(*)[16]>(pk + 16));
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(ds_full);
    }
    if (ok) ok = __all_sync(0xffffffffu, mbar_wait(acc_done, (n_sub - 1) & 1));
    if (!KEYS) {  // both column halves' sums of the row
      float* sums = reinterpret_cast<float*>(smem + BwdSmem::A + 2 * kTileBytes);
      if (ok) sums[half * 128 + row] = left.x + left.y;
      named_barrier_sync(1, 256);
      if (ok) left.x = sums[row] + sums[128 + row];
    }
    if (ok) {
      tc_fence_after();
      const bool live = t < len;
      // A single frame has P = 1 and no gradient through the softmax: dP and
      // rowsum(dO o O) are the same number there, summed in two orders.
      const float back = len == 1 ? 0.f : 0.125f * unscale * exp2f(static_cast<float>(-down));
      // over A1 and A2, which no product reads any more
      if (KEYS) {
        stage_row_part<BF16>(tAcc2 + lane_base + half * 32, smem + BwdSmem::A, row, half * 4, back, live);
        stage_row_part<BF16>(tAcc1 + lane_base + half * 32, smem + BwdSmem::A + 2 * kTileBytes, row, half * 4, unscale,
                             live);
      } else {
        stage_row_difference<BF16>(tAcc2 + lane_base + half * 32, tAcc1 + lane_base + half * 32, smem + BwdSmem::A, row,
                                   half * 4, back, left.x * unscale, live);
      }
    } else if (lane == 0) {
      atomicOr(a.err, kErrWaitSoftmax);
    }
    named_barrier_sync(1, 256);
    const int rows = min(128, a.T - tile * 128);
    const int64_t at = b * a.g.bs + static_cast<int64_t>(tile) * 128 * a.g.ld + h * kHd;
    store_tile(smem + BwdSmem::A, (KEYS ? a.g.dk : a.g.dq) + at, a.g.ld, rows, threadIdx.x, 256);
    if (KEYS) store_tile(smem + BwdSmem::A + 2 * kTileBytes, a.g.dv + at, a.g.ld, rows, threadIdx.x, 256);
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
  // In this order: key CTAs (the longer ones) and query CTAs of tiles with frames,
  // and CTAs with nothing to do (the grid is for full clips).
  int live = a.tiles * a.batch * a.H;
  pdl_wait();  // before tensor memory is asked for, as in the forward kernel
  if (a.frames) live = live_units(a.frames, a.batch, a.T, a.H, live, threadIdx.x & 31);
  // (with its own statistics the kernel also writes the zeros of empty clips: there
  // the units without frames follow, key units first)
  const int u = blockIdx.x, units = a.tiles * a.batch * a.H;
  if (u >= 2 * live && !a.dout) return;
  if (u < live || (u >= 2 * live && u < units + live))
    bwd_body<BF16, true>(tmK, tmV, tmQ, tmDo, a, u < live ? u : u - live);
  else
    bwd_body<BF16, false>(tmQ, tmDo, tmK, tmV, a, u < 2 * live ? u - live : u - units);
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
                    s.T, s.H, s.batch, tiles, static_cast<uint16_t*>(out), s.out_ld, s.out_bs, lse, err);
}

size_t attention_bwd_ws_bytes(int batch, int T, int H) {
  const size_t tiles = (static_cast<size_t>(T) + 127) / 128, bh = static_cast<size_t>(batch) * H;
  if (tiles == 1) return 0;  // the statistics stay in shared memory
  return bh * tiles * (128 * 2 * kAugRow + sizeof(float2));
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
  uint8_t* aug_l = static_cast<uint8_t*>(ws);
  uint8_t* aug_d = aug_l + rows * kAugRow;
  float2* peak = reinterpret_cast<float2*>(aug_d + rows * kAugRow);
  auto u16 = [](const void* p) { return static_cast<const uint16_t*>(p); };
  BwdArgs a;
  a.g = {static_cast<uint16_t*>(dq), static_cast<uint16_t*>(dk), static_cast<uint16_t*>(dv), s.grad_ld, s.grad_bs};
  const bool own = tiles == 1;
  if (!own) {
    r = launch_pdl(s.bf16 ? attention_bwd_rows_kernel<true> : attention_bwd_rows_kernel<false>, dim3(tiles * bh),
                   dim3(256), 0, st, u16(dout), u16(out), s.out_ld, s.out_bs, u16(v), s.qkv_ld, s.qkv_bs, lse,
                   s.frames, s.T, s.H, tiles, aug_l, aug_d, peak, a.g);
    if (r != cudaSuccess) return r;
  }
  a.dout = own ? u16(dout) : nullptr;
  a.out = u16(out);
  a.v = u16(v);
  a.lse = lse;
  a.out_ld = s.out_ld; a.out_bs = s.out_bs;
  a.v_ld = s.qkv_ld; a.v_bs = s.qkv_bs;
  a.frames = s.frames;
  a.aug_l = aug_l;
  a.aug_d = aug_d;
  a.peak = peak;
  a.T = s.T; a.H = s.H; a.batch = s.batch; a.tiles = tiles;
  a.err = err;
  auto kernel = s.bf16 ? attention_bwd_kernel<true> : attention_bwd_kernel<false>;
  if ((r = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, BwdSmem::TOTAL)) != cudaSuccess)
    return r;
  return launch_pdl(kernel, dim3(2 * tiles * bh), dim3(kBwdThreads), BwdSmem::TOTAL, st, tq, tk, tv, td, a);
}

}  // namespace w2v
