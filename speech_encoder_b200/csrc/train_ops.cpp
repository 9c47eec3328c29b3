// C ABI of the operators for training (w2v_train.h): argument checks, then the
// kernel launches of k_attention_train.cu, k_layernorm_train.cu and
// k_grad_clip.cu.
#include "w2v_train.h"

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "extent.h"
#include "w2v.h"
#include "w2v_internal.h"

using namespace w2v;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int status(cudaError_t e) { return e == cudaSuccess ? W2V_OK : W2V_ECUDA; }

// Row and clip strides of one set of operands: multiples of 16 bytes, rows of
// `width` elements apart from one another whichever of the two strides is the
// longer.  A stride of an axis with a single entry is not used.
bool strides_ok(int64_t* ld, int64_t* bs, int64_t T, int64_t batch, int64_t width) {
  constexpr int64_t kMost = int64_t(1) << 38;  // a tensor map's strides stay below 2^40 bytes
  if (T == 1) *ld = width;
  if (batch == 1) *bs = T * std::max(*ld, width);
  if (*ld < width || *bs < width || *ld % 8 != 0 || *bs % 8 != 0 || *ld > kMost || *bs > kMost) return false;
  if (T == 1 || batch == 1) return true;
  return *bs >= (T - 1) * *ld + width || *ld >= (batch - 1) * *bs + width;
}

int attention_args(const w2v_attention_shape* s, bool grads, AttnTrain* a) {
  if (!s) return W2V_EINVAL;
  if (s->dtype != W2V_F16 && s->dtype != W2V_BF16) return W2V_EINVAL;
  if (s->batch < 1 || s->T < 1 || s->H < 1 || s->T >= (1 << 24) || s->H > (1 << 24)) return W2V_ESHAPE;
  const int64_t tiles = (static_cast<int64_t>(s->T) + 127) / 128;
  const int64_t heads = static_cast<int64_t>(s->batch) * s->H;
  if (heads > (1 << 30) || 2 * tiles * heads >= (int64_t(1) << 31)) return W2V_ESHAPE;
  a->bf16 = s->dtype == W2V_BF16;
  a->batch = s->batch;
  a->T = s->T;
  a->H = s->H;
  a->qkv_ld = s->qkv_ld; a->qkv_bs = s->qkv_bs;
  a->out_ld = s->out_ld; a->out_bs = s->out_bs;
  a->grad_ld = s->grad_ld; a->grad_bs = s->grad_bs;
  a->frames = s->frames;
  if (reinterpret_cast<uintptr_t>(s->frames) % 4 != 0) return W2V_EINVAL;
  const int64_t width = 64 * static_cast<int64_t>(s->H);
  if (!strides_ok(&a->qkv_ld, &a->qkv_bs, s->T, s->batch, width)) return W2V_EINVAL;
  if (!strides_ok(&a->out_ld, &a->out_bs, s->T, s->batch, width)) return W2V_EINVAL;
  if (grads && !strides_ok(&a->grad_ld, &a->grad_bs, s->T, s->batch, width)) return W2V_EINVAL;
  return W2V_OK;
}

bool type_ok(int t) { return t == W2V_F16 || t == W2V_BF16 || t == W2V_F32; }

int layernorm_args(int x_type, int64_t x_ld, int y_type, int64_t y_ld, int64_t rows, int cols, const float* gamma,
                   const float* beta, int act, LnTrain* a) {
  if (!type_ok(x_type) || !type_ok(y_type) || (y_type != x_type && x_type != W2V_F32)) return W2V_EINVAL;
  if (act < 0 || act > 2) return W2V_EINVAL;
  if (rows < 0 || rows >= (int64_t(1) << 31) || cols < 1 || cols > W2V_LAYERNORM_MAX_COLS) return W2V_ESHAPE;
  if (!gamma || !beta) return W2V_EINVAL;
  if (x_ld < cols || y_ld < cols) return W2V_EINVAL;
  a->x_type = x_type;
  a->y_type = y_type;
  a->rows = rows;
  a->cols = cols;
  a->x_ld = x_ld;
  a->y_ld = y_ld;
  a->gamma = gamma;
  a->beta = beta;
  a->act = act;
  return W2V_OK;
}

size_t type_size(int t) { return t == W2V_F32 ? 4 : 2; }

constexpr int64_t kMostStride = int64_t(1) << 56;  // elements: longer rows than any memory holds

bool aligned_to(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// A workspace of no bytes may be anything.
bool workspace_ok(const void* ws, size_t has, size_t needs) {
  return needs == 0 || (ws && aligned16(ws) && has >= needs);
}

// The operands of a call: false if one that is written shares memory with another
// one, or if one is longer than any memory.
struct Operands {
  Extent writes[5], reads[7];
  int n_writes = 0, n_reads = 0;
  bool fit = true;
  void rows(bool write, const void* p, int64_t width, int64_t stride0, int64_t n0, int64_t stride1 = 0, int64_t n1 = 1) {
    fit = make_extent(p, width, stride0, n0, stride1, n1, write ? writes + n_writes++ : reads + n_reads++) && fit;
  }
  void bytes(bool write, const void* p, int64_t n) { rows(write, p, n, 0, 1); }
  // one 16-bit operand of an attention call; strides in elements
  void clips(bool write, const void* p, const AttnTrain& a, int64_t ld, int64_t bs) {
    rows(write, p, 128 * static_cast<int64_t>(a.H), 2 * ld, a.T, a.batch == 1 ? 0 : 2 * bs, a.batch);
  }
  bool apart() const { return fit && !writes_overlap(writes, n_writes, reads, n_reads); }
};

}  // namespace

extern "C" int w2v_op_attention_fwd(const w2v_attention_shape* shape, const void* q, const void* k, const void* v,
                                    void* out, float* lse, int* err_dev, void* stream) {
  AttnTrain a;
  const int rc = attention_args(shape, false, &a);
  if (rc != W2V_OK) return rc;
  if (!q || !k || !v || !out || !lse || !err_dev) return W2V_EINVAL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned_to(lse, 4) ||
      !aligned_to(err_dev, 4))
    return W2V_EINVAL;
  Operands o;
  // (a CTA reads the rows of q that it writes, and no other: out may be q)
  const bool in_place = q == out && a.qkv_ld == a.out_ld && a.qkv_bs == a.out_bs;
  if (!in_place) o.clips(false, q, a, a.qkv_ld, a.qkv_bs);
  for (const void* p : {k, v}) o.clips(false, p, a, a.qkv_ld, a.qkv_bs);
  if (a.frames) o.bytes(false, a.frames, 4 * static_cast<int64_t>(a.batch));
  o.clips(true, out, a, a.out_ld, a.out_bs);
  o.bytes(true, lse, 4 * static_cast<int64_t>(a.batch) * a.H * a.T);
  o.bytes(true, err_dev, 4);
  if (!o.apart()) return W2V_EINVAL;
  return status(launch_attention_fwd(a, q, k, v, out, lse, err_dev, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t w2v_op_attention_bwd_workspace(int batch, int T, int H) {
  if (batch < 1 || T < 1 || H < 1) return 0;
  return attention_bwd_ws_bytes(batch, T, H);
}

extern "C" int w2v_op_attention_bwd(const w2v_attention_shape* shape, const void* dout, const void* q, const void* k,
                                    const void* v, const void* out, const float* lse, void* dq, void* dk, void* dv,
                                    void* ws, size_t ws_bytes, int* err_dev, void* stream) {
  AttnTrain a;
  const int rc = attention_args(shape, true, &a);
  if (rc != W2V_OK) return rc;
  if (!dout || !q || !k || !v || !out || !lse || !dq || !dk || !dv || !err_dev) return W2V_EINVAL;
  for (const void* p : {dout, q, k, v, out, static_cast<const void*>(dq), static_cast<const void*>(dk),
                        static_cast<const void*>(dv)})
    if (!aligned16(p)) return W2V_EINVAL;
  if (!aligned_to(lse, 4) || !aligned_to(err_dev, 4)) return W2V_EINVAL;
  const size_t needs = attention_bwd_ws_bytes(a.batch, a.T, a.H);
  if (!workspace_ok(ws, ws_bytes, needs)) return W2V_EINVAL;
  Operands o;
  for (const void* p : {q, k, v}) o.clips(false, p, a, a.qkv_ld, a.qkv_bs);
  for (const void* p : {out, dout}) o.clips(false, p, a, a.out_ld, a.out_bs);
  o.bytes(false, lse, 4 * static_cast<int64_t>(a.batch) * a.H * a.T);
  if (a.frames) o.bytes(false, a.frames, 4 * static_cast<int64_t>(a.batch));
  for (const void* p : {dq, dk, dv}) o.clips(true, p, a, a.grad_ld, a.grad_bs);
  o.bytes(true, ws, static_cast<int64_t>(needs));
  o.bytes(true, err_dev, 4);
  if (!o.apart()) return W2V_EINVAL;
  return status(launch_attention_bwd(a, dout, q, k, v, out, lse, dq, dk, dv, ws, err_dev,
                                     static_cast<cudaStream_t>(stream)));
}

extern "C" int w2v_op_layernorm_fwd(const void* x, int x_type, int64_t x_ld, void* y, int y_type, int64_t y_ld,
                                    int64_t rows, int cols, const float* gamma, const float* beta, float eps, int act,
                                    float* mean, float* rstd, void* stream) {
  LnTrain a;
  const int rc = layernorm_args(x_type, x_ld, y_type, y_ld, rows, cols, gamma, beta, act, &a);
  if (rc != W2V_OK) return rc;
  if (!(eps > 0.f)) return W2V_EINVAL;
  if (rows > 0 && (!x || !y || !mean || !rstd)) return W2V_EINVAL;
  if (!aligned_to(x, type_size(x_type)) || !aligned_to(y, type_size(y_type)) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4) || !aligned_to(gamma, 4) || !aligned_to(beta, 4))
    return W2V_EINVAL;
  Operands o;
  const int64_t xs = type_size(x_type), ys = type_size(y_type);
  if (x_ld > kMostStride || y_ld > kMostStride) return W2V_EINVAL;
  o.rows(false, x, xs * cols, xs * x_ld, rows);
  for (const float* p : {gamma, beta}) o.bytes(false, p, 4 * static_cast<int64_t>(cols));
  o.rows(true, y, ys * cols, ys * y_ld, rows);
  for (const float* p : {mean, rstd}) o.bytes(true, p, 4 * rows);
  if (!o.apart()) return W2V_EINVAL;
  return status(launch_layernorm_fwd(a, x, y, eps, mean, rstd, static_cast<cudaStream_t>(stream)));
}

extern "C" size_t w2v_op_layernorm_bwd_workspace(int64_t rows, int cols) {
  if (rows < 0 || cols < 1 || cols > W2V_LAYERNORM_MAX_COLS) return 0;
  return layernorm_bwd_ws_bytes(rows, cols);
}

extern "C" int w2v_op_layernorm_bwd(const void* dy, int y_type, int64_t dy_ld, const void* x, int x_type, int64_t x_ld,
                                    int64_t rows, int cols, const float* gamma, const float* beta, const float* mean,
                                    const float* rstd, int act, const void* dres, int64_t dres_ld, void* dx,
                                    int64_t dx_ld, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                    void* stream) {
  LnTrain a;
  const int rc = layernorm_args(x_type, x_ld, y_type, dy_ld, rows, cols, gamma, beta, act, &a);
  if (rc != W2V_OK) return rc;
  if (!dgamma || !dbeta || (rows > 0 && (!dy || !x || !mean || !rstd || !dx))) return W2V_EINVAL;
  if (dx_ld < cols || (dres && dres_ld < cols) || (dres && dres == dx && dres_ld != dx_ld)) return W2V_EINVAL;
  if (!aligned_to(dy, type_size(y_type)) || !aligned_to(x, type_size(x_type)) || !aligned_to(dx, type_size(x_type)) ||
      !aligned_to(dres, type_size(x_type)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(gamma, 4) ||
      !aligned_to(beta, 4) || !aligned_to(dgamma, 4) || !aligned_to(dbeta, 4))
    return W2V_EINVAL;
  const size_t needs = layernorm_bwd_ws_bytes(rows, cols);
  if (!workspace_ok(ws, ws_bytes, needs)) return W2V_EINVAL;
  Operands o;
  const int64_t xs = type_size(x_type), ys = type_size(y_type);
  if (x_ld > kMostStride || dy_ld > kMostStride || dx_ld > kMostStride || (dres && dres_ld > kMostStride))
    return W2V_EINVAL;
  o.rows(false, dy, ys * cols, ys * dy_ld, rows);
  o.rows(false, x, xs * cols, xs * x_ld, rows);
  if (dres && dres != dx) o.rows(false, dres, xs * cols, xs * dres_ld, rows);
  for (const float* p : {gamma, beta}) o.bytes(false, p, 4 * static_cast<int64_t>(cols));
  for (const float* p : {mean, rstd}) o.bytes(false, p, 4 * rows);
  o.rows(true, dx, xs * cols, xs * dx_ld, rows);
  for (const float* p : {dgamma, dbeta}) o.bytes(true, p, 4 * static_cast<int64_t>(cols));
  o.bytes(true, ws, static_cast<int64_t>(needs));
  if (!o.apart()) return W2V_EINVAL;
  return status(launch_layernorm_bwd(a, dy, x, mean, rstd, dres, dres_ld, dx, dx_ld, dgamma, dbeta, ws,
                                     static_cast<cudaStream_t>(stream)));
}

extern "C" size_t w2v_op_grad_clip_workspace(int n) { return n < 0 ? 0 : grad_clip_ws_bytes(n); }

extern "C" int w2v_op_grad_clip(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                                const int* types, float scale, float max_norm, float* norm_dev, void* ws,
                                size_t ws_bytes, void* stream) {
  if (n < 0) return W2V_ESHAPE;
  if (!norm_dev || !aligned_to(norm_dev, 4)) return W2V_EINVAL;
  if (n > 0 && (!grads || !outs || !counts || !types)) return W2V_EINVAL;
  if (!(scale > 0.f) || !(scale < INFINITY) || !(max_norm > 0.f)) return W2V_EINVAL;
  if (!workspace_ok(ws, ws_bytes, grad_clip_ws_bytes(n))) return W2V_EINVAL;
  try {
    // Byte ranges written (the norm and the workspace among them), and each tensor's
    // read range: an output may be its own gradient's memory, and nothing else that the
    // call reads or writes.
    struct Range {
      uintptr_t from, to;
    };
    std::vector<Range> ranges;
    ranges.reserve(2 * static_cast<size_t>(n) + 2);
    const uintptr_t norm_at = reinterpret_cast<uintptr_t>(norm_dev), ws_at = reinterpret_cast<uintptr_t>(ws);
    ranges.push_back({norm_at, norm_at + sizeof(float)});
    ranges.push_back({ws_at, ws_at + grad_clip_ws_bytes(n)});
    for (int i = 0; i < n; ++i) {
      if (!type_ok(types[i])) return W2V_EINVAL;
      if (counts[i] < 0 || counts[i] >= (int64_t(1) << 33)) return W2V_ESHAPE;
      if (counts[i] == 0) continue;
      const size_t size = type_size(types[i]);
      if (!grads[i] || !outs[i] || !aligned_to(grads[i], size) || !aligned_to(outs[i], size)) return W2V_EINVAL;
      const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
      const uintptr_t bytes = static_cast<uintptr_t>(counts[i]) * size;
      ranges.push_back({g, g + bytes});
      if (o != g) ranges.push_back({o, o + bytes});
    }
    std::sort(ranges.begin(), ranges.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
    for (size_t i = 1; i < ranges.size(); ++i)
      if (ranges[i].from < ranges[i - 1].to) return W2V_EINVAL;
    return status(launch_grad_clip(n, grads, outs, counts, types, scale, max_norm, norm_dev, ws,
                                   static_cast<cudaStream_t>(stream)));
  } catch (const std::bad_alloc&) {
    return W2V_ENOMEM;
  }
}
