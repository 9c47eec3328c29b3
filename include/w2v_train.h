/*
 * w2v_train.h — the operators that fine-tuning an encoder block needs beside
 * the forward pass: attention with its gradients, LayerNorm with its gradients,
 * and the gradient norm with clipping.  Same conventions as w2v_ops.h: plain
 * device pointers owned by the caller, cudaStream_t as void*, an int status
 * (W2V_OK or W2V_E*), asynchronous on the stream, on the current device.
 *
 * None of these calls allocates, synchronises or keeps anything from one call
 * to the next, so each may be recorded into a CUDA graph.  Scratch is a
 * workspace that the caller passes (16-byte aligned device memory of at least
 * the size its w2v_op_*_workspace function returns; nothing in it needs to be
 * initialised or kept; a size of 0 means that NULL will do).  Calls whose work
 * may overlap on the GPU — two streams, two graphs — need a workspace each.
 *
 * What a call writes (outputs, workspace, error word) must not share memory with
 * anything else that it reads or writes, except where a call says so; rows that lie
 * between one another's, as those of a fused projection, do not.  A call whose
 * operands do is refused with W2V_EINVAL.
 *
 * Sums run in a fixed order: the same call gives the same bits.
 */
#ifndef W2V_TRAIN_H
#define W2V_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types. */
enum { W2V_F16 = 0, W2V_BF16 = 1, W2V_F32 = 2 };

/* Sizes and layout of one attention call.  Every operand is [batch][T][H][64]
 * with the 64 channels of a head, and the heads of a row, contiguous; *_ld is
 * the distance in elements between rows, *_bs between clips, so a slice of a
 * fused [batch][T][3 * H * 64] projection (ld = 3 * H * 64) and time-major
 * tensors (ld = batch * H * 64, bs = H * 64) are read and written in place.
 * Strides must be multiples of 8 elements, and rows must not overlap. */
typedef struct {
  int dtype;                 /* W2V_F16 or W2V_BF16, of every operand and gradient */
  int batch, T, H;           /* clips, frames of the padded batch, heads; T < 2^24 */
  int64_t qkv_ld, qkv_bs;    /* q, k and v */
  int64_t out_ld, out_bs;    /* out and dout */
  int64_t grad_ld, grad_bs;  /* dq, dk and dv (backward only) */
  const int32_t* frames;     /* DEVICE int32 [batch]: frames of each clip, in [0, T] (other
                                values are clamped), or NULL when every clip has T */
} w2v_attention_shape;

/* out = softmax(q k^T / 8) v per (clip, head), over the clip's own frames only
 * (the plain SDPA of w2v_op_attention at every clip's true length), and
 * lse [batch][H][T] (fp32), the natural logarithm of each row's sum of
 * exponentials, which the backward pass recomputes the probabilities from.
 * out may be q, with the same strides (a forward pass without a backward one).
 * Rows past a clip's frames are written: out 0, lse -infinity; what the inputs
 * hold there, NaN included, is not used.  err_dev as in w2v_ops.h.
 * A row of a clip's own frames with a score that is NaN or +infinity, or with
 * none above -infinity, has no softmax: its out and lse are NaN.
 * Scores, softmax and sums are fp32 (an exponential within 3e-6 of itself, and so
 * lse within 3e-6 beside the scores' own roundings); the probabilities are rounded to
 * dtype for the product with v.
 * Errors: W2V_EINVAL (null or misaligned pointer, dtype, strides, overlap),
 * W2V_ESHAPE (batch, T or H < 1, T or the number of tiles too large), W2V_ECUDA. */
int w2v_op_attention_fwd(const w2v_attention_shape* shape, const void* q, const void* k, const void* v, void* out,
                         float* lse, int* err_dev, void* stream);

/* Bytes of the backward pass's workspace (0 up to 128 frames, and if batch, T or
 * H < 1). */
size_t w2v_op_attention_bwd_workspace(int batch, int T, int H);

/* Gradients of w2v_op_attention_fwd: with P = exp(q k^T / 8 - lse),
 *   dv = P^T dout,  dS = P o (dout v^T - rowsum(dout o out)),
 *   dq = dS k / 8,  dk = dS^T q / 8.
 * out and lse are the forward call's.  dq, dk and dv are overwritten, with
 * zeros past a clip's frames; dout, like the other inputs, is not used there.
 * The rounding of out in the row sum leaves an error in proportion to P in dS; dq has
 * it taken out again (what a row of dS sums to, times P k), and in clips of up to 64
 * frames dk too.
 * P and dS are rounded to dtype for the products (dS, in fp16, after scaling by
 * a power of two per clip and head that keeps it in range); everything else is
 * fp32.  In fp16 a row whose |rowsum| or 8 |lse| is above 65504 * 2^15 (2^31) has
 * gradients that are not finite.  No atomics.  Errors as above, and W2V_EINVAL if
 * ws_bytes is too small. */
int w2v_op_attention_bwd(const w2v_attention_shape* shape, const void* dout, const void* q, const void* k,
                         const void* v, const void* out, const float* lse, void* dq, void* dk, void* dv, void* ws,
                         size_t ws_bytes, int* err_dev, void* stream);

/* Widest row of the LayerNorm calls. */
#define W2V_LAYERNORM_MAX_COLS 8192

/* y = f((x - mean) rstd gamma + beta) per row of `cols` channels, f by act (0
 * none, 1 exact GELU, 2 tanh GELU), biased variance, rstd = 1 / sqrt(var + eps);
 * mean and rstd (fp32 [rows]) are kept for the backward pass.  In the exact GELU and
 * its slope Phi is within 3e-7; with an fp32 y Phi(-|z|) is within 2^-19 + z^2 2^-23
 * of its own value up to |z| = 13, and with a 16-bit y within 2^-13.  x_type and
 * y_type are equal, or x is fp32 and y fp16 or bf16 (the fp32 residual stream
 * normalised for the next projection).  x_ld and y_ld: elements between rows,
 * >= cols; any alignment of the element type (rows of 16-byte multiples on
 * 16-byte boundaries are the fast case).  gamma, beta: fp32 [cols].
 * rows = 0 does nothing (x, y, mean and rstd may then be NULL).
 * Errors: W2V_EINVAL (null or misaligned pointer, types, strides, act, eps <= 0,
 * overlap), W2V_ESHAPE (rows < 0 or >= 2^31, cols outside [1, W2V_LAYERNORM_MAX_COLS]),
 * W2V_ECUDA. */
int w2v_op_layernorm_fwd(const void* x, int x_type, int64_t x_ld, void* y, int y_type, int64_t y_ld, int64_t rows,
                         int cols, const float* gamma, const float* beta, float eps, int act, float* mean, float* rstd,
                         void* stream);

/* Bytes of the backward pass's workspace (0 for few rows, and if a size is out of
 * range). */
size_t w2v_op_layernorm_bwd_workspace(int64_t rows, int cols);

/* Gradients of w2v_op_layernorm_fwd (and of w2v_op_layernorm, with the mean and
 * rstd of its rows): with xh = (x - mean) rstd, dz = dy f'(xh gamma + beta) and
 * w = dz gamma,
 *   dx = rstd (w - mean_cols(w) - xh mean_cols(w xh)) + dres,
 *   dgamma = sum_rows dz xh,  dbeta = sum_rows dz     (fp32 [cols], overwritten).
 * dy is of y_type; dres (the gradient that reached x past the LayerNorm, or NULL
 * for none) and dx are of x_type.  dx may be dres, with the same stride (the sum
 * in place).
 * rows = 0 writes zeros to dgamma and dbeta.  Errors as above, and W2V_EINVAL if
 * ws_bytes is too small. */
int w2v_op_layernorm_bwd(const void* dy, int y_type, int64_t dy_ld, const void* x, int x_type, int64_t x_ld,
                         int64_t rows, int cols, const float* gamma, const float* beta, const float* mean,
                         const float* rstd, int act, const void* dres, int64_t dres_ld, void* dx, int64_t dx_ld,
                         float* dgamma, float* dbeta, void* ws, size_t ws_bytes, void* stream);

/* Bytes of the workspace of w2v_op_grad_clip for n tensors (0 if n < 0). */
size_t w2v_op_grad_clip_workspace(int n);

/* Gradient norm over n tensors, and clipping:
 *   norm = scale sqrt(sum over all tensors of g^2),
 *   outs[i] = grads[i] scale min(1, max_norm / (norm + 1e-6)).
 * grads, outs, counts (elements), types: HOST arrays [n] (of device pointers,
 * the first two), read during the call; an output has its gradient's type.
 * scale (> 0) undoes a loss scale; max_norm = INFINITY only scales.  norm_dev:
 * one fp32, on the device.  counts below 2^33 each.  The sum is fp64.  If the norm
 * is not finite, or past fp32's range and so written as infinity, nothing is clipped
 * (outs = grads scale): a caller that reads norm_dev can drop the step.  outs[i] may
 * be grads[i] (in place); otherwise no tensor may overlap another one.  Empty tensors
 * are allowed.
 * Errors: W2V_EINVAL (null or misaligned pointer, type, overlap, scale,
 * max_norm <= 0 or NaN, ws_bytes too small), W2V_ESHAPE (n or a count out of
 * range), W2V_ENOMEM (host), W2V_ECUDA. */
int w2v_op_grad_clip(int n, const void* const* grads, void* const* outs, const int64_t* counts, const int* types,
                     float scale, float max_norm, float* norm_dev, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W2V_TRAIN_H */
