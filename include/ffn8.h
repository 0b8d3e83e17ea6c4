/*
 * ffn8.h -- what a feed-forward block needs around the W8A8 products, on AMD
 * Instinct MI355X (gfx950): an RMS norm that emits INT8 codes, products with bias,
 * activation, gate and residual, a router, and a layer of INT8 experts for few
 * tokens. Part of libw4a4.so; the conventions of w4a4.h hold (device pointers,
 * validation first, asynchronous on `stream`, no allocation, status codes).
 */
#ifndef FFN8_H
#define FFN8_H

#include "w4a4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations of the epilogues: none, max(v, 0), v / (1 + exp(-v)), v Phi(v), and
 * v (1 + tanh(sqrt(2 / pi) (v + 0.044715 v^3))) / 2. */
enum {
  W8A8_ACT_NONE = 0,
  W8A8_ACT_RELU = 1,
  W8A8_ACT_SILU = 2,
  W8A8_ACT_GELU = 3,
  W8A8_ACT_GELU_TANH = 4
};

/*
 * Residual addition, RMS norm and symmetric INT8 quantization per row, in one pass:
 *   h = x + residual, rounded to x's type (h = x without a residual)
 *   t = fl32(h * weight);  rstd = 1 / sqrt(mean(h^2) + eps);  a = max|t|
 *   xq = rne(fl32(t / fl32(a / 127))), held in [-127, 127];  xs = fl32(fl32(a rstd) / 127)
 *   y = t rstd, rounded to x's type
 * xq * xs stands for t rstd; the row's factor rstd does not enter the codes. A row
 * with a = 0 gives xs = 0 and codes 0 (codes 0 also where a / 127 rounds to 0); one
 * with a NaN or an infinity in h or t gives xs = NaN and any codes. Squares past fp32's
 * range (bf16) do not overflow.
 *
 *   x         [M][ldx] of x_dtype W4A4_Y_F16 or W4A4_Y_BF16, 16-byte aligned, ldx % 8 == 0
 *   residual  NULL or [M][ldr], as x
 *   weight    [K] of w_dtype W4A4_Y_F32 or x_dtype, 16-byte aligned
 *   eps       >= 2^-126 (fp32's smallest normal value), finite
 *   M, K      K > 0, K % 16 == 0, K <= 2^30, M < 2^24
 *   xq, xs    out: int8 [M][K], 16-byte aligned; f32 [M] (the input of w8a8_gemm)
 *   h         out, with a residual: [M][ldh] as x; may be x or residual itself (same
 *             pointer and stride), else must not overlap them
 *   y         out: NULL or [M][ldy] as x
 * The outputs lie apart from one another and, but for h, from the inputs
 * (W4A4_E_OVERLAP; here and below).
 */
w4a4_status_t w8a8_rmsnorm_quantize(const void* x, int32_t x_dtype, int64_t ldx, const void* residual, int64_t ldr,
                                    const void* weight, int32_t w_dtype, float eps, int64_t M, int64_t K,
                                    int8_t* xq, float* xs, void* h, int64_t ldh, void* y, int64_t ldy, void* stream);

/*
 * W8A8 GEMM with an epilogue. P = sum_k xq wq exactly,
 *   v[m,n] = fl32(fl32(fl32(P) * fl32(xs[m] * ws[n])) + bias[n])
 *   Y[m,n] = act(v[m,n]) + residual[m,n]                       (gated == 0)
 *   Y[m,n] = act(v[m,2n]) * v[m,2n+1] + residual[m,n]          (gated != 0)
 * in fp32, rounded once to y_dtype (W4A4_Y_F16 or W4A4_Y_BF16). The residual is +0 where
 * there is none.
 *
 *   N         outputs. wq, ws, bias hold N channels, or 2 N when gated: channel 2n
 *             is output n's gate, 2n + 1 what it multiplies
 *   residual  NULL or [M][ldr] of y_dtype; may be y itself (same pointer and stride),
 *             else must not overlap y (nor may the other inputs)
 *   xq, xs, wq, ws, bias, M, K, y, ldy: as for w8a8_gemm (channels <= 2^22 - 4)
 *   workspace at least w8a8_gemm_act_workspace(M, N, K, gated, wide) bytes, 16-byte
 *             aligned, overwritten; may be NULL when that is 0
 */
w4a4_status_t w8a8_gemm_act(const int8_t* xq, const float* xs, const int8_t* wq, const float* ws, const float* bias,
                            int32_t act, int32_t gated, const void* residual, int64_t ldr,
                            int64_t M, int64_t N, int64_t K, void* workspace, int64_t workspace_bytes,
                            void* y, int32_t y_dtype, int64_t ldy, void* stream);

/* Workspace bytes w8a8_gemm_act needs, or -1 for invalid extents. Host-only. wide: y
 * and the residual are 16-byte aligned with strides that are multiples of 8 below 2^22 (what
 * other rows need is never less). */
int64_t w8a8_gemm_act_workspace(int64_t M, int64_t N, int64_t K, int32_t gated, int32_t wide);

/*
 * A W8A8 linear layer with an epilogue: w8a8_quantize_act of X, then w8a8_gemm_act
 * (few tokens: one launch without a workspace). Arguments as for those; y must not
 * overlap x.
 */
w4a4_status_t w8a8_linear_act(const void* x, int32_t x_dtype, int64_t M, int64_t K, int64_t ldx,
                              const int8_t* wq, const float* ws, const float* bias, int32_t act, int32_t gated,
                              const void* residual, int64_t ldr, int64_t N, void* workspace, int64_t workspace_bytes,
                              void* y, int32_t y_dtype, int64_t ldy, void* stream);

/* Workspace bytes w8a8_linear_act needs, as w8a8_gemm_act_workspace. Host-only. */
int64_t w8a8_linear_act_workspace(int64_t M, int64_t N, int64_t K, int32_t gated, int32_t wide);

/*
 * Router: the k largest of each token's logits, largest first, the lower index first
 * among equals, and their softmax weights
 *   weights[t][j] = exp(l_j - max) / sum exp(l - max)
 * over all E experts, or with `renormalize` over the k chosen. A logit of minus
 * infinity, or NaN, is never chosen and weighs nothing; where fewer than k are left,
 * the other ids are -1 and their weights 0. Plus infinity counts as the largest
 * finite value.
 *
 *   logits   [T][ldl] of dtype (any W4A4_Y_*), ldl >= E;  E <= 512, 0 < k <= 64, T < 2^24
 *   ids      out: int32 [T][k];  weights  out: f32 [T][k], apart and apart from logits
 */
w4a4_status_t moe_route(const void* logits, int32_t dtype, int64_t T, int64_t E, int64_t ldl, int64_t k,
                        int32_t renormalize, int32_t* ids, float* weights, void* stream);

/*
 * A mixture-of-experts layer of few tokens on INT8 experts. For token t, choice j with
 * expert e = ids[t][j], and exact integer products:
 *   h = act(g) * u,  g and u channels 2i and 2i + 1 of w13[e] on (xq[t], xs[t]), as v of
 *       w8a8_gemm_act;  (hq, hs) = INT8 codes and scale of h (the rule of
 *       w8a8_quantize_act, on fp32 values, codes held in [-127, 127])
 *   y[t] = sum_j weights[t][j] * fl32(fl32(P') * fl32(hs * s2[e])), P' = w2[e] hq
 * summed over j in order and rounded once. An id outside 0 .. E - 1 adds nothing
 * (experts of another rank; the ids of a token may repeat).
 *
 *   xq, xs   int8 [T][H], 16-byte aligned; f32 [T]
 *   ids, weights  int32, f32 [T][k], read on the device; T k <= 512
 *   w13, s13 int8 [E][2 I][H], f32 [E][2 I];  w2, s2  int8 [E][H][I], f32 [E][H]; E <= 512
 *   H, I     multiples of 16, <= 131056
 *   y        out: [T][ldy] of y_dtype W4A4_Y_F16 or W4A4_Y_BF16, ldy >= H, apart from ids,
 *            weights, w2 and s2
 *   workspace at least w8a8_moe_workspace(T, k, E, H, I) bytes, 16-byte aligned,
 *            overwritten
 */
w4a4_status_t w8a8_moe(const int8_t* xq, const float* xs, const int32_t* ids, const float* weights, int64_t T, int64_t k,
                       const int8_t* w13, const float* s13, const int8_t* w2, const float* s2,
                       int64_t E, int64_t H, int64_t I, int32_t act, void* workspace, int64_t workspace_bytes,
                       void* y, int32_t y_dtype, int64_t ldy, void* stream);

/* Workspace bytes w8a8_moe needs, or -1 for invalid extents. Host-only. */
int64_t w8a8_moe_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I);

#ifdef __cplusplus
}
#endif

#endif /* FFN8_H */
