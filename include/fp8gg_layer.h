/*
 * fp8gg_layer.h -- C ABI of the operators around the grouped GEMM in a
 * mixture-of-experts layer (MI355X, gfx950): the norm that makes the fp8 operand,
 * the routing of tokens to experts, the exchange of rows between token order and
 * expert order, and the 8-bit activation checkpoints with their backward use.
 *
 * A layer's forward pass, with the products of fp8gg.h between them:
 *
 *     rmsnorm_quantize -> route -> moe_dispatch -> grouped product (gate and up)
 *       -> silu_mul_quantize -> grouped product (down) -> moe_combine
 *
 * Conventions (as in fp8gg.h unless said otherwise)
 *   - Device pointers, dense row-major tensors, bf16 as raw uint16_t bits, fp8 as raw
 *     e4m3fn bytes.  Work is only enqueued on `stream`; nothing is allocated, copied to
 *     the host or synchronised, and every call may be captured into a graph.
 *   - Results are deterministic: no floating-point atomics, fixed orders of summation.
 *   - A row of codes with its scale s stands for e4m3fn(code) * s.  Everywhere below a
 *     scale is s = max(amax, 2^-100) / 448 (1 when amax is 0), where amax is the largest
 *     magnitude that it covers, and a code is the value divided by s, rounded to nearest
 *     even; the values are fp32 before that one rounding.  The floor keeps 448 / amax
 *     finite; it is far below what activations and gradients hold.  fp32 arithmetic may
 *     place a value that lies within about 2^-21 of the midpoint of two codes on either
 *     side (an activation of silu_mul_quantize with gate g: (|g| + 4) 2^-22).  The sign of a
 *     zero code is unspecified.
 *   - Inputs are expected finite.  A NaN or infinity makes the values that depend on it
 *     unspecified (its row; its scale block; its group's column) and no others.
 *   - Sums, norms, softmax statistics and dot products are held in fp32 or more.
 *   - Buffers of one call must not overlap, except where a line says that one may be
 *     another.  Optional pointers are marked (or NULL).
 *   - A failed check returns a non-zero status, enqueues nothing and leaves a message
 *     for f8f8bf16_layer_last_error().
 */
#ifndef FP8GG_LAYER_H_
#define FP8GG_LAYER_H_

#include <stdint.h>

#include "fp8gg.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8GG_DTYPE_BF16 = 0,
  FP8GG_DTYPE_F32 = 1,
  FP8GG_DTYPE_E4M3 = 2
} fp8gg_dtype;

typedef enum {
  FP8GG_SCORE_SOFTMAX = 0,
  FP8GG_SCORE_SIGMOID = 1
} fp8gg_score;

/*
 * Root-mean-square norm with the residual's addition and an fp8 output (the scale's floor
 * is applied to h * weight, before rstd; h^2, h * weight and rstd have to be finite in
 * fp32, so without eps a row's root mean square has to be above 2^-128):
 *
 *     h    = bf16_rne(X + residual)          (h = X without a residual)
 *     rstd = 1 / sqrt(mean_k h^2 + eps)   (0 for a row of zeros when eps is 0)
 *     y    = h * rstd * weight
 *     XQ, x_scale = codes and scales of y;   Y = bf16_rne(y)
 *
 *   X             [rows, K]         bf16
 *   residual      [rows, K]         bf16 (or NULL)
 *   weight        [K]               bf16 or fp32 (weight_dtype)
 *   block                           0: one scale per row; 128: one per row and 128 columns
 *   XQ            [rows, K]         e4m3fn
 *   x_scale       [rows] or [rows, K / 128]   fp32
 *   Y             [rows, K]         bf16 (or NULL)
 *   residual_out  [rows, K]         bf16, h; given exactly when residual is; may be residual itself
 *   rstd          [rows]            fp32 (or NULL): what the backward pass needs
 *
 * K % 8 == 0 (block 128: K % 128 == 0), 0 < K <= 32768.  bf16 and fp32 tensors with a
 * K axis 16-byte aligned, XQ 8-byte, the others 4-byte.
 */
fp8gg_status f8f8bf16_rmsnorm_quantize(
    const uint16_t* X, const uint16_t* residual, const void* weight, int weight_dtype, float eps, int block,
    uint8_t* XQ, float* x_scale, uint16_t* Y, uint16_t* residual_out, float* rstd,
    int64_t rows, int64_t K, void* stream);

/*
 * Its gradient; the fp8 rounding passes gradients through (dY is the gradient of y).
 * With xhat = h * rstd:
 *
 *     dX      = bf16_rne(rstd * (w dY - xhat * mean_k(w dY xhat)) + dresidual)
 *     dweight = sum_rows dY * xhat
 *
 *   dY         [rows, K]   bf16          H     [rows, K]   bf16, h of the forward pass
 *   weight     [K]         as above      rstd  [rows]      fp32, of the forward pass
 *   dresidual  [rows, K]   bf16 (or NULL): the gradient that reaches residual_out
 *   dX         [rows, K]   bf16: the gradient of X and of residual alike; may be dY or dresidual itself
 *   dweight    [K]         fp32
 *   workspace              f8f8bf16_rmsnorm_backward_workspace(rows, K) bytes, 16-byte aligned
 *
 * Shapes and alignment as above.  rows == 0 writes dweight = 0.
 */
fp8gg_status f8f8bf16_rmsnorm_backward(
    const uint16_t* dY, const uint16_t* H, const void* weight, int weight_dtype, const float* rstd,
    const uint16_t* dresidual, uint16_t* dX, float* dweight, void* workspace, int64_t workspace_bytes,
    int64_t rows, int64_t K, void* stream);
int64_t f8f8bf16_rmsnorm_backward_workspace(int64_t rows, int64_t K);

/*
 * Routing: for each token the k experts with the highest keys, their weights, and the
 * places of the (token, expert) pairs in the experts' order.
 *
 *     p      = softmax(logits) or sigmoid(logits) over the E experts
 *     key    = p + bias        (the bias decides the choice only, never the weights)
 *     groups of E / n_group neighbouring experts: a group's score is the sum of its
 *     group_top highest keys; only experts of the topk_group best groups stay
 *     chosen = the k highest keys, descending; ties go to the lowest index
 *     weight = scale * p / (sum of the chosen p)     (renormalize)   or   scale * p
 *
 * The choice is that of exact arithmetic on the given logits and bias, as far as fp64
 * tells: without a bias experts rank by their logits, else by their keys in fp64 (a score
 * below 2^-53 of its bias does not count); a group's sum of two keys is rounded to 44
 * significant bits, so that sums which are equal, as sigmoid(x) + sigmoid(-x) = 1, tie.
 * A logit or bias of -infinity or NaN takes its expert out; +infinity counts as the
 * largest finite fp32.  A group without an expert left is never kept.  Slots for which
 * no expert is left hold id -1, weight 0 and dst_row -1, as in a row whose logits are
 * all masked.
 *
 *   logits    [T, E]   fp32 or bf16 (logits_dtype)
 *   bias      [E]      fp32 (or NULL)
 *   weights   [T, k]   fp32             ids  [T, k]  int32
 *   M_sizes   [E]      int64: rows per expert (the stacked layout's operand)
 *   dst_row   [T, k]   int32: the row of pair (t, j) when pairs are sorted by expert, and
 *                      within an expert by t, then j
 *   M_sizes and dst_row may both be NULL (no plan).
 *   workspace          f8f8bf16_route_workspace(T, E, k) bytes, 16-byte aligned; may be
 *                      NULL when that is 0 or there is no plan
 *
 * 1 <= k <= 16, k <= E <= 1024, E % n_group == 0, n_group <= 16,
 * 1 <= topk_group <= n_group, group_top 1 or 2, T * k < 2^31 - 256.  logits 16-byte aligned.
 */
fp8gg_status f8f8bf16_route(
    const void* logits, int logits_dtype, const float* bias, int score, int64_t n_group, int64_t topk_group,
    int group_top, int renormalize, float scale, float* weights, int32_t* ids, int64_t* M_sizes,
    int32_t* dst_row, void* workspace, int64_t workspace_bytes, int64_t T, int64_t E, int64_t k, void* stream);
int64_t f8f8bf16_route_workspace(int64_t T, int64_t E, int64_t k);

/*
 * The gradient of the logits through the weights (the choice is held fixed):
 * dlogits [T, E] of logits' type from dweights [T, k] (fp32).  ids as route wrote them:
 * distinct within a row; an id outside [0, E) adds nothing.  Every element is written.
 */
fp8gg_status f8f8bf16_route_backward(
    const void* logits, int logits_dtype, const int32_t* ids, const float* dweights, int score, int renormalize,
    float scale, void* dlogits, int64_t T, int64_t E, int64_t k, void* stream);

/*
 * Token order to expert order: row dst_row[t, j] of XQs and xs_out = row t of XQ and
 * x_scale, for every j.  Entries of dst_row outside [0, R) are left out; rows that no
 * entry names are not written; two entries must not name the same row.
 *
 *   XQ       [T, K]            bytes        XQs     [R, K]
 *   x_scale  [T, scale_cols]   fp32         xs_out  [R, scale_cols]
 *   dst_row  [T, k]            int32
 *
 * K % 16 == 0, 1 <= scale_cols <= K, k <= 64; XQ and XQs 16-byte aligned.
 */
fp8gg_status f8f8bf16_moe_dispatch(
    const uint8_t* XQ, const float* x_scale, int64_t scale_cols, const int32_t* dst_row, uint8_t* XQs, float* xs_out,
    int64_t T, int64_t k, int64_t R, int64_t K, void* stream);

/*
 * Expert order back to token order:
 *     out[t] = bf16_rne(sum_j weights[t, j] * Y[dst_row[t, j]] + addend[t])
 * over the j whose dst_row lies in [0, R) (rows left out are not read: what they hold,
 * NaN included, does not matter).
 *
 *   Y        [R, N]  bf16        weights  [T, k]  fp32 (or NULL: ones)
 *   addend   [T, N]  bf16 (or NULL)
 *   out      [T, N]  bf16; may be addend itself
 *
 * With weights NULL it is also the gradient of a bf16 dispatch.  N % 8 == 0, k <= 64;
 * bf16 tensors 16-byte aligned.
 */
fp8gg_status f8f8bf16_moe_combine(
    const uint16_t* Y, const int32_t* dst_row, const float* weights, const uint16_t* addend, uint16_t* out,
    int64_t T, int64_t k, int64_t R, int64_t N, void* stream);

/*
 * The gradients of combine:
 *     dY[dst_row[t, j]] = bf16_rne(weights[t, j] * dout[t])
 *     dweights[t, j]    = sum_n dout[t, n] * Y[dst_row[t, j], n]     (0 where dst_row is left out)
 * Two entries must not name the same row (combine itself allows it): one of their
 * gradients would be lost.  Rows of dY that no entry names are not written.  weights NULL:
 * ones.  Y and dweights may both be NULL: then it is a dispatch of bf16 rows.  dY may be Y
 * itself.
 */
fp8gg_status f8f8bf16_moe_combine_backward(
    const uint16_t* dout, const int32_t* dst_row, const float* weights, const uint16_t* Y, uint16_t* dY,
    float* dweights, int64_t T, int64_t k, int64_t R, int64_t N, void* stream);

/*
 * The gated activation between the two products, its fp8 output and the 8-bit
 * checkpoint of its input.  H = [gate | up]:
 *     a = silu(gate) * up,  silu(g) = g / (1 + exp(-g))
 *     AQ, a_scale = codes and scales of a
 *     HQ, h_scale = codes and scales of H, one scale per row, half and 128 columns
 *                   (the last block of a half may be shorter)
 *
 * a has to be finite in fp32.  A sigmoid below 2^-126 (gates below -87) may count as 0, here
 * and in the gradient.
 *
 *   H        [rows, 2 I]   bf16
 *   AQ       [rows, I]     e4m3fn      a_scale  [rows] (block 0) or [rows, I / 128] (block 128)  fp32
 *   HQ       [rows, 2 I]   e4m3fn      h_scale  [rows, 2, ceil(I / 128)]  fp32     (both or neither NULL)
 *
 * I % 8 == 0 (block 128: I % 128 == 0), 0 < I <= 32768.  H 16-byte, AQ and HQ 8-byte aligned.
 */
fp8gg_status f8f8bf16_silu_mul_quantize(
    const uint16_t* H, int block, uint8_t* AQ, float* a_scale, uint8_t* HQ, float* h_scale,
    int64_t rows, int64_t I, void* stream);

/*
 * Its gradient from the checkpoint: with gate and up as HQ and h_scale give them back,
 * dH = bf16_rne([dA * up * sig * (1 + gate * (1 - sig)) | dA * silu(gate)]), sig = 1 / (1 + exp(-gate)).
 *
 *   dA  [rows, I]  bf16     dH  [rows, 2 I]  bf16     HQ, h_scale as above
 */
fp8gg_status f8f8bf16_silu_mul_backward(
    const uint16_t* dA, const uint8_t* HQ, const float* h_scale, uint16_t* dH, int64_t rows, int64_t I, void* stream);

/*
 * The operand of the weight gradient (f8f8bf16_rowwise_grouped_k_offsets) from rows in
 * expert order: the rows of group g become the columns [k_offsets[g-1], k_offsets[g - 1] +
 * M_sizes[g]) of XT, requantised with one scale per group and column of X (the scale
 * that the product applies outside its sum).  Each group's columns are rounded up to 16;
 * the columns between and after are zero.  Every element of XT is written.
 *
 *   X          [R, K]   bf16, or e4m3fn codes (x_dtype) with
 *   x_scale    [R, scale_cols]  fp32, scale_cols 1 or K / 128 (codes only, else NULL and 0)
 *   M_sizes    [G]      int64 rows per group, clamped like the stacked layout's; rows past
 *                       their sum are not read
 *   XT         [K, cap] e4m3fn, cap = f8f8bf16_k_offsets_capacity(R, G)
 *   t_scale    [G, K]   fp32 (1 for an empty group)
 *   k_offsets  [G]      int32 inclusive prefix, multiples of 16
 *   workspace           f8f8bf16_quantize_k_offsets_workspace(R, G, K) bytes, 16-byte aligned
 *
 * K % 16 == 0 (scale_cols K / 128: K % 128 == 0), G <= 1024; X and XT 16-byte aligned.
 */
fp8gg_status f8f8bf16_quantize_k_offsets(
    const void* X, int x_dtype, const float* x_scale, int64_t scale_cols, const int64_t* M_sizes, uint8_t* XT,
    float* t_scale, int32_t* k_offsets, void* workspace, int64_t workspace_bytes,
    int64_t R, int64_t G, int64_t K, void* stream);
int64_t f8f8bf16_quantize_k_offsets_workspace(int64_t R, int64_t G, int64_t K);
int64_t f8f8bf16_k_offsets_capacity(int64_t R, int64_t G);

/* Message describing the last failure of these calls on the calling thread ("" if none). */
const char* f8f8bf16_layer_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* FP8GG_LAYER_H_ */
