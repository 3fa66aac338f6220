/*
 * fp8gg_train.h -- C ABI of the operators for training the experts of a mixture-of-experts
 * layer (MI355X, gfx950): the products by group in bf16 with both gradients, the operands of
 * the block-scaled products, and the norm of all gradients with their clipping.
 *
 * A training step of a layer kept in bf16 (the gated activation between its products is the
 * caller's: fp8gg_layer.h has it for 8-bit operands only):
 *
 *     grouped_stacked -> ... -> grouped_stacked_dgrad, grouped_stacked_wgrad -> grad_clip
 *
 * and of one in fp8 with a scale per block of 128 (fp8gg.h has the product):
 *
 *     quantize_groupwise_weight once per step -> f8f8bf16_groupwise_grouped_stacked on WQ
 *       -> quantize_groupwise of dY -> f8f8bf16_groupwise_grouped_stacked on WQt for the
 *       input's gradient, grouped_stacked_wgrad for the weights' -> grad_clip
 *
 * Conventions are those of fp8gg_layer.h: device pointers, dense row-major tensors, work
 * only enqueued on `stream`, nothing allocated, copied to the host or synchronised, every
 * call may be captured into a graph, results deterministic; a failed check returns a
 * non-zero status, enqueues nothing and leaves a message for f8f8bf16_layer_last_error().
 * Buffers of one call must not overlap unless a line says so.  A workspace may serve any
 * number of calls one after the other on a stream; calls that may run at the same time
 * (other streams, graphs launched side by side) need one each.
 */
#ifndef FP8GG_TRAIN_H_
#define FP8GG_TRAIN_H_

#include <stdint.h>

#include "fp8gg_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Products of bf16 matrices by group, in the stacked layout: group g owns the next
 * M_sizes[g] rows of X, Y, dX and dY.  Sums of products in fp32, rounded once (to nearest
 * even) where the output is bf16.  The order of a sum's terms depends on G, total_M, N and K,
 * in bf16_grouped_stacked also on the group's index (groups of few rows start at different
 * places of the contraction), and on nothing else: at the same sizes a row of Y or dX has the
 * same bits wherever it lies in its group and whatever the other rows and M_sizes are, and
 * dW[g] depends on its group's rows and their order alone.
 *
 *     Y[m, n]  = sum_k X[m, k] W[g, n, k]              bf16_grouped_stacked
 *     dX[m, k] = sum_n dY[m, n] W[g, n, k]             bf16_grouped_stacked_dgrad
 *     dW[g, n, k] (+)= sum_{m in g} dY[m, n] X[m, k]   bf16_grouped_stacked_wgrad
 *
 *   X, dX    [total_M, K]   bf16
 *   Y, dY    [total_M, N]   bf16
 *   W        [G, N, K]      bf16, read as it lies by both
 *   M_sizes  [G]            int64 rows per group, on the device, clamped like the stacked
 *                           layout's of fp8gg.h (negative: 0, ends past total_M: total_M)
 *   dW       [G, N, K]      bf16 or fp32 (dw_dtype); accumulate (fp32 only): added to what
 *                           dW holds, else every element is written, zeros for a group
 *                           without rows
 *   workspace               bf16_grouped_stacked_wgrad_workspace(G, total_M, N, K) bytes
 *                           (often 0, and for negative sizes or those past the bounds below),
 *                           16-byte aligned; NULL when that is 0
 *
 * Rows at or beyond the groups' end are neither read nor written.  What a row or column
 * holds, infinities and NaN included, reaches only the results that depend on it.  An empty
 * contraction (K or N = 0) gives zeros.
 *
 * N % 8 == 0, K % 8 == 0, both at most 2^22; tensors 16-byte aligned, M_sizes 8-byte.  G and
 * total_M below 2^31 - 256, every tensor at most 2^47 bytes.
 */
fp8gg_status bf16_grouped_stacked(
    const uint16_t* X, const uint16_t* W, const int64_t* M_sizes, uint16_t* Y,
    int64_t G, int64_t total_M, int64_t N, int64_t K, void* stream);
fp8gg_status bf16_grouped_stacked_dgrad(
    const uint16_t* dY, const uint16_t* W, const int64_t* M_sizes, uint16_t* dX,
    int64_t G, int64_t total_M, int64_t N, int64_t K, void* stream);
fp8gg_status bf16_grouped_stacked_wgrad(
    const uint16_t* dY, const uint16_t* X, const int64_t* M_sizes, void* dW, int dw_dtype, int accumulate,
    void* workspace, int64_t workspace_bytes, int64_t G, int64_t total_M, int64_t N, int64_t K, void* stream);
int64_t bf16_grouped_stacked_wgrad_workspace(int64_t G, int64_t total_M, int64_t N, int64_t K);

/*
 * Rows as an operand of the block-scaled products: one scale per row and 128 columns.  Codes
 * and scales are those of fp8gg_layer.h (s = max(amax, 2^-100) / 448, 1 when amax is 0), but
 * for the midpoints: here a code is always the nearest to the value over the real s (of
 * which the scale returned is a rounding), ties to the even one.  The same of the weights' below.
 *
 *   X        [rows, K]         bf16
 *   XQ       [rows, K]         e4m3fn
 *   x_scale  [rows, K / 128]   fp32
 *
 * K % 128 == 0, K > 0; X and XQ 16-byte aligned.
 */
fp8gg_status f8f8bf16_quantize_groupwise(
    const uint16_t* X, uint8_t* XQ, float* x_scale, int64_t rows, int64_t K, void* stream);

/*
 * Weights as operands of the block-scaled products: one scale per 128 x 128 block, and from
 * the same codes the transposed operand that the input's gradient takes (a block's scale
 * serves both), in one pass over the weights.
 *
 *   W         [G, N, K]               bf16 or fp32 (w_dtype)
 *   WQ        [G, N, K]               e4m3fn
 *   w_scale   [G, N / 128, K / 128]   fp32
 *   WQt       [G, K, N]               e4m3fn, WQt[g, k, n] = WQ[g, n, k]     (both or neither NULL)
 *   wt_scale  [G, K / 128, N / 128]   fp32
 *
 * N % 128 == 0, K % 128 == 0; W, WQ and WQt 16-byte aligned, fewer than 2^24 blocks
 * (2^38 values).
 */
fp8gg_status f8f8bf16_quantize_groupwise_weight(
    const void* W, int w_dtype, uint8_t* WQ, float* w_scale, uint8_t* WQt, float* wt_scale,
    int64_t G, int64_t N, int64_t K, void* stream);

/*
 * The norm of all gradients taken together, and their scaling down to a bound.
 *
 *     square_sum = sum_i sum_j grads[i][j]^2                       (fp64)
 *     norm       = sqrt(square_sum)
 *     outs[i]    = grads[i] * factor                               (rounded to the type)
 *     factor     = min(1, max_norm / (norm + eps));  1 where max_norm is infinite or norm + eps is 0
 *
 *   grads, outs   n device pointers each, in host memory: bf16 or fp32 tensors (dtypes),
 *                 counts[i] values (366 GB at most), aligned to their type; an empty tensor's
 *                 may be NULL.
 *                 outs[i] may be grads[i] (the whole of it); nothing is written there when
 *                 the factor is 1.  The arrays are read before the call returns.
 *   square_sum    [1] fp64: grad_square_sum writes it; grad_clip takes it where it is given
 *                 (sums of several ranks, added up), else (NULL) forms its own
 *   norm          [1] fp32 (infinite where fp32 does not hold it; the factor goes by fp64's)
 *   max_norm      >= 0, infinity: the norm alone            eps  >= 0, finite
 *   workspace     f8f8bf16_grad_workspace(n) bytes, 16-byte aligned; not read where
 *                 grad_clip is given square_sum
 *
 * Under a finite max_norm a norm that is infinite gives the factor 0 (finite gradients become
 * 0, infinite ones NaN), one that is NaN makes every gradient NaN.  Under an infinite max_norm
 * the factor is 1 whatever the norm, so that a step can be left out by its norm.  The factor
 * is rounded to fp32 before it multiplies.
 */
fp8gg_status f8f8bf16_grad_square_sum(
    const void* const* grads, const int64_t* counts, const int32_t* dtypes, int64_t n, double* square_sum,
    void* workspace, int64_t workspace_bytes, void* stream);
fp8gg_status f8f8bf16_grad_clip(
    const void* const* grads, void* const* outs, const int64_t* counts, const int32_t* dtypes, int64_t n,
    const double* square_sum, double max_norm, double eps, float* norm,
    void* workspace, int64_t workspace_bytes, void* stream);
int64_t f8f8bf16_grad_workspace(int64_t n);

#ifdef __cplusplus
}
#endif

#endif /* FP8GG_TRAIN_H_ */
