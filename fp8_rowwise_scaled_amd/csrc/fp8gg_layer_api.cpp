// Host side of the layer operators' C ABI: argument checks and dispatch.  Every check
// runs before anything is enqueued; nothing here throws or allocates device memory.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "fp8gg_checks.h"
#include "fp8gg_layer.h"
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

// A plain buffer, so that no error path allocates.
thread_local char g_error[512] = "";

}  // namespace

fp8gg_status fail(fp8gg_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_error, sizeof g_error, fmt, ap);
  va_end(ap);
  return st;
}

fp8gg_status ok() {
  g_error[0] = 0;
  return FP8GG_OK;
}

}  // namespace fp8gg

using namespace fp8gg;

namespace {

fp8gg_status check_pairs(int64_t T, int64_t k, int64_t R) {
  if (T < 0 || k < 0 || R < 0)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative size (T=%lld k=%lld R=%lld)", (long long)T, (long long)k, (long long)R);
  if (k > 64) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "k=%lld exceeds 64", (long long)k);
  if (T > kMaxDim || R > kMaxDim || T * k > kMaxDim)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "T=%lld k=%lld R=%lld is too large", (long long)T, (long long)k, (long long)R);
  return FP8GG_OK;
}

}  // namespace

extern "C" {

fp8gg_status f8f8bf16_rmsnorm_quantize(const uint16_t* X, const uint16_t* residual, const void* weight, int weight_dtype,
                                       float eps, int block, uint8_t* XQ, float* x_scale, uint16_t* Y,
                                       uint16_t* residual_out, float* rstd, int64_t rows, int64_t K, void* stream) {
  FP8GG_TRY(check_width(rows, "rows", K, "K", 8, kMaxRowWidth));
  FP8GG_TRY(check_block(block, K, "K"));
  FP8GG_TRY(check_float_type(weight_dtype, "weight_dtype"));
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "eps=%g must be finite and not negative", eps);
  if ((residual != nullptr) != (residual_out != nullptr))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "residual and residual_out are given together or not at all");
  if (rows == 0) return ok();
  const int64_t n = rows * K, scales = block ? rows * (K / 128) : rows;
  FP8GG_TRY(check({{"X", X, 2 * n, 16, false, false},
                   {"residual", residual, 2 * n, 16, false, true},
                   {"weight", weight, K * (weight_dtype == FP8GG_DTYPE_F32 ? 4 : 2), 16, false, false},
                   {"XQ", XQ, n, 8, true, false},
                   {"x_scale", x_scale, 4 * scales, 4, true, false},
                   {"Y", Y, 2 * n, 16, true, true},
                   {"residual_out", residual_out, 2 * n, 16, true, true},
                   {"rstd", rstd, 4 * rows, 4, true, true}},
                  {{"residual", "residual_out"}}));
  const fp8gg::NormArgs a{X, residual, weight, XQ, x_scale, Y, residual_out, rstd, rows, (int32_t)K,
                          weight_dtype == FP8GG_DTYPE_F32, eps, 0};
  return launched(fp8gg::launch_rmsnorm_quantize(a, block, static_cast<hipStream_t>(stream)), "rmsnorm_quantize");
}

int64_t f8f8bf16_rmsnorm_backward_workspace(int64_t rows, int64_t K) {
  if (rows <= 0 || K <= 0 || K > kMaxRowWidth) return 0;
  return (int64_t)fp8gg::norm_backward_parts(rows, K) * K * 4;
}

fp8gg_status f8f8bf16_rmsnorm_backward(const uint16_t* dY, const uint16_t* H, const void* weight, int weight_dtype,
                                       const float* rstd, const uint16_t* dresidual, uint16_t* dX, float* dweight,
                                       void* workspace, int64_t workspace_bytes, int64_t rows, int64_t K, void* stream) {
  FP8GG_TRY(check_width(rows, "rows", K, "K", 8, kMaxRowWidth));
  FP8GG_TRY(check_float_type(weight_dtype, "weight_dtype"));
  const int64_t n = rows * K, need = f8f8bf16_rmsnorm_backward_workspace(rows, K);
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, need));
  FP8GG_TRY(check({{"dY", dY, 2 * n, 16, false, false},
                   {"H", H, 2 * n, 16, false, false},
                   {"weight", weight, rows ? K * (weight_dtype == FP8GG_DTYPE_F32 ? 4 : 2) : 0, 16, false, false},
                   {"rstd", rstd, 4 * rows, 4, false, false},
                   {"dresidual", dresidual, 2 * n, 16, false, true},
                   {"dX", dX, 2 * n, 16, true, false},
                   {"dweight", dweight, 4 * K, 16, true, false},
                   {"workspace", workspace, need, 16, true, true}},
                  {{"dX", "dY"}, {"dX", "dresidual"}}));
  const fp8gg::NormBackwardArgs a{dY, H, weight, rstd, dresidual, dX, dweight, static_cast<float*>(workspace), rows,
                                  (int32_t)K, weight_dtype == FP8GG_DTYPE_F32,
                                  rows ? fp8gg::norm_backward_parts(rows, K) : 0};
  return launched(fp8gg::launch_rmsnorm_backward(a, static_cast<hipStream_t>(stream)), "rmsnorm_backward");
}

int64_t f8f8bf16_route_workspace(int64_t T, int64_t E, int64_t k) {
  if (T <= 0 || E <= 0 || k <= 0 || T > kMaxDim || E > 1024 || k > 16 || T * k <= fp8gg::kLonePairs) return 0;
  return fp8gg::route_count_rows(T, E) * fp8gg::count_row(E) * 4;
}

// Sizes and enumerations shared by route and its gradient.
static fp8gg_status check_route(int logits_dtype, int score, float scale, int64_t T, int64_t E, int64_t k) {
  FP8GG_TRY(check_float_type(logits_dtype, "logits_dtype"));
  if (score != FP8GG_SCORE_SOFTMAX && score != FP8GG_SCORE_SIGMOID)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "score=%d must be softmax (0) or sigmoid (1)", score);
  if (!std::isfinite(scale)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "scale must be finite");
  if (T < 0 || E < 0 || k < 0)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative size (T=%lld E=%lld k=%lld)", (long long)T, (long long)E, (long long)k);
  if (E < 1 || E > 1024) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "E=%lld must lie in 1..1024", (long long)E);
  if (k < 1 || k > 16 || k > E)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "k=%lld must lie in 1..16 and not exceed E=%lld", (long long)k, (long long)E);
  if (T > kMaxDim || T * k > kMaxDim) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "T=%lld is too large", (long long)T);
  return FP8GG_OK;
}

fp8gg_status f8f8bf16_route(const void* logits, int logits_dtype, const float* bias, int score, int64_t n_group,
                            int64_t topk_group, int group_top, int renormalize, float scale, float* weights, int32_t* ids,
                            int64_t* M_sizes, int32_t* dst_row, void* workspace, int64_t workspace_bytes, int64_t T,
                            int64_t E, int64_t k, void* stream) {
  FP8GG_TRY(check_route(logits_dtype, score, scale, T, E, k));
  if (n_group < 1 || n_group > 16 || E % n_group != 0)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "n_group=%lld must lie in 1..16 and divide E=%lld", (long long)n_group,
                (long long)E);
  if (topk_group < 1 || topk_group > n_group)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "topk_group=%lld must lie in 1..n_group=%lld", (long long)topk_group,
                (long long)n_group);
  if (group_top != 1 && group_top != 2) return fail(FP8GG_ERR_INVALID_ARGUMENT, "group_top=%d must be 1 or 2", group_top);
  if (T > 0 && (M_sizes != nullptr) != (dst_row != nullptr))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "M_sizes and dst_row are given together or not at all");
  const bool plan = M_sizes != nullptr;
  const int64_t need = plan ? f8f8bf16_route_workspace(T, E, k) : 0;
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, need));
  const int64_t elem = logits_dtype == FP8GG_DTYPE_F32 ? 4 : 2;
  FP8GG_TRY(check({{"logits", logits, T * E * elem, 16, false, false},
                   {"bias", bias, 4 * E, 4, false, true},
                   {"weights", weights, 4 * T * k, 4, true, false},
                   {"ids", ids, 4 * T * k, 4, true, false},
                   {"M_sizes", M_sizes, 8 * E, 8, true, true},
                   {"dst_row", dst_row, 4 * T * k, 4, true, true},
                   {"workspace", workspace, need, 16, true, true}}));
  const fp8gg::RouteArgs a{logits, bias, weights, ids, M_sizes, dst_row,
                           need > 0 ? static_cast<int32_t*>(workspace) : nullptr, T, (int32_t)E, (int32_t)k, (int32_t)n_group, (int32_t)topk_group, group_top,
                           logits_dtype == FP8GG_DTYPE_BF16, score == FP8GG_SCORE_SIGMOID, renormalize != 0,
                           scale, 0, 0, 0, false};
  return launched(fp8gg::launch_route(a, static_cast<hipStream_t>(stream)), "route");
}

fp8gg_status f8f8bf16_route_backward(const void* logits, int logits_dtype, const int32_t* ids, const float* dweights,
                                     int score, int renormalize, float scale, void* dlogits, int64_t T, int64_t E,
                                     int64_t k, void* stream) {
  FP8GG_TRY(check_route(logits_dtype, score, scale, T, E, k));
  const int64_t elem = logits_dtype == FP8GG_DTYPE_F32 ? 4 : 2;
  FP8GG_TRY(check({{"logits", logits, T * E * elem, 16, false, false},
                   {"ids", ids, 4 * T * k, 4, false, false},
                   {"dweights", dweights, 4 * T * k, 4, false, false},
                   {"dlogits", dlogits, T * E * elem, 16, true, false}}));
  const fp8gg::RouteBackwardArgs a{logits, ids, dweights, dlogits, T, (int32_t)E, (int32_t)k,
                                   logits_dtype == FP8GG_DTYPE_BF16, score == FP8GG_SCORE_SIGMOID, renormalize != 0, scale};
  return launched(fp8gg::launch_route_backward(a, static_cast<hipStream_t>(stream)), "route_backward");
}

fp8gg_status f8f8bf16_moe_dispatch(const uint8_t* XQ, const float* x_scale, int64_t scale_cols, const int32_t* dst_row,
                                   uint8_t* XQs, float* xs_out, int64_t T, int64_t k, int64_t R, int64_t K, void* stream) {
  FP8GG_TRY(check_width(T, "T", K, "K", 16, kMaxDim));
  FP8GG_TRY(check_pairs(T, k, R));
  if (scale_cols < 1 || scale_cols > K)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "scale_cols=%lld must lie in 1..K=%lld", (long long)scale_cols, (long long)K);
  if (R > (int64_t(1) << 46) / K) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "R=%lld is too large", (long long)R);
  if (T == 0 || k == 0 || R == 0) return ok();
  FP8GG_TRY(check({{"XQ", XQ, T * K, 16, false, false},
                   {"x_scale", x_scale, 4 * T * scale_cols, 4, false, false},
                   {"dst_row", dst_row, 4 * T * k, 4, false, false},
                   {"XQs", XQs, R * K, 16, true, false},
                   {"xs_out", xs_out, 4 * R * scale_cols, 4, true, false}}));
  const fp8gg::DispatchArgs a{XQ, x_scale, dst_row, XQs, xs_out, T, R, (int32_t)k, (int32_t)K, (int32_t)scale_cols};
  return launched(fp8gg::launch_dispatch(a, static_cast<hipStream_t>(stream)), "moe_dispatch");
}

fp8gg_status f8f8bf16_moe_combine(const uint16_t* Y, const int32_t* dst_row, const float* weights, const uint16_t* addend,
                                  uint16_t* out, int64_t T, int64_t k, int64_t R, int64_t N, void* stream) {
  FP8GG_TRY(check_width(T, "T", N, "N", 8, kMaxDim));
  FP8GG_TRY(check_pairs(T, k, R));
  if (R > (int64_t(1) << 46) / N) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "R=%lld is too large", (long long)R);
  if (T == 0) return ok();
  FP8GG_TRY(check({{"Y", Y, k ? 2 * R * N : 0, 16, false, false},
                   {"dst_row", dst_row, 4 * T * k, 4, false, false},
                   {"weights", weights, 4 * T * k, 4, false, true},
                   {"addend", addend, 2 * T * N, 16, false, true},
                   {"out", out, 2 * T * N, 16, true, false}},
                  {{"out", "addend"}}));
  const fp8gg::ExchangeArgs a{Y, dst_row, weights, addend, out, nullptr, T, R, (int32_t)k, (int32_t)N};
  return launched(fp8gg::launch_combine(a, static_cast<hipStream_t>(stream)), "moe_combine");
}

fp8gg_status f8f8bf16_moe_combine_backward(const uint16_t* dout, const int32_t* dst_row, const float* weights,
                                           const uint16_t* Y, uint16_t* dY, float* dweights, int64_t T, int64_t k,
                                           int64_t R, int64_t N, void* stream) {
  FP8GG_TRY(check_width(T, "T", N, "N", 8, kMaxDim));
  FP8GG_TRY(check_pairs(T, k, R));
  if (R > (int64_t(1) << 46) / N) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "R=%lld is too large", (long long)R);
  if (T == 0 || k == 0) return ok();
  if (R > 0 && (Y != nullptr) != (dweights != nullptr))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "Y and dweights are given together or not at all");
  FP8GG_TRY(check({{"dout", dout, 2 * T * N, 16, false, false},
                   {"dst_row", dst_row, 4 * T * k, 4, false, false},
                   {"weights", weights, 4 * T * k, 4, false, true},
                   {"Y", Y, 2 * R * N, 16, false, true},
                   {"dY", dY, 2 * R * N, 16, true, false},
                   {"dweights", dweights, 4 * T * k, 4, true, true}},
                  {{"dY", "Y"}}));
  const fp8gg::ExchangeArgs a{dout, dst_row, weights, Y, dY, dweights, T, R, (int32_t)k, (int32_t)N};
  return launched(fp8gg::launch_combine_backward(a, static_cast<hipStream_t>(stream)), "moe_combine_backward");
}

fp8gg_status f8f8bf16_silu_mul_quantize(const uint16_t* H, int block, uint8_t* AQ, float* a_scale, uint8_t* HQ,
                                        float* h_scale, int64_t rows, int64_t I, void* stream) {
  FP8GG_TRY(check_width(rows, "rows", I, "I", 8, kMaxRowWidth));
  FP8GG_TRY(check_block(block, I, "I"));
  if ((HQ != nullptr) != (h_scale != nullptr))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "HQ and h_scale are given together or not at all");
  if (rows == 0) return ok();
  const int64_t n = rows * I;
  FP8GG_TRY(check({{"H", H, 4 * n, 16, false, false},
                   {"AQ", AQ, n, 8, true, false},
                   {"a_scale", a_scale, 4 * (block ? rows * (I / 128) : rows), 4, true, false},
                   {"HQ", HQ, 2 * n, 8, true, true},
                   {"h_scale", h_scale, 8 * rows * ((I + 127) / 128), 4, true, true}}));
  const fp8gg::SiluArgs a{H, AQ, a_scale, HQ, h_scale, rows, (int32_t)I, 0};
  return launched(fp8gg::launch_silu_mul_quantize(a, block, static_cast<hipStream_t>(stream)), "silu_mul_quantize");
}

fp8gg_status f8f8bf16_silu_mul_backward(const uint16_t* dA, const uint8_t* HQ, const float* h_scale, uint16_t* dH,
                                        int64_t rows, int64_t I, void* stream) {
  FP8GG_TRY(check_width(rows, "rows", I, "I", 8, kMaxRowWidth));
  if (rows == 0) return ok();
  const int64_t n = rows * I;
  FP8GG_TRY(check({{"dA", dA, 2 * n, 16, false, false},
                   {"HQ", HQ, 2 * n, 8, false, false},
                   {"h_scale", h_scale, 8 * rows * ((I + 127) / 128), 4, false, false},
                   {"dH", dH, 4 * n, 16, true, false}}));
  const fp8gg::SiluBackwardArgs a{dA, HQ, h_scale, dH, rows, (int32_t)I};
  return launched(fp8gg::launch_silu_mul_backward(a, static_cast<hipStream_t>(stream)), "silu_mul_backward");
}

int64_t f8f8bf16_k_offsets_capacity(int64_t R, int64_t G) {
  if (R < 0 || G < 0 || R > kMaxDim || G > 1024) return 0;
  return fp8gg::k_offsets_cap(R, G);
}

int64_t f8f8bf16_quantize_k_offsets_workspace(int64_t R, int64_t G, int64_t K) {
  if (R <= 0 || G <= 0 || K <= 0 || R > kMaxDim || K > kMaxDim || G > 1024) return 0;
  return fp8gg::k_offsets_chunks(R, G) * (K * 4 + (int64_t)sizeof(fp8gg::KChunk));
}

fp8gg_status f8f8bf16_quantize_k_offsets(const void* X, int x_dtype, const float* x_scale, int64_t scale_cols,
                                         const int64_t* M_sizes, uint8_t* XT, float* t_scale, int32_t* k_offsets,
                                         void* workspace, int64_t workspace_bytes, int64_t R, int64_t G, int64_t K,
                                         void* stream) {
  FP8GG_TRY(check_width(R, "R", K, "K", 16, kMaxDim));
  if (G < 1 || G > 1024) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "G=%lld must lie in 1..1024", (long long)G);
  const bool codes = x_dtype == FP8GG_DTYPE_E4M3;
  if (!codes && x_dtype != FP8GG_DTYPE_BF16)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "x_dtype=%d must be bf16 (0) or e4m3 codes (2)", x_dtype);
  if (codes ? (scale_cols != 1 && (scale_cols * 128 != K)) : (x_scale != nullptr || scale_cols != 0))
    return fail(FP8GG_ERR_INVALID_ARGUMENT,
                "codes take x_scale with 1 or K / 128 columns, bf16 rows take none (K=%lld scale_cols=%lld)", (long long)K,
                (long long)scale_cols);
  const int64_t cap = fp8gg::k_offsets_cap(R, G), chunks = fp8gg::k_offsets_chunks(R, G);
  if (cap > kMaxDim || (chunks + 1) * ((K + 127) / 128) > (int64_t(1) << 24) - 1)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "R=%lld K=%lld is too large", (long long)R, (long long)K);
  const int64_t need = f8f8bf16_quantize_k_offsets_workspace(R, G, K);
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, need));
  if (codes && !x_scale && R > 0) return fail(FP8GG_ERR_INVALID_ARGUMENT, "x_scale is null");
  FP8GG_TRY(check({{"X", X, R * K * (codes ? 1 : 2), 16, false, false},
                   {"x_scale", x_scale, 4 * R * scale_cols, 4, false, true},
                   {"M_sizes", M_sizes, 8 * G, 8, false, false},
                   {"XT", XT, K * cap, 16, true, false},
                   {"t_scale", t_scale, 4 * G * K, 4, true, false},
                   {"k_offsets", k_offsets, 4 * G, 4, true, false},
                   {"workspace", workspace, need, 16, true, true}}));
  float* partial = static_cast<float*>(workspace);   // K % 16 == 0 keeps the table behind it aligned
  const fp8gg::KOffsetsArgs a{X, x_scale, M_sizes, XT, t_scale, k_offsets, partial,
                              reinterpret_cast<fp8gg::KChunk*>(partial + chunks * K), R, cap, (int32_t)G, (int32_t)K,
                              (int32_t)scale_cols};
  return launched(fp8gg::launch_quantize_k_offsets(a, static_cast<hipStream_t>(stream)), "quantize_k_offsets");
}

const char* f8f8bf16_layer_last_error(void) { return g_error; }

}  // extern "C"
