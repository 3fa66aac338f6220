// Host side of the training operators' C ABI: argument checks and dispatch.  Every check
// runs before anything is enqueued; nothing here throws or allocates device memory.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <new>
#include <vector>

#include "fp8gg_checks.h"
#include "fp8gg_train.h"
#include "fp8gg_train_internal.h"

using namespace fp8gg;

namespace {

// Compute units of the current device, asked for once per device.
int compute_units() {
  static std::atomic<int> known[64];
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64 && (cus = known[dev].load(std::memory_order_relaxed)) > 0) return cus;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
  if (dev < 64) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

// N and K: the kernels' offsets within 256 rows have 32 bits.
constexpr int64_t kMaxProductWidth = 1 << 22;

fp8gg_status check_product(int64_t G, int64_t M, int64_t N, int64_t K, int weight_size = 2) {
  if (G < 0 || M < 0 || N < 0 || K < 0)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative size (G=%lld total_M=%lld N=%lld K=%lld)", (long long)G, (long long)M,
                (long long)N, (long long)K);
  if (N % 8 != 0 || K % 8 != 0)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "N=%lld and K=%lld must be multiples of 8", (long long)N, (long long)K);
  if (G > kMaxDim || M > kMaxDim || N > kMaxProductWidth || K > kMaxProductWidth)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "G=%lld total_M=%lld N=%lld K=%lld is too large", (long long)G, (long long)M,
                (long long)N, (long long)K);
  // tensors of at most 2^47 bytes
  const double most = std::ldexp(1.0, 47);
  if ((double)M * N * 2 > most || (double)M * K * 2 > most || (double)G * N * K * weight_size > most)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "a tensor of G=%lld total_M=%lld N=%lld K=%lld exceeds 2^47 bytes", (long long)G,
                (long long)M, (long long)N, (long long)K);
  return FP8GG_OK;
}

fp8gg_status check_grid(int64_t grid) {
  if (grid > 0x7FFFFFFFLL)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "grid of %lld workgroups exceeds the launch limit", (long long)grid);
  return FP8GG_OK;
}

// The tensors of a call over gradients.
struct Grads {
  const void* const* g;
  void* const* out;               // or null: not written
  const int64_t* counts;
  const int32_t* dtypes;
  int64_t n;
  int size(int64_t i) const { return dtypes[i] == FP8GG_DTYPE_F32 ? 4 : 2; }
};

fp8gg_status check_grads(const Grads& s) {
  if (s.n < 0) return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative number of tensors (%lld)", (long long)s.n);
  if (s.n > kMaxDim) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "%lld tensors are too many", (long long)s.n);
  if (s.n > 0 && (!s.g || !s.counts || !s.dtypes)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "grads, counts or dtypes is null");
  for (int64_t i = 0; i < s.n; ++i) {
    if (s.dtypes[i] != FP8GG_DTYPE_BF16 && s.dtypes[i] != FP8GG_DTYPE_F32)
      return fail(FP8GG_ERR_INVALID_ARGUMENT, "dtypes[%lld]=%d must be bf16 (0) or fp32 (1)", (long long)i, s.dtypes[i]);
    if (s.counts[i] < 0) return fail(FP8GG_ERR_INVALID_ARGUMENT, "counts[%lld] is negative", (long long)i);
    // the chunks of a launch's tensors are counted in 32 bits (366 GB a tensor)
    if (s.counts[i] > 0x7FFFFFFF / kGradTensors * (int64_t)(kGradChunk / s.size(i)))
      return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "counts[%lld] is too large", (long long)i);
    if (s.counts[i] == 0) continue;
    if (!s.g[i]) return fail(FP8GG_ERR_INVALID_ARGUMENT, "grads[%lld] is null", (long long)i);
    if ((uintptr_t)s.g[i] % s.size(i)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "grads[%lld] is not aligned to its type", (long long)i);
    if (!s.out) continue;
    if (!s.out[i]) return fail(FP8GG_ERR_INVALID_ARGUMENT, "outs[%lld] is null", (long long)i);
    if ((uintptr_t)s.out[i] % s.size(i)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "outs[%lld] is not aligned to its type", (long long)i);
  }
  return FP8GG_OK;
}

// A buffer of the call's own shares no memory with any tensor.
fp8gg_status check_apart(const Grads& s, const char* name, const void* p, int64_t bytes) {
  const uintptr_t from = (uintptr_t)p, to = from + (uintptr_t)bytes;
  if (!p || bytes <= 0) return FP8GG_OK;
  for (int64_t i = 0; i < s.n; ++i) {
    const uintptr_t size = (uintptr_t)s.counts[i] * s.size(i), g = (uintptr_t)s.g[i], o = s.out ? (uintptr_t)s.out[i] : g;
    if (size == 0) continue;
    if (from < g + size && g < to) return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s overlaps grads[%lld]", name, (long long)i);
    if (from < o + size && o < to) return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s overlaps outs[%lld]", name, (long long)i);
  }
  return FP8GG_OK;
}

// No output shares memory with another tensor, its own gradient (the whole of it) aside.
fp8gg_status check_outs(const Grads& s) {
  struct Range {
    uintptr_t from, to;
    int64_t i;
    bool out;
  };
  try {
    std::vector<Range> r;
    r.reserve(2 * s.n);
    for (int64_t i = 0; i < s.n; ++i) {
      if (s.counts[i] == 0) continue;
      const uintptr_t bytes = (uintptr_t)s.counts[i] * s.size(i), o = (uintptr_t)s.out[i], g = (uintptr_t)s.g[i];
      r.push_back({o, o + bytes, i, true});
      if (g != o) r.push_back({g, g + bytes, i, false});
    }
    std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
    // gradients that are only read may overlap each other: the furthest end of either kind so far
    const Range* out = nullptr;
    const Range* in = nullptr;
    for (const Range& x : r) {
      const Range* hit = out && x.from < out->to ? out : x.out && in && x.from < in->to ? in : nullptr;
      if (hit)
        return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s[%lld] overlaps %s[%lld]", x.out ? "outs" : "grads", (long long)x.i,
                    hit->out ? "outs" : "grads", (long long)hit->i);
      const Range*& last = x.out ? out : in;
      if (!last || x.to > last->to) last = &x;
    }
  } catch (const std::bad_alloc&) {
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "no host memory to check %lld tensors", (long long)s.n);
  }
  return FP8GG_OK;
}

// Calls f on the tensors in launches of kGradTensors at most.
template <typename F>
fp8gg_status for_each_launch(const Grads& s, F f) {
  GradArgs a;
  a.tensors = 0;
  a.chunks = 0;
  for (int64_t i = 0; i < s.n; ++i) {
    if (s.counts[i] == 0) continue;
    if (a.tensors == kGradTensors) {
      FP8GG_TRY(f(a));
      a.tensors = 0;
      a.chunks = 0;
    }
    a.t[a.tensors++] = {s.g[i], s.out ? s.out[i] : nullptr, s.counts[i], a.chunks, s.dtypes[i] == FP8GG_DTYPE_F32};
    a.chunks += (uint32_t)grad_chunks(s.g[i], s.counts[i], s.size(i));
  }
  return a.tensors ? f(a) : FP8GG_OK;
}

// The squares' sum as `n` partial sums at `from`: those of the workgroups, or their sum if there were
// several launches.
fp8gg_status squares(const Grads& s, double* sums, int64_t most, hipStream_t stream, const double** from, int* n) {
  int launches = 0, blocks = 0;
  FP8GG_TRY(for_each_launch(s, [&](const GradArgs& a) {
    ++launches;
    const fp8gg_status st = launched(launch_grad_squares(a, sums + blocks, stream), "gradient norm");
    blocks += grad_blocks(a);
    return st;
  }));
  *from = sums;
  *n = blocks;
  if (launches > 1) {
    FP8GG_TRY(launched(launch_grad_join(sums, blocks, sums + most, stream), "gradient norm"));
    *from = sums + most;
    *n = 1;
  }
  return FP8GG_OK;
}

int64_t partial_sums(int64_t n) { return (n + kGradTensors - 1) / kGradTensors * kGradBlocks; }

}  // namespace

extern "C" {

fp8gg_status bf16_grouped_stacked(const uint16_t* X, const uint16_t* W, const int64_t* M_sizes, uint16_t* Y, int64_t G,
                                  int64_t total_M, int64_t N, int64_t K, void* stream) {
  FP8GG_TRY(check_product(G, total_M, N, K));
  if (G == 0 || total_M == 0 || N == 0) return ok();
  FP8GG_TRY(check({{"X", X, total_M * K * 2, 16, false, false},
                   {"W", W, G * N * K * 2, 16, false, false},
                   {"M_sizes", M_sizes, G * 8, 8, false, false},
                   {"Y", Y, total_M * N * 2, 16, true, false}}));
  ProductArgs a{};
  a.P = X;
  a.Q = W;
  a.out = Y;
  a.M_sizes = M_sizes;
  a.M = total_M;
  a.L = K;
  a.C = N;
  a.G = G;
  FP8GG_TRY(check_grid(product_grid(a)));
  return launched(launch_product(false, a, compute_units(), static_cast<hipStream_t>(stream)), "product");
}

fp8gg_status bf16_grouped_stacked_dgrad(const uint16_t* dY, const uint16_t* W, const int64_t* M_sizes, uint16_t* dX,
                                        int64_t G, int64_t total_M, int64_t N, int64_t K, void* stream) {
  FP8GG_TRY(check_product(G, total_M, N, K));
  if (G == 0 || total_M == 0 || K == 0) return ok();
  FP8GG_TRY(check({{"dY", dY, total_M * N * 2, 16, false, false},
                   {"W", W, G * N * K * 2, 16, false, false},
                   {"M_sizes", M_sizes, G * 8, 8, false, false},
                   {"dX", dX, total_M * K * 2, 16, true, false}}));
  ProductArgs a{};
  a.P = dY;
  a.Q = W;
  a.out = dX;
  a.M_sizes = M_sizes;
  a.M = total_M;
  a.L = N;
  a.C = K;
  a.G = G;
  FP8GG_TRY(check_grid(product_grid(a)));
  return launched(launch_product(true, a, compute_units(), static_cast<hipStream_t>(stream)), "product");
}

int64_t bf16_grouped_stacked_wgrad_workspace(int64_t G, int64_t total_M, int64_t N, int64_t K) {
  if (G > kMaxDim || total_M > kMaxDim || N > kMaxProductWidth || K > kMaxProductWidth) return 0;
  const int64_t splits = wgrad_splits(G, total_M, N, K);
  return splits > 1 ? splits * G * N * K * 4 : 0;
}

fp8gg_status bf16_grouped_stacked_wgrad(const uint16_t* dY, const uint16_t* X, const int64_t* M_sizes, void* dW, int dw_dtype,
                                        int accumulate, void* workspace, int64_t workspace_bytes, int64_t G, int64_t total_M,
                                        int64_t N, int64_t K, void* stream) {
  FP8GG_TRY(check_float_type(dw_dtype, "dw_dtype"));
  const bool f32 = dw_dtype == FP8GG_DTYPE_F32;
  FP8GG_TRY(check_product(G, total_M, N, K, f32 ? 4 : 2));
  if (accumulate && !f32) return fail(FP8GG_ERR_INVALID_ARGUMENT, "accumulate needs an fp32 dW");
  if (G == 0 || N == 0 || K == 0) return ok();
  const int64_t need = bf16_grouped_stacked_wgrad_workspace(G, total_M, N, K);
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, need));
  FP8GG_TRY(check({{"dY", dY, total_M * N * 2, 16, false, false},
                   {"X", X, total_M * K * 2, 16, false, false},
                   {"M_sizes", M_sizes, G * 8, 8, false, false},
                   {"dW", dW, G * N * K * (f32 ? 4 : 2), 16, true, false},
                   {"workspace", need ? workspace : nullptr, need, 16, true, true}}));
  ProductArgs a{};
  a.P = dY;
  a.Q = X;
  a.out = dW;
  a.M_sizes = M_sizes;
  a.M = total_M;
  a.L = N;
  a.C = K;
  a.G = G;
  a.partial = static_cast<float*>(workspace);
  a.accumulate = accumulate != 0;
  if (wgrad_tiles(a) > 0x7FFFFFFFLL)             // counted in 32 bits
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "N=%lld and K=%lld make too many tiles", (long long)N, (long long)K);
  return launched(launch_wgrad(f32, a, compute_units(), static_cast<hipStream_t>(stream)), "weight gradient");
}

fp8gg_status f8f8bf16_quantize_groupwise(const uint16_t* X, uint8_t* XQ, float* x_scale, int64_t rows, int64_t K, void* stream) {
  FP8GG_TRY(check_width(rows, "rows", K, "K", 128, kMaxDim));
  if (rows == 0) return ok();
  FP8GG_TRY(check({{"X", X, rows * K * 2, 16, false, false},
                   {"XQ", XQ, rows * K, 16, true, false},
                   {"x_scale", x_scale, rows * (K / 128) * 4, 4, true, false}}));
  return launched(launch_quantize_groupwise(X, XQ, x_scale, rows, K, static_cast<hipStream_t>(stream)), "quantize_groupwise");
}

fp8gg_status f8f8bf16_quantize_groupwise_weight(const void* W, int w_dtype, uint8_t* WQ, float* w_scale, uint8_t* WQt,
                                                float* wt_scale, int64_t G, int64_t N, int64_t K, void* stream) {
  FP8GG_TRY(check_float_type(w_dtype, "w_dtype"));
  if (G < 0 || N < 0 || K < 0)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative size (G=%lld N=%lld K=%lld)", (long long)G, (long long)N, (long long)K);
  if (N % 128 != 0 || K % 128 != 0)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "N=%lld and K=%lld must be multiples of 128", (long long)N, (long long)K);
  if ((WQt == nullptr) != (wt_scale == nullptr))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "WQt and wt_scale are given together or not at all");
  // a workgroup of 256 threads per block, and a launch holds fewer than 2^32 threads
  const double blocks = (double)G * (N / 128) * (K / 128);
  if (G > kMaxDim || N > kMaxDim || K > kMaxDim || blocks >= 1 << 24)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "G=%lld N=%lld K=%lld is too large", (long long)G, (long long)N, (long long)K);
  if (blocks == 0) return ok();
  const int64_t n = G * N * K, scales = (int64_t)blocks * 4;
  const bool f32 = w_dtype == FP8GG_DTYPE_F32;
  FP8GG_TRY(check({{"W", W, n * (f32 ? 4 : 2), 16, false, false},
                   {"WQ", WQ, n, 16, true, false},
                   {"w_scale", w_scale, scales, 4, true, false},
                   {"WQt", WQt, n, 16, true, true},
                   {"wt_scale", wt_scale, scales, 4, true, true}}));
  return launched(launch_quantize_weight({W, WQ, w_scale, WQt, wt_scale, G, N, K, f32}, static_cast<hipStream_t>(stream)),
                  "quantize_groupwise_weight");
}

int64_t f8f8bf16_grad_workspace(int64_t n) { return n <= 0 || n > kMaxDim ? 0 : (partial_sums(n) + 1) * 8; }

fp8gg_status f8f8bf16_grad_square_sum(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int64_t n,
                                      double* square_sum, void* workspace, int64_t workspace_bytes, void* stream) {
  const Grads s{grads, nullptr, counts, dtypes, n};
  FP8GG_TRY(check_grads(s));
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, f8f8bf16_grad_workspace(n)));
  FP8GG_TRY(check({{"square_sum", square_sum, 8, 8, true, false},
                   {"workspace", n ? workspace : nullptr, f8f8bf16_grad_workspace(n), 16, true, true}}));
  FP8GG_TRY(check_apart(s, "square_sum", square_sum, 8));
  FP8GG_TRY(check_apart(s, "workspace", workspace, f8f8bf16_grad_workspace(n)));
  const hipStream_t stream_ = static_cast<hipStream_t>(stream);
  const double* from = nullptr;
  int parts = 0;
  FP8GG_TRY(squares(s, static_cast<double*>(workspace), partial_sums(n), stream_, &from, &parts));
  return launched(launch_grad_join(from, parts, square_sum, stream_), "gradient norm");
}

fp8gg_status f8f8bf16_grad_clip(const void* const* grads, void* const* outs, const int64_t* counts, const int32_t* dtypes,
                                int64_t n, const double* square_sum, double max_norm, double eps, float* norm, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  const Grads s{grads, outs, counts, dtypes, n};
  FP8GG_TRY(check_grads(s));
  if (n > 0 && !outs) return fail(FP8GG_ERR_INVALID_ARGUMENT, "outs is null");
  if (!(max_norm >= 0)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "max_norm=%g must not be negative", max_norm);
  if (!(eps >= 0) || std::isinf(eps)) return fail(FP8GG_ERR_INVALID_ARGUMENT, "eps=%g must be finite and not negative", eps);
  const int64_t need = square_sum ? 0 : f8f8bf16_grad_workspace(n);
  FP8GG_TRY(check_workspace(workspace, workspace_bytes, need));
  FP8GG_TRY(check({{"square_sum", square_sum, 8, 8, false, true},
                   {"norm", norm, 4, 4, true, false},
                   {"workspace", need ? workspace : nullptr, need, 16, true, true}}));
  FP8GG_TRY(check_apart(s, "norm", norm, 4));
  FP8GG_TRY(check_apart(s, "square_sum", square_sum, 8));
  FP8GG_TRY(check_apart(s, "workspace", workspace, need));
  FP8GG_TRY(check_outs(s));
  const hipStream_t stream_ = static_cast<hipStream_t>(stream);
  const double* from = square_sum;
  int parts = 1;
  if (!square_sum) {
    FP8GG_TRY(squares(s, static_cast<double*>(workspace), partial_sums(n), stream_, &from, &parts));
  }
  bool first = true;
  FP8GG_TRY(for_each_launch(s, [&](const GradArgs& a) {
    const fp8gg_status st = launched(launch_grad_scale(a, from, parts, max_norm, eps, first ? norm : nullptr, stream_), "clip");
    first = false;
    return st;
  }));
  if (first) {                        // no values at all: the norm alone
    GradArgs a;
    a.tensors = 0;
    a.chunks = 0;
    return launched(launch_grad_scale(a, from, parts, max_norm, eps, norm, stream_), "clip");
  }
  return ok();
}

}  // extern "C"
