// Internal interface of the training operators (include/fp8gg_train.h): arguments as the
// kernels see them, and launchers.
#ifndef FP8GG_TRAIN_INTERNAL_H_
#define FP8GG_TRAIN_INTERNAL_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8gg {

// A product of bf16 matrices by group.
//   forward              P = X [M, L]    Q = W [G, C, L]   out [M, C]
//   input's gradient     P = dY [M, L]   Q = W [G, L, C]   out [M, C]
//   weights' gradient    P = dY [M, L]   Q = X [M, C]      out [G, L, C]
struct ProductArgs {
  const uint16_t* P;
  const uint16_t* Q;
  void* out;
  const int64_t* M_sizes;
  int64_t M, L, C;
  int64_t G;
  float* partial;                 // [splits, G, L, C], splits > 1 only
  int32_t accumulate;
  // set by the launcher
  uint32_t splits;
  uint32_t row_tiles, col_tiles;
};

struct WeightBlocksArgs {
  const void* W;                  // bf16, or fp32 when f32
  uint8_t* WQ;
  float* w_scale;
  uint8_t* WQt;                   // or null
  float* wt_scale;
  int64_t G, N, K;
  int32_t f32;
};

// Tensors of one launch over gradients, 32 bytes each: a launch's arguments stay below 4 KB.
constexpr int kGradTensors = 96;
struct GradTensor {
  const void* g;
  void* out;
  int64_t n;
  uint32_t first;                 // the tensor's first chunk in the launch
  uint32_t f32;
};
struct GradArgs {
  GradTensor t[kGradTensors];
  int32_t tensors;
  uint32_t chunks;
};
// Bytes of a gradient that one workgroup takes at a time, and the most workgroups of a launch.
constexpr int kGradChunk = 16384;
constexpr int kGradBlocks = 2048;
// Values before a tensor's first 16-byte boundary.
__host__ __device__ inline int64_t grad_head(const void* p, int64_t n, int size) {
  const int64_t h = (int64_t)((16 - (uintptr_t)p % 16) % 16) / size;
  return h < n ? h : n;
}
__host__ __device__ inline int64_t grad_chunks(const void* p, int64_t n, int size) {
  const int64_t body = n - grad_head(p, n, size), per = kGradChunk / size;
  return body <= per ? 1 : (body + per - 1) / per;
}

// Parts that the rows of each group are split into for the weights' gradient, from the sizes that
// the host knows.
int wgrad_splits(int64_t G, int64_t M, int64_t N, int64_t K);

hipError_t launch_product(bool transposed, ProductArgs a, int cus, hipStream_t stream);
hipError_t launch_wgrad(bool f32, ProductArgs a, int cus, hipStream_t stream);
// Workgroups of the largest launch that a product may need, to be checked against the limit.
int64_t product_grid(const ProductArgs& a);
int64_t wgrad_tiles(const ProductArgs& a);
hipError_t launch_quantize_groupwise(const uint16_t* X, uint8_t* XQ, float* x_scale, int64_t rows, int64_t K,
                                     hipStream_t stream);
hipError_t launch_quantize_weight(const WeightBlocksArgs& a, hipStream_t stream);
hipError_t launch_grad_squares(const GradArgs& a, double* partial, hipStream_t stream);
int grad_blocks(const GradArgs& a);
// partial[0 .. n) to one sum.
hipError_t launch_grad_join(const double* partial, int n, double* sum, hipStream_t stream);
hipError_t launch_grad_scale(const GradArgs& a, const double* partial, int n, double max_norm, double eps, float* norm,
                             hipStream_t stream);

}  // namespace fp8gg

#endif  // FP8GG_TRAIN_INTERNAL_H_
