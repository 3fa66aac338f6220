// The norm of all gradients together, and their scaling down to a bound.
//
// The tensors of a launch come in its arguments (no table to copy, so a call may be captured), cut
// into chunks of 16 KB that start on 16-byte boundaries of the tensor's own; workgroup w takes
// chunks w, w + grid, ....  Squares are formed and added in fp64: no gradient that fp32 holds
// over- or underflows there, and the sum does not depend on how many terms it has.  Every
// workgroup's sum goes to a place of its own and these are added in a fixed order: results are
// the same on every run.
//
// Memory is the bound: 270 million values of both types, norm and clipping into other tensors, in 596 us (5.4 TB/s
// over two reads and a write); the additions in fp64 are hidden behind the loads.  A million values in 12 tensors
// take 10 us, two launches of 3 us that wait for one another: every workgroup of the second adds up the first's
// sums, since one more launch between them costs as much as either.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8gg_layer_internal.h"
#include "fp8gg_train_internal.h"

namespace fp8gg {

namespace {

constexpr int kThreads = 256;

// The first chunk of every tensor, one or two per lane.
struct Firsts {
  uint32_t lo, hi;
  __device__ __forceinline__ explicit Firsts(const GradArgs& a) {
    const int lane = threadIdx.x & 63;
    static_assert(kGradTensors <= 128, "two per lane");
    lo = lane < a.tensors ? a.t[lane].first : ~0u;
    hi = lane + 64 < a.tensors ? a.t[lane + 64].first : ~0u;
  }
  // The tensor that chunk c belongs to (every tensor has at least one).
  __device__ __forceinline__ int of(uint32_t c) const {
    return __builtin_popcountll(__ballot(lo <= c)) + __builtin_popcountll(__ballot(hi <= c)) - 1;
  }
};

// A chunk's values: [s0, s1) one by one, then n16 vectors of 16 bytes from v0 on, then [e0, e1).
struct Chunk {
  int64_t s0, s1, v0, e0, e1;
  int n16;
};

template <int SIZE>
__device__ __forceinline__ Chunk chunk_of(const GradTensor& t, uint32_t nth) {
  constexpr int PER = 16 / SIZE;
  const int64_t head = grad_head(t.g, t.n, SIZE), at = head + (int64_t)nth * (kGradChunk / SIZE);
  const int64_t end = at + kGradChunk / SIZE < t.n ? at + kGradChunk / SIZE : t.n;
  Chunk c;
  c.s0 = 0;
  c.s1 = nth == 0 ? head : 0;
  c.v0 = at;
  c.n16 = end > at ? (int)((end - at) / PER) : 0;
  c.e0 = at + (int64_t)c.n16 * PER;
  c.e1 = end;
  return c;
}

__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }

__device__ __forceinline__ double square(float x, double sum) { return __builtin_fma((double)x, (double)x, sum); }

template <typename T>
__device__ __forceinline__ double chunk_squares(const GradTensor& t, uint32_t nth) {
  constexpr int SIZE = sizeof(T), VECS = kGradChunk / 16 / kThreads;
  const Chunk c = chunk_of<SIZE>(t, nth);
  const T* g = (const T*)t.g;
  u32x4 v[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int at = i * kThreads + threadIdx.x;
    v[i] = at < c.n16 ? __builtin_nontemporal_load((const u32x4*)(g + c.v0) + at) : u32x4{0, 0, 0, 0};
  }
  double s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < VECS; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (SIZE == 4) {
        s[e] = square(__uint_as_float(v[i][e]), s[e]);
      } else {
        s[e] = square(__uint_as_float(v[i][e] << 16), s[e]);
        s[e] = square(__uint_as_float(v[i][e] & 0xFFFF0000u), s[e]);
      }
    }
  for (int64_t i = c.s0 + threadIdx.x; i < c.s1; i += kThreads) s[0] = square(value(g + i), s[0]);
  for (int64_t i = c.e0 + threadIdx.x; i < c.e1; i += kThreads) s[0] = square(value(g + i), s[0]);
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// The sum over a workgroup, in every thread.
__device__ __forceinline__ double block_sum(double s, double* lds) {
  s = wave_reduce(s, AddF{});
  if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = s;
  __syncthreads();
  double all = lds[0];
#pragma unroll
  for (int w = 1; w < kThreads / 64; ++w) all += lds[w];
  return all;
}

__global__ void __launch_bounds__(kThreads) grad_squares_kernel(GradArgs a, double* __restrict__ partial) {
  __shared__ double lds[kThreads / 64];
  const Firsts first(a);
  double sum = 0;
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int i = __builtin_amdgcn_readfirstlane(first.of(c));
    const GradTensor& t = a.t[i];
    sum += t.f32 ? chunk_squares<float>(t, c - t.first) : chunk_squares<uint16_t>(t, c - t.first);
  }
  sum = block_sum(sum, lds);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// The same order of additions wherever it is done.
__device__ __forceinline__ double join(const double* partial, int n, double* lds) {
  double s = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += partial[i];
  return block_sum(s, lds);
}

__global__ void __launch_bounds__(kThreads) grad_join_kernel(const double* __restrict__ partial, int n, double* __restrict__ sum) {
  __shared__ double lds[kThreads / 64];
  const double s = join(partial, n, lds);
  if (threadIdx.x == 0) *sum = s;
}

__device__ __forceinline__ uint32_t scaled2(uint32_t w, float f) {
  return pack_bf16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const GradTensor& t, uint32_t nth, float f) {
  constexpr int SIZE = sizeof(T), VECS = kGradChunk / 16 / kThreads;
  Chunk c = chunk_of<SIZE>(t, nth);
  const T* g = (const T*)t.g;
  T* o = (T*)t.out;
  const auto one = [&](int64_t i) {
    if constexpr (SIZE == 4) o[i] = g[i] * f;
    else o[i] = __builtin_bit_cast(uint16_t, (__bf16)(value(g + i) * f));
  };
  if (((uintptr_t)g - (uintptr_t)o) % 16 != 0) {   // the output's boundaries lie elsewhere
    c.e0 = c.v0;
    c.n16 = 0;
  }
  u32x4 v[VECS];
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int at = i * kThreads + threadIdx.x;
    v[i] = at < c.n16 ? __builtin_nontemporal_load((const u32x4*)(g + c.v0) + at) : u32x4{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < VECS; ++i) {
    const int at = i * kThreads + threadIdx.x;
    u32x4 r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = SIZE == 4 ? __float_as_uint(__uint_as_float(v[i][e]) * f) : scaled2(v[i][e], f);
    if (at < c.n16) store_out((u32x4*)(o + c.v0) + at, r);
  }
  for (int64_t i = c.s0 + threadIdx.x; i < c.s1; i += kThreads) one(i);
  for (int64_t i = c.e0 + threadIdx.x; i < c.e1; i += kThreads) one(i);
}

__global__ void __launch_bounds__(kThreads) grad_scale_kernel(GradArgs a, const double* __restrict__ partial, int n, double max_norm,
                                                              double eps, float* __restrict__ norm_out) {
  __shared__ double lds[kThreads / 64];
  const double norm = __builtin_sqrt(join(partial, n, lds));
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = (float)norm;
  // Without a bound, or over a denominator of 0, there is nothing to scale down, whatever the norm: the quotient would be
  // NaN there.  Otherwise only a NaN norm gives NaN, which reaches the gradients (the comparison is false).
  const double under = norm + eps, factor = __builtin_isinf(max_norm) || under == 0.0 ? 1.0 : max_norm / under;
  const bool keep = factor >= 1.0;
  const float f = keep ? 1.0f : (float)factor;
  const Firsts first(a);
  for (uint32_t c = blockIdx.x; c < a.chunks; c += gridDim.x) {
    const int i = __builtin_amdgcn_readfirstlane(first.of(c));
    const GradTensor& t = a.t[i];
    if (keep && t.out == t.g) continue;
    if (t.f32) scale_chunk<float>(t, c - t.first, f);
    else scale_chunk<uint16_t>(t, c - t.first, f);
  }
}

}  // namespace

int grad_blocks(const GradArgs& a) { return a.chunks < (uint32_t)kGradBlocks ? (int)a.chunks : kGradBlocks; }

hipError_t launch_grad_squares(const GradArgs& a, double* partial, hipStream_t stream) {
  hipLaunchKernelGGL(grad_squares_kernel, dim3((uint32_t)grad_blocks(a)), dim3(kThreads), 0, stream, a, partial);
  return hipGetLastError();
}

hipError_t launch_grad_join(const double* partial, int n, double* sum, hipStream_t stream) {
  hipLaunchKernelGGL(grad_join_kernel, dim3(1), dim3(kThreads), 0, stream, partial, n, sum);
  return hipGetLastError();
}

hipError_t launch_grad_scale(const GradArgs& a, const double* partial, int n, double max_norm, double eps, float* norm,
                             hipStream_t stream) {
  const int blocks = grad_blocks(a);
  hipLaunchKernelGGL(grad_scale_kernel, dim3((uint32_t)(blocks > 0 ? blocks : 1)), dim3(kThreads), 0, stream, a, partial, n,
                     max_norm, eps, norm);
  return hipGetLastError();
}

}  // namespace fp8gg
