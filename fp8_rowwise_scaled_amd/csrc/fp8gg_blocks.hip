// Operands of the block-scaled products: bf16 rows with one scale per row and 128 columns, and
// weights with one scale per block of 128 x 128 in both orders.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8gg_layer_internal.h"
#include "fp8gg_train_internal.h"

namespace fp8gg {

namespace {

// 448 / amax in two parts, whose sum has twice fp32's bits: a value's quotient by its scale is then rounded once
// before its code is, and bf16 values, whose quotients are the middle between two codes or well away from it, get
// the nearest code, ties the even one.  fp32 values need the rest that this rounding drops: where it leaves the
// middle, `nearest` goes a step to the rest's side.  A quotient that is not the middle m itself (5 bits) is 2^-28.95 of m
// away at least: 448 |v| and m amax are whole numbers of some unit below 31 * 2^24.  One that is has a rest of rounding
// errors alone, below 2^-31 of m: those of the second part, which is off by 2^-24 of itself or, below fp32's normal range
// (amax above 2^109), by 2^-150, that is 2^-31.8 of the first part at the largest amax.  So 2^-30 tells the two apart.
// (v times the rounded inverse puts one value in 10^6 on the wrong side; the times are the same.)  The second part is 0
// where amax is not finite.
struct Inverse {
  float hi, lo;
  __device__ __forceinline__ explicit Inverse(float amax) {
    const float a = floored(amax);
    hi = inverse_scale(amax);
    lo = mag(amax) < 0x7F800000u ? __builtin_fmaf(-hi, a, kCodeMax) / a : 0.f;
  }
  __device__ __forceinline__ float operator()(float v) const { return __builtin_fmaf(v, hi, v * lo); }
  __device__ __forceinline__ float nearest(float v) const {
    const float low = v * lo, q = __builtin_fmaf(v, hi, low), rest = __builtin_fmaf(v, hi, -q) + low;
    const uint32_t u = __float_as_uint(q);
    // the middle between two codes has 19 zeros at its end; a step from any other such number keeps its code
    const bool off = (u & 0xFFFFu) == 0 && __builtin_fabsf(rest) > 0x1p-30f * __builtin_fabsf(q);
    return off ? __uint_as_float((rest > 0.f) == (q > 0.f) ? u + 1 : u - 1) : q;
  }
};

// ---------------------------------------------------------------------------
// Rows
// ---------------------------------------------------------------------------
//
// A row is a whole number of blocks, so the tensor is one run of blocks of 128 values (256 bytes),
// and block b's scale is x_scale[b].  Eight lanes take a block, sixteen values each: 32 bytes in, 16 out, and three
// swaps within the eight for the largest magnitude.  Memory is the bound: 16383 x 4096 in 34 us, 5.9 TB/s
// (a 1 GiB copy reaches 5.1 to 5.2); 64 x 7168 in 2.4 us, a launch's latency.  Inputs beyond the caches are read
// past them.

constexpr int kRowsThreads = 256;

template <bool STREAM>
__global__ void __launch_bounds__(kRowsThreads) quantize_groupwise_kernel(const u32x4* __restrict__ X, u32x4* __restrict__ XQ,
                                                                          float* __restrict__ x_scale, int64_t parts) {
  // part: sixteen values, an eighth of a block
  for (int64_t i = (int64_t)blockIdx.x * kRowsThreads + threadIdx.x; i < parts; i += (int64_t)gridDim.x * kRowsThreads) {
    F8 lo = unpack_bf16(load_in<STREAM>(X + 2 * i)), hi = unpack_bf16(load_in<STREAM>(X + 2 * i + 1));
    uint32_t m = mag_max(hi, mag_max(lo, 0));
    m = umax(m, dpp<0xB1>(m));     // lanes 1 0 3 2
    m = umax(m, dpp<0x4E>(m));     // lanes 2 3 0 1
    m = umax(m, dpp<0x141>(m));    // mirror in each half row of eight
    const float amax = __uint_as_float(m);
    const Inverse inv(amax);
#pragma unroll
    for (int e = 0; e < 8; ++e) lo.v[e] = inv(lo.v[e]), hi.v[e] = inv(hi.v[e]);
    const u32x2 a = codes_of(lo, 1.f), b = codes_of(hi, 1.f);
    store_out(XQ + i, u32x4{a[0], a[1], b[0], b[1]});
    if (i % 8 == 0) x_scale[i / 8] = scale_of(amax);
  }
}

// ---------------------------------------------------------------------------
// Weights
// ---------------------------------------------------------------------------
//
// One workgroup per block of 128 x 128.  Thread (j, c) of 8 x 32 holds rows 16 j .. 16 j + 15 of
// columns 4 c .. 4 c + 3: one pass over the block in registers, its largest magnitude, then the
// codes.  Four rows' codes of four columns, a word each, turn into four columns' codes of four rows
// by byte permutations, so a thread has sixteen neighbouring bytes of the transposed block for each
// of its columns; the block is put together in LDS, whose row q * 32 + c holds column 4 c + q and
// whose 16-byte chunks are swapped by c, so that sixteen neighbouring lanes meet no bank twice.  Memory is the bound: fp32 of
// 8 x 4096 x 7168 to both orders in 247 us, 5.7 TB/s (1.41 GB; reading the block again for the transposed
// order would be 0.94 GB more).

constexpr int kWeightThreads = 256;

template <bool F32>
__device__ __forceinline__ uint32_t codes4(const f32x4& v, const Inverse& inv) {
  float x[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = F32 ? inv.nearest(v[e]) : inv(v[e]);
  const int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], w, true);
}

template <bool F32, bool T>
__global__ void __launch_bounds__(kWeightThreads) quantize_weight_kernel(WeightBlocksArgs a) {
  __shared__ uint32_t wave_max[kWeightThreads / 64];
  __shared__ __attribute__((aligned(16))) uint8_t turned[T ? 128 * 128 : 16];
  const int64_t kb = a.K / 128, nb = a.N / 128;
  const int64_t b = blockIdx.x, x = b % kb, gy = b / kb;     // block column, block row over all groups
  const int j = threadIdx.x / 32, c = threadIdx.x % 32;
  const int64_t first = (gy * 128 + 16 * j) * a.K + x * 128 + 4 * c;
  f32x4 v[16];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if constexpr (F32) {
      v[i] = __builtin_nontemporal_load((const f32x4*)((const float*)a.W + first + i * a.K));
    } else {
      const u32x2 w = __builtin_nontemporal_load((const u32x2*)((const uint16_t*)a.W + first + i * a.K));
      v[i] = f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xFFFF0000u), __uint_as_float(w[1] << 16),
                   __uint_as_float(w[1] & 0xFFFF0000u)};
    }
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = umax(m, mag(v[i][e]));
  m = wave_reduce(m, MaxU{});
  if (threadIdx.x % 64 == 0) wave_max[threadIdx.x / 64] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWeightThreads / 64; ++w) m = umax(m, wave_max[w]);
  const float amax = __uint_as_float(m);
  const Inverse inv(amax);
  uint32_t q[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    q[i] = codes4<F32>(v[i], inv);
    store_out((uint32_t*)(a.WQ + first + i * a.K), q[i]);
  }
  const int64_t g = gy / nb, y = gy % nb;
  if (threadIdx.x == 0) {
    a.w_scale[gy * kb + x] = scale_of(amax);
    if constexpr (T) a.wt_scale[(g * kb + x) * nb + y] = scale_of(amax);
  }
  if constexpr (T) {
    u32x4 t[4];                      // column e of the thread's four: its sixteen rows
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // bytes 0 1 of two rows and of the other two, then 2 3
      const uint32_t a01 = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x05010400);
      const uint32_t b01 = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x05010400);
      const uint32_t a23 = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x07030602);
      const uint32_t b23 = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x07030602);
      t[0][i] = __builtin_amdgcn_perm(b01, a01, 0x05040100);
      t[1][i] = __builtin_amdgcn_perm(b01, a01, 0x07060302);
      t[2][i] = __builtin_amdgcn_perm(b23, a23, 0x05040100);
      t[3][i] = __builtin_amdgcn_perm(b23, a23, 0x07060302);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) *(u32x4*)(turned + (e * 32 + c) * 128 + (j ^ ((c >> 1) & 7)) * 16) = t[e];
    __syncthreads();
    // 128 rows of eight chunks: four per thread
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int r = s * 32 + threadIdx.x / 8, chunk = threadIdx.x % 8;   // LDS row r holds column 4 (r % 32) + s
      const u32x4 w = *(const u32x4*)(turned + r * 128 + (chunk ^ (((r % 32) >> 1) & 7)) * 16);
      const int64_t k = x * 128 + 4 * (r % 32) + s;
      store_out((u32x4*)(a.WQt + (g * a.K + k) * a.N + y * 128 + 16 * chunk), w);
    }
  }
}

}  // namespace

hipError_t launch_quantize_groupwise(const uint16_t* X, uint8_t* XQ, float* x_scale, int64_t rows, int64_t K,
                                     hipStream_t stream) {
  const int64_t parts = rows * K / 16;
  if (parts == 0) return hipSuccess;
  const int64_t blocks = (parts + kRowsThreads - 1) / kRowsThreads;
  const dim3 grid((uint32_t)(blocks < (1 << 20) ? blocks : (1 << 20)));
  if (rows * K * 2 > kStreamBytes)
    hipLaunchKernelGGL((quantize_groupwise_kernel<true>), grid, dim3(kRowsThreads), 0, stream, (const u32x4*)X, (u32x4*)XQ,
                       x_scale, parts);
  else
    hipLaunchKernelGGL((quantize_groupwise_kernel<false>), grid, dim3(kRowsThreads), 0, stream, (const u32x4*)X, (u32x4*)XQ,
                       x_scale, parts);
  return hipGetLastError();
}

hipError_t launch_quantize_weight(const WeightBlocksArgs& a, hipStream_t stream) {
  const int64_t blocks = a.G * (a.N / 128) * (a.K / 128);
  if (blocks == 0) return hipSuccess;
  const dim3 grid((uint32_t)blocks), threads(kWeightThreads);
  if (a.f32) {
    if (a.WQt) hipLaunchKernelGGL((quantize_weight_kernel<true, true>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((quantize_weight_kernel<true, false>), grid, threads, 0, stream, a);
  } else {
    if (a.WQt) hipLaunchKernelGGL((quantize_weight_kernel<false, true>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((quantize_weight_kernel<false, false>), grid, threads, 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace fp8gg
