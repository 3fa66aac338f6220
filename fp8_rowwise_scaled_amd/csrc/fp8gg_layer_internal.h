// Internal interface of the layer operators (include/fp8gg_layer.h): arguments as
// the kernels see them, launchers, and the device helpers they share.
#ifndef FP8GG_LAYER_INTERNAL_H_
#define FP8GG_LAYER_INTERNAL_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8gg {

struct NormArgs {
  const uint16_t* X;
  const uint16_t* residual;     // or null
  const void* weight;           // bf16, or fp32 when w_f32
  uint8_t* XQ;
  float* x_scale;
  uint16_t* Y;                  // or null
  uint16_t* residual_out;       // given exactly when residual is
  float* rstd;                  // or null
  int64_t rows;
  int32_t K;
  int32_t w_f32;
  float eps;
  int32_t stream;               // set by the launcher: load_in<true>
};

struct NormBackwardArgs {
  const uint16_t* dY;
  const uint16_t* H;
  const void* weight;
  const float* rstd;
  const uint16_t* dresidual;    // or null
  uint16_t* dX;
  float* dweight;
  float* partial;               // [parts, K]
  int64_t rows;
  int32_t K;
  int32_t w_f32;
  int32_t parts;
};

struct RouteArgs {
  const void* logits;           // fp32, or bf16 when bf16 is set
  const float* bias;            // or null
  float* weights;
  int32_t* ids;
  int64_t* M_sizes;             // null: no plan
  int32_t* dst_row;
  int32_t* hist;                // [blocks, count_row(E)]; null up to kLonePairs pairs
  int64_t T;
  int32_t E, k;
  int32_t n_group, topk_group, group_top;
  int32_t bf16, sigmoid, renormalize;
  float scale;
  // set by the launcher
  int32_t block_tokens;         // tokens of one workgroup
  int32_t threads;              // blockDim.x, here because the other arguments are loaded anyway
  int32_t token_lds;            // bytes of LDS per token
  bool alone;                   // one workgroup chooses and plans
};

struct RouteBackwardArgs {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t T;
  int32_t E, k;
  int32_t bf16, sigmoid, renormalize;
  float scale;
};

struct ExchangeArgs {
  const uint16_t* rows_in;      // combine: Y; backward: dout
  const int32_t* dst_row;
  const float* weights;         // or null
  const uint16_t* other;        // combine: addend (or null); backward: Y (or null)
  uint16_t* rows_out;           // combine: out; backward: dY
  float* dweights;              // backward, given with Y
  int64_t T, R;
  int32_t k, N;
};

struct DispatchArgs {
  const uint8_t* XQ;
  const float* x_scale;
  const int32_t* dst_row;
  uint8_t* XQs;
  float* xs_out;
  int64_t T, R;
  int32_t k, K, scale_cols;
};

struct SiluArgs {
  const uint16_t* H;
  uint8_t* AQ;
  float* a_scale;
  uint8_t* HQ;                  // or null, with h_scale
  float* h_scale;
  int64_t rows;
  int32_t I;
  int32_t stream;               // set by the launcher: load_in<true>
};

struct SiluBackwardArgs {
  const uint16_t* dA;
  const uint8_t* HQ;
  const float* h_scale;
  uint16_t* dH;
  int64_t rows;
  int32_t I;
};

// At most kChunkRows rows of one group.
struct KChunk {
  int32_t row;       // first row in X
  int32_t col;       // first column in XT
  int32_t group;     // -1: past the last chunk
  int32_t rows;
  int32_t first;     // the group's first chunk
  int32_t chunks;    // the group's chunks
};

struct KOffsetsArgs {
  const void* X;                // bf16, or e4m3fn codes when x_scale is given
  const float* x_scale;
  const int64_t* M_sizes;
  uint8_t* XT;
  float* t_scale;
  int32_t* k_offsets;
  float* partial;               // [chunks, K] largest magnitudes
  KChunk* table;                // [chunks]
  int64_t R, cap;
  int32_t G, K, scale_cols;
};

// Workgroups that the norm's backward pass spreads its rows over (rows of its partial sums
// of dweight), and rows of counts that routing hands on.
int norm_backward_parts(int64_t rows, int64_t K);
int64_t route_count_rows(int64_t T, int64_t E);
// Up to so many (token, expert) pairs one workgroup makes the plan by itself.
constexpr int64_t kLonePairs = 4096;
// Counts of one workgroup, rounded up to whole 128-byte lines: workgroups on different
// XCDs write neighbouring rows.
constexpr int count_row(int64_t E) { return (int)((E + 31) / 32 * 32); }

// Rows of X that one workgroup of quantize_k_offsets takes; a chunk never holds
// rows of two groups.
constexpr int kChunkRows = 128;
inline int64_t k_offsets_chunks(int64_t R, int64_t G) {
  const int64_t ub = (R + kChunkRows - 1) / kChunkRows + G;
  return ub < R ? ub : R;
}
inline int64_t k_offsets_cap(int64_t R, int64_t G) { return (R + 15 * (R < G ? R : G) + 15) / 16 * 16; }

hipError_t launch_rmsnorm_quantize(const NormArgs& a, int block, hipStream_t stream);
hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream);
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);
hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream);
hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream);
hipError_t launch_combine(const ExchangeArgs& a, hipStream_t stream);
hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t stream);
hipError_t launch_silu_mul_quantize(const SiluArgs& a, int block, hipStream_t stream);
hipError_t launch_silu_mul_backward(const SiluBackwardArgs& a, hipStream_t stream);
hipError_t launch_quantize_k_offsets(const KOffsetsArgs& a, hipStream_t stream);

#ifdef __HIPCC__

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Eight fp32 values from eight bf16 ones (16 bytes).
struct F8 {
  float v[8];
};

__device__ __forceinline__ F8 unpack_bf16(const u32x4& w) {
  F8 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    r.v[2 * i] = __uint_as_float(w[i] << 16);
    r.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return r;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  // one v_cvt_pk_bf16_f32 (round to nearest even)
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) |
         ((uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16);
}

__device__ __forceinline__ u32x4 pack_bf16(const F8& f) {
  return u32x4{pack_bf16(f.v[0], f.v[1]), pack_bf16(f.v[2], f.v[3]), pack_bf16(f.v[4], f.v[5]),
               pack_bf16(f.v[6], f.v[7])};
}

// Eight e4m3fn codes of v * inv (hardware convert: round to nearest even; |v * inv|
// is at most 448 up to rounding, far below the 464 from which the format overflows).
__device__ __forceinline__ u32x2 codes_of(const F8& f, float inv) {
  u32x2 q;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(f.v[4 * h] * inv, f.v[4 * h + 1] * inv, 0, false);
    q[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f.v[4 * h + 2] * inv, f.v[4 * h + 3] * inv, w, true);
  }
  return q;
}

// Eight fp32 values from eight e4m3fn codes.
__device__ __forceinline__ F8 values_of(const u32x2& q) {
  F8 r;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
    r.v[4 * h] = a[0];
    r.v[4 * h + 1] = a[1];
    r.v[4 * h + 2] = b[0];
    r.v[4 * h + 3] = b[1];
  }
  return r;
}

// Outputs are stored past the caches: they are written once, whole lines at a time, and
// the next kernel finds them no slower (norm, 4096 x 7168, followed by a kernel that
// reads what it wrote: 69.2 -> 65.9 us; at 256 rows 10.0 -> 9.7).
template <typename T>
__device__ __forceinline__ void store_out(T* p, const T& v) {
  __builtin_nontemporal_store(v, p);
}

// Rows read once: past the caches where a call reads more than kStreamBytes of them, so
// that they do not push each other out (combine, 470 MB: 109 -> 96 us; norm, 470 MB: 187
// -> 182), from the caches below, where a producer may have left them (norm, 59 MB: 20.7
// against 25.2 us; combine, 29 MB: 7.7 against 8.1; level near 100 MB).
constexpr int64_t kStreamBytes = 100 * 1000 * 1000;
template <bool STREAM, typename T>
__device__ __forceinline__ T load_in(const T* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(p);
  else return *p;
}

constexpr float kCodeMax = 448.0f;

// amax with the scale's floor: 448 / floored(amax) and floored(amax) / 448 are normal
// fp32 numbers for every finite amax.
__device__ __forceinline__ float floored(float amax) { return amax > 0x1p-100f ? amax : 0x1p-100f; }
__device__ __forceinline__ float inverse_scale(float amax) { return kCodeMax / floored(amax); }
__device__ __forceinline__ float scale_of(float amax) {
  return amax == 0.f ? 1.f : floored(amax) * (1.0f / kCodeMax);
}

// Magnitudes compare as unsigned integers; so their maxima need no NaN handling.
__device__ __forceinline__ uint32_t mag(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

__device__ __forceinline__ uint32_t mag_max(const F8& f, uint32_t m) {
#pragma unroll
  for (int i = 0; i < 8; ++i) m = umax(m, mag(f.v[i]));
  return m;
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(x)));
}
template <int CTRL>
__device__ __forceinline__ double dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  return __builtin_bit_cast(double, (uint64_t)dpp<CTRL>((uint32_t)u) | ((uint64_t)dpp<CTRL>((uint32_t)(u >> 32)) << 32));
}

// All-reduce over each row of 16 lanes: exchanges inside quads, of the quads of a half
// row, of the half rows (data-parallel-primitive moves, no LDS).  op is commutative, so
// every lane gets the same bits.
template <typename T, typename Op>
__device__ __forceinline__ T row16_reduce(T x, Op op) {
  x = op(x, dpp<0xB1>(x));    // lanes 1 0 3 2
  x = op(x, dpp<0x4E>(x));    // lanes 2 3 0 1
  x = op(x, dpp<0x141>(x));   // mirror in each half row
  return op(x, dpp<0x140>(x)); // mirror in the row
}

// ... and over the wave's 64 lanes: swaps of 16-lane rows, then of 32-lane halves.  A
// swap of x with itself gives, in every lane, the two values that its pair holds.
template <bool HALVES>
__device__ __forceinline__ void swapped(uint32_t x, uint32_t& a, uint32_t& b) {
  if constexpr (HALVES) {
    const auto r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    a = r[0];
    b = r[1];
  }
}
template <bool HALVES, typename T, typename Op>
__device__ __forceinline__ T swap_reduce(T x, Op op) {
  static_assert(sizeof(T) == 4 || sizeof(T) == 8, "32- or 64-bit values");
  if constexpr (sizeof(T) == 4) {
    uint32_t a, b;
    swapped<HALVES>(__builtin_bit_cast(uint32_t, x), a, b);
    return op(__builtin_bit_cast(T, a), __builtin_bit_cast(T, b));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    uint32_t a0, b0, a1, b1;
    swapped<HALVES>((uint32_t)u, a0, b0);
    swapped<HALVES>((uint32_t)(u >> 32), a1, b1);
    return op(__builtin_bit_cast(T, (uint64_t)a0 | ((uint64_t)a1 << 32)),
              __builtin_bit_cast(T, (uint64_t)b0 | ((uint64_t)b1 << 32)));
  }
}
template <typename T, typename Op>
__device__ __forceinline__ T wave_reduce(T x, Op op) {
  return swap_reduce<true>(swap_reduce<false>(row16_reduce(x, op), op), op);
}

// Inclusive scan over the wave: shifts within rows of 16 lanes, then the last lane of a
// row (of the lower half) to the rows after it.  0 is op's neutral element.
template <typename Op>
__device__ __forceinline__ uint32_t wave_scan(uint32_t x, Op op) {
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));   // row_shr 1
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));   // row_shr 2
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));   // row_shr 4
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));   // row_shr 8
  x = op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));   // row_bcast 15
  return op(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));   // row_bcast 31
}

struct AddF {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct MaxU {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return umax(a, b); }
};
struct MinU {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return umin(a, b); }
};

#endif  // __HIPCC__

}  // namespace fp8gg

#endif  // FP8GG_LAYER_INTERNAL_H_
