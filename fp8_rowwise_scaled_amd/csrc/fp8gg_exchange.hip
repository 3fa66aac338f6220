// Rows between token order and expert order (gfx950): dispatch of codes and scales,
// the weighted combine, and its gradients.
//
// All three are driven from the token side: dst_row[t, j] is the place of token t's
// j-th row in the experts' order, the same for every lane of a workgroup.  Lane j of
// each wave loads place (and weight) j, all of them in one load, and the loop over j
// reads them from that lane; loading them one by one in the loop waits for memory k
// times over.  Each token's own row is read (or written) once: every byte moves once,
// and the calls are bound by HBM.
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxPlaces = 64;
constexpr int64_t kMaxGrid = 1 << 20;

// Places and weights of one token, the j-th in lane j (k <= 64).  Read with every lane
// of the wave active.
struct Places {
  int row;
  float weight;
};
__device__ __forceinline__ Places load_places(const int32_t* dst_row, const float* weights, int64_t t, int k) {
  const int lane = threadIdx.x & 63;
  Places p{-1, 1.f};
  if (lane < k) {
    p.row = dst_row[t * k + lane];
    if (weights) p.weight = weights[t * k + lane];
  }
  return p;
}
__device__ __forceinline__ int64_t row_of(const Places& p, int j) { return __builtin_amdgcn_readlane(p.row, j); }
__device__ __forceinline__ float weight_of(const Places& p, int j) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(p.weight), j));
}

// One workgroup copies 4 KiB of one token's codes (16 bytes per thread) to its k places.
__global__ void __launch_bounds__(kThreads) dispatch_kernel(DispatchArgs a, int chunks, int64_t work) {
  const int nvec = a.K / 16;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t t = i / chunks;
    const int c = (int)(i - t * chunks);
    const int v = c * kThreads + threadIdx.x;
    u32x4 x = {0, 0, 0, 0};
    if (v < nvec) x = reinterpret_cast<const u32x4*>(a.XQ)[t * nvec + v];
    const Places p = load_places(a.dst_row, nullptr, t, a.k);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = row_of(p, j);
      if (r < 0 || r >= a.R) continue;
      if (v < nvec) reinterpret_cast<u32x4*>(a.XQs)[r * nvec + v] = x;
      if (c == 0)
        for (int s = threadIdx.x; s < a.scale_cols; s += kThreads)
          a.xs_out[r * a.scale_cols + s] = a.x_scale[t * a.scale_cols + s];
    }
  }
}

// One workgroup sums 2048 columns of one token, eight per thread.
__global__ void __launch_bounds__(kThreads) combine_kernel(ExchangeArgs a, int chunks, int64_t work) {
  const int nvec = a.N / 8;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t t = i / chunks;
    const int v = (int)(i - t * chunks) * kThreads + threadIdx.x;
    const bool inside = v < nvec;
    const Places p = load_places(a.dst_row, a.weights, t, a.k);
    F8 sum = {};
    // up to eight rows in flight
    for (int j0 = 0; j0 < a.k; j0 += 8) {
      u32x4 y[8];
      float w[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        y[u] = u32x4{0, 0, 0, 0};
        w[u] = 0.f;
        if (j0 + u < a.k) {
          const int64_t r = row_of(p, j0 + u);
          if (r >= 0 && r < a.R) {
            w[u] = weight_of(p, j0 + u);
            if (inside) y[u] = reinterpret_cast<const u32x4*>(a.rows_in)[r * nvec + v];
          }
        }
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const F8 f = unpack_bf16(y[u]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum.v[e] = __builtin_fmaf(w[u], f.v[e], sum.v[e]);
      }
    }
    if (!inside) continue;
    if (a.other) {
      const F8 f = unpack_bf16(reinterpret_cast<const u32x4*>(a.other)[t * nvec + v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum.v[e] += f.v[e];
    }
    reinterpret_cast<u32x4*>(a.rows_out)[t * nvec + v] = pack_bf16(sum);
  }
}

// One workgroup per token.  NV > 0: the token's row of dout stays in registers
// (N <= 2048 NV); NV == 0: it is read again for every place.
template <int NV>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(ExchangeArgs a) {
  __shared__ float part[2][kThreads / 64][kMaxPlaces];
  const int nvec = a.N / 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool dots = a.dweights != nullptr;
  int slot = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    u32x4 d[NV > 0 ? NV : 1];
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * kThreads + threadIdx.x;
        d[i] = u32x4{0, 0, 0, 0};
        if (v < nvec) d[i] = reinterpret_cast<const u32x4*>(a.rows_in)[t * nvec + v];
      }
    }
    const Places p = load_places(a.dst_row, a.weights, t, a.k);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = row_of(p, j);
      float dot = 0.f;
      if (r >= 0 && r < a.R) {
        const float w = weight_of(p, j);
        const auto one = [&](const u32x4& raw, int v) {
          const F8 g = unpack_bf16(raw);
          if (dots) {
            const F8 y = unpack_bf16(reinterpret_cast<const u32x4*>(a.other)[r * nvec + v]);
#pragma unroll
            for (int e = 0; e < 8; ++e) dot = __builtin_fmaf(g.v[e], y.v[e], dot);
          }
          F8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o.v[e] = w * g.v[e];
          reinterpret_cast<u32x4*>(a.rows_out)[r * nvec + v] = pack_bf16(o);
        };
        if constexpr (NV > 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * kThreads + threadIdx.x;
            if (v < nvec) one(d[i], v);
          }
        } else {
          for (int v = threadIdx.x; v < nvec; v += kThreads)
            one(reinterpret_cast<const u32x4*>(a.rows_in)[t * nvec + v], v);
        }
      }
      if (dots) {
        dot = wave_reduce(dot, AddF());
        if (lane == 0) part[slot][wave][j] = dot;
      }
    }
    if (dots) {
      __syncthreads();
      if ((int)threadIdx.x < a.k) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 64; ++w) s += part[slot][w][threadIdx.x];
        a.dweights[t * a.k + threadIdx.x] = s;
      }
      slot ^= 1;   // rewritten only after the next token's barrier
    }
  }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.k == 0 || a.R == 0) return hipSuccess;
  const int nvec = a.K / 16;
  const int chunks = nvec > 0 ? (nvec + kThreads - 1) / kThreads : 1;
  const int64_t work = a.T * chunks;
  hipLaunchKernelGGL(dispatch_kernel, dim3((uint32_t)(work < kMaxGrid ? work : kMaxGrid)), dim3(kThreads), 0, stream, a,
                     chunks, work);
  return hipGetLastError();
}

hipError_t launch_combine(const ExchangeArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.N == 0) return hipSuccess;
  const int chunks = (a.N / 8 + kThreads - 1) / kThreads;
  const int64_t work = a.T * chunks;
  hipLaunchKernelGGL(combine_kernel, dim3((uint32_t)(work < kMaxGrid ? work : kMaxGrid)), dim3(kThreads), 0, stream, a,
                     chunks, work);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.k == 0) return hipSuccess;
  const dim3 grid((uint32_t)(a.T < kMaxGrid ? a.T : kMaxGrid)), threads(kThreads);
  const int nvec = a.N / 8;
  if (nvec <= kThreads) hipLaunchKernelGGL((combine_backward_kernel<1>), grid, threads, 0, stream, a);
  else if (nvec <= 2 * kThreads) hipLaunchKernelGGL((combine_backward_kernel<2>), grid, threads, 0, stream, a);
  else if (nvec <= 4 * kThreads) hipLaunchKernelGGL((combine_backward_kernel<4>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((combine_backward_kernel<0>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8gg
