// Rows between token order and expert order (gfx950): dispatch of codes and scales,
// the weighted combine, and its gradients.
//
// All three are driven from the token side: dst_row[t, j] is the place of token t's
// j-th row in the experts' order, the same for every lane of a workgroup.  Lane j of
// each wave loads place (and weight) j, all of them in one load, and the loop over j
// reads them from that lane; loading them one by one in the loop waits for memory k
// times over.  Each token's own row is read (or written) once: every byte moves once,
// and the calls are bound by HBM.  Combine, 4096 tokens x 8 x 7168 and an addend: 93 us,
// 6.3 TB/s; its gradients, 2047 x 8 x 7168: 88 us, 5.7 TB/s; dispatch, 64 x 8 x 7168 codes:
// 4.0 us for 4.1 MB, most of it latency.
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxGrid = 1 << 20;

// Pieces of a row of nvec vectors, one workgroup each, and the threads of a workgroup: as
// many waves as have something to do, since those without take the place of others on the
// CU (us, and with 256 threads whatever the row: combine, 6696 tokens x 8 x 416: 11.6,
// 18.2; 3650 x 1 x 4512: 19.4, 22.6; dispatch, 4096 x 8 x 256 codes: 5.1, 7.4; combine's
// gradients, 6696 x 8 x 416: 17.8, 29.3).
struct Split {
  int chunks, threads;
};
Split split_row(int nvec) {
  const int waves = nvec > 0 ? (nvec + 63) / 64 : 1;
  const int chunks = (waves + kThreads / 64 - 1) / (kThreads / 64);
  return {chunks, (waves + chunks - 1) / chunks * 64};
}

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

// One workgroup copies up to 4 KiB of one token's codes (16 bytes per thread) to its k places.
__global__ void __launch_bounds__(kThreads) dispatch_kernel(DispatchArgs a, Split split, int64_t work) {
  const int nvec = a.K / 16;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t t = i / split.chunks;
    const int c = (int)(i - t * split.chunks);
    const int v = c * split.threads + threadIdx.x;
    u32x4 x = {0, 0, 0, 0};
    if (v < nvec) x = reinterpret_cast<const u32x4*>(a.XQ)[t * nvec + v];
    const Places p = load_places(a.dst_row, nullptr, t, a.k);
    for (int j = 0; j < a.k; ++j) {
      const int64_t r = row_of(p, j);
      if (r < 0 || r >= a.R) continue;
      if (v < nvec) store_out(reinterpret_cast<u32x4*>(a.XQs) + r * nvec + v, x);
    }
    if (c == 0) {
      // in whole waves: the places are read from lanes that may have no scale of their own
      for (int s0 = 0; s0 < a.scale_cols; s0 += split.threads) {
        const int s = s0 + threadIdx.x;
        float scale = 0.f;
        if (s < a.scale_cols) scale = a.x_scale[t * a.scale_cols + s];
        for (int j = 0; j < a.k; ++j) {
          const int64_t r = row_of(p, j);
          if (s < a.scale_cols && r >= 0 && r < a.R) a.xs_out[r * a.scale_cols + s] = scale;
        }
      }
    }
  }
}

// One workgroup sums up to 2048 columns of one token, eight per thread.
template <bool STREAM>
__global__ void __launch_bounds__(kThreads) combine_kernel(ExchangeArgs a, Split split, int64_t work) {
  const int nvec = a.N / 8;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t t = i / split.chunks;
    const int v = (int)(i - t * split.chunks) * split.threads + threadIdx.x;
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
            if (inside) y[u] = load_in<STREAM>(reinterpret_cast<const u32x4*>(a.rows_in) + r * nvec + v);
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
    store_out(reinterpret_cast<u32x4*>(a.rows_out) + t * nvec + v, pack_bf16(sum));
  }
}

// A workgroup takes two places of one token, both of whose rows of Y are asked for before
// one is used or any row stored: a load that follows stores waits for them too.  NV > 0:
// the token's row of dout stays in registers (N <= 2048 NV; NV == 1: as many waves as the
// row needs, else four); NV == 0: it is read again for every place.  The workgroups of one token follow each other on one XCD, whose L2
// holds its dout.  2047 tokens x 8 x 7168: all eight places in one workgroup 110 us, in
// a workgroup of its own each four 98 us, each two 96 us; 90 us with STREAM.
constexpr int kRowsAtOnce = 2;

template <int NV, bool STREAM>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(ExchangeArgs a, int waves, int batches, int64_t work) {
  __shared__ float part[2][kThreads / 64][kRowsAtOnce];
  const int nvec = a.N / 8;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const bool dots = a.dweights != nullptr;
  const u32x4* rows_in = reinterpret_cast<const u32x4*>(a.rows_in);
  const u32x4* other = reinterpret_cast<const u32x4*>(a.other);
  u32x4* rows_out = reinterpret_cast<u32x4*>(a.rows_out);
  const auto product = [](const u32x4& d, const u32x4& y, float sum) {
    const F8 g = unpack_bf16(d), f = unpack_bf16(y);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(g.v[e], f.v[e], sum);
    return sum;
  };
  const auto times = [](const u32x4& d, float w) {
    F8 g = unpack_bf16(d);
#pragma unroll
    for (int e = 0; e < 8; ++e) g.v[e] *= w;
    return pack_bf16(g);
  };
  int slot = 0;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    // eight neighbouring workgroups lie on the eight XCDs
    const int64_t eight = i / (8 * batches);
    const int within = (int)(i - eight * (8 * batches));
    const int64_t t = eight * 8 + (within & 7);
    const int j0 = (within >> 3) * kRowsAtOnce;
    if (t >= a.T) continue;                          // the same for the whole workgroup
    const Places p = load_places(a.dst_row, a.weights, t, a.k);
    int64_t row[kRowsAtOnce];
    float w[kRowsAtOnce], dot[kRowsAtOnce] = {};
#pragma unroll
    for (int u = 0; u < kRowsAtOnce; ++u) {
      row[u] = j0 + u < a.k ? row_of(p, j0 + u) : -1;
      if (row[u] >= a.R) row[u] = -1;
      w[u] = j0 + u < a.k ? weight_of(p, j0 + u) : 0.f;
    }
    if constexpr (NV > 0) {
      u32x4 d[NV], y[kRowsAtOnce][NV];
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int v = c * kThreads + threadIdx.x;
        d[c] = u32x4{0, 0, 0, 0};
        if (v < nvec) d[c] = rows_in[t * nvec + v];
      }
#pragma unroll
      for (int u = 0; u < kRowsAtOnce; ++u)
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int v = c * kThreads + threadIdx.x;
          y[u][c] = u32x4{0, 0, 0, 0};
          if (dots && row[u] >= 0 && v < nvec) y[u][c] = load_in<STREAM>(other + row[u] * nvec + v);
        }
#pragma unroll
      for (int u = 0; u < kRowsAtOnce; ++u)
#pragma unroll
        for (int c = 0; c < NV; ++c) {
          const int v = c * kThreads + threadIdx.x;
          dot[u] = product(d[c], y[u][c], dot[u]);
          if (row[u] >= 0 && v < nvec) store_out(rows_out + row[u] * nvec + v, times(d[c], w[u]));
        }
    } else {
#pragma unroll
      for (int u = 0; u < kRowsAtOnce; ++u) {
        if (row[u] < 0) continue;
        for (int v = threadIdx.x; v < nvec; v += kThreads) {
          const u32x4 d = rows_in[t * nvec + v];
          if (dots) dot[u] = product(d, load_in<STREAM>(other + row[u] * nvec + v), dot[u]);
          store_out(rows_out + row[u] * nvec + v, times(d, w[u]));
        }
      }
    }
    if (dots) {
#pragma unroll
      for (int u = 0; u < kRowsAtOnce; ++u) {
        // a place left out has 0, also where d times the zeros in its y is NaN
        dot[u] = row[u] >= 0 ? wave_reduce(dot[u], AddF()) : 0.f;
        if (lane == 0) part[slot][wave][u] = dot[u];
      }
      __syncthreads();
      if (threadIdx.x < kRowsAtOnce && j0 + (int)threadIdx.x < a.k) {
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < kThreads / 64; ++x) s += NV != 1 || x < waves ? part[slot][x][threadIdx.x] : 0.f;
        a.dweights[t * a.k + j0 + threadIdx.x] = s;
      }
      slot ^= 1;   // rewritten only after the next token's barrier
    }
  }
}

}  // namespace

hipError_t launch_dispatch(const DispatchArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.k == 0 || a.R == 0) return hipSuccess;
  const Split split = split_row(a.K / 16);
  const int64_t work = a.T * split.chunks;
  hipLaunchKernelGGL(dispatch_kernel, dim3((uint32_t)(work < kMaxGrid ? work : kMaxGrid)), dim3(split.threads), 0, stream,
                     a, split, work);
  return hipGetLastError();
}

hipError_t launch_combine(const ExchangeArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.N == 0) return hipSuccess;
  const Split split = split_row(a.N / 8);
  const int64_t work = a.T * split.chunks;
  const dim3 grid((uint32_t)(work < kMaxGrid ? work : kMaxGrid)), threads(split.threads);
  if (a.T * a.k * a.N * 2 > kStreamBytes)
    hipLaunchKernelGGL((combine_kernel<true>), grid, threads, 0, stream, a, split, work);
  else
    hipLaunchKernelGGL((combine_kernel<false>), grid, threads, 0, stream, a, split, work);
  return hipGetLastError();
}

template <int NV>
static hipError_t launch_back(const ExchangeArgs& a, hipStream_t stream) {
  const int batches = (a.k + kRowsAtOnce - 1) / kRowsAtOnce;
  const int waves = NV == 1 ? split_row(a.N / 8).threads / 64 : kThreads / 64;
  const int64_t work = (a.T + 7) / 8 * 8 * batches;
  const dim3 grid((uint32_t)(work < kMaxGrid ? work : kMaxGrid)), threads(64 * waves);
  if (a.T * a.k * a.N * 2 > kStreamBytes)
    hipLaunchKernelGGL((combine_backward_kernel<NV, true>), grid, threads, 0, stream, a, waves, batches, work);
  else
    hipLaunchKernelGGL((combine_backward_kernel<NV, false>), grid, threads, 0, stream, a, waves, batches, work);
  return hipGetLastError();
}

hipError_t launch_combine_backward(const ExchangeArgs& a, hipStream_t stream) {
  if (a.T == 0 || a.k == 0) return hipSuccess;
  const int nvec = a.N / 8;
  if (nvec <= kThreads) return launch_back<1>(a, stream);
  if (nvec <= 2 * kThreads) return launch_back<2>(a, stream);
  if (nvec <= 4 * kThreads) return launch_back<4>(a, stream);
  return launch_back<0>(a, stream);
}

}  // namespace fp8gg
