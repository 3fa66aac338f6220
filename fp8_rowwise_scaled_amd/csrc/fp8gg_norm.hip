// Root-mean-square norm with the residual's addition and an fp8 output, and its
// gradient (gfx950).
//
// Forward.  With h = bf16(x + residual), y = h rstd w and q = y / (amax|y| / 448):
// rstd is common to the row, so
//     amax|y| = rstd amax|h w|   and   q = (h w) (448 / amax|h w|),
// and the sum of squares and the largest |h w| are gathered in the same pass over the
// row: one exchange between the waves per row, and with block scales none at all
// before the codes are stored (a block is the 16 lanes x 8 columns of one load).  The
// row stays in registers between the pass and the codes, so the call moves what it has
// to: 2 bytes per element in (4 with a residual), 1 out (2 more for h, 2 more for Y).
// It is bound by HBM: 16384 x 7168 with residual, block scales and Y moves 1.06 GB in 173
// us, 6.1 TB/s (a copy of 1 GiB reaches 5.2); counters show each byte moved once.  8 x
// 7168: 3.9 us, the latency of a load, two reductions and a launch.
//
// Backward.  Each team of threads walks every n-th row, n being the launch's teams: one pass
// gathers mean(w dY xhat), the row (still in registers up to K = 16384) gives dX, and every
// thread keeps the sum of dY xhat of its own columns in fp32 over all its rows.  A
// workgroup's teams join their sums, which go to the workspace, one row per workgroup, and a
// second kernel adds those in a fixed order.  4093 x 7184 with the
// residual's gradient: 46 us, 5.1 TB/s, and 5 us for the 256 partial sums.  Loads past the
// caches do not help here (55.2 against 54.1 us).
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

__device__ __forceinline__ F8 load_weight(const void* w, int f32, int64_t j) {
  F8 r;
  if (f32) {
    const f32x4 a = reinterpret_cast<const f32x4*>(w)[2 * j];
    const f32x4 b = reinterpret_cast<const f32x4*>(w)[2 * j + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r.v[i] = a[i];
      r.v[4 + i] = b[i];
    }
  } else {
    r = unpack_bf16(reinterpret_cast<const u32x4*>(w)[j]);
  }
  return r;
}

// A team of TPR threads works on one row; teams of one wave share a workgroup.
constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

// Sum and maximum over the team.  `slot` alternates from row to row, so that one
// barrier per row is enough: a slot is rewritten only after the next row's barrier,
// which every thread reaches after it has read this row's values.
template <int TPR>
__device__ __forceinline__ void team_reduce(float& sum, uint32_t& most, int slot) {
  sum = wave_reduce(sum, AddF());
  most = wave_reduce(most, MaxU());
  if constexpr (TPR > 64) {
    __shared__ float sums[2][TPR / 64];
    __shared__ uint32_t mosts[2][TPR / 64];
    if ((threadIdx.x & 63) == 0) {
      sums[slot][threadIdx.x >> 6] = sum;
      mosts[slot][threadIdx.x >> 6] = most;
    }
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) {
      sum += sums[slot][w];
      most = umax(most, mosts[slot][w]);
    }
  }
}

template <bool STREAM, int TPR, int NV>
__device__ __forceinline__ void load_row(const NormArgs& a, int64_t base, int lane, u32x4 (&raw)[NV], u32x4 (&res)[NV]) {
  const int nvec = a.K / 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = i * TPR + lane;
    raw[i] = res[i] = u32x4{0, 0, 0, 0};
    if (j < nvec) {
      raw[i] = load_in<STREAM>(reinterpret_cast<const u32x4*>(a.X) + base + j);
      if (a.residual) res[i] = load_in<STREAM>(reinterpret_cast<const u32x4*>(a.residual) + base + j);
    }
  }
}

// Below this mean of squares (plus eps) the squares have left what fp32 holds in full: above
// it those that underflow, by at most 2^-150 each, change the mean by less than 2^-50 of it.
constexpr float kSmallMean = 0x1p-100f;

// The mean of such a row's (h 2^96)^2, plus eps 2^192: the largest |h| is below 2^-42 (K <=
// 2^15), so no square overflows, and the smallest bf16 value, 2^-133, has a square of 2^-74.
// Such rows are rare: every wave reads all of h again, after the barrier of the team that
// wrote it, and there is no second one.  The check costs the other rows about 1% (8 x 7168:
// 3.60 -> 3.66 us; 1500 x 16384: 33.0 -> 33.3).
__device__ __forceinline__ float mean_of_small(const NormArgs& a, int64_t base, int lane, float inv_k) {
  const u32x4* rows = reinterpret_cast<const u32x4*>(a.residual ? a.residual_out : a.X) + base;
  float sum = 0.f;
#pragma unroll 1
  for (int j = lane & 63; j < a.K / 8; j += 64) {
    const F8 h = unpack_bf16(rows[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = __builtin_fmaf(h.v[e] * 0x1p96f, h.v[e] * 0x1p96f, sum);
  }
  return __builtin_fmaf(wave_reduce(sum, AddF()), inv_k, a.eps * 0x1p96f * 0x1p96f);
}

template <int TPR, int NV, bool BLOCKED>
__global__ void __launch_bounds__(threads_of(TPR)) rmsnorm_quantize_kernel(NormArgs a) {
  constexpr int kTeams = threads_of(TPR) / TPR;
  const int team = threadIdx.x / TPR;
  const int nvec = a.K / 8;
  const float inv_k = 1.0f / (float)a.K;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kTeams + team; row < a.rows; row += (int64_t)gridDim.x * kTeams) {
    int lane = threadIdx.x % TPR;
    // 1024 threads: opaque to the compiler in each row, or it keeps all addresses in registers
    // across the rows, 78 with two vectors, and only one workgroup fits a CU (34.9 against
    // 33.2 us at 1500 x 16384).  Not the smaller ones: their weights are then asked for
    // later (8 x 7168: 3.76 against 3.66 us).
    if constexpr (TPR == 1024) asm volatile("" : "+v"(lane));
    const int64_t base = row * nvec;
    u32x4 raw[NV], res[NV];
    if (a.stream) load_row<true, TPR>(a, base, lane, raw, res);
    else load_row<false, TPR>(a, base, lane, raw, res);
    F8 hw[NV];
    float sum = 0.f;
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * TPR + lane;
      F8 h = unpack_bf16(raw[i]);
      if (a.residual) {
        const F8 r = unpack_bf16(res[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) h.v[e] += r.v[e];
        const u32x4 rounded = pack_bf16(h);
        if (j < nvec) store_out(reinterpret_cast<u32x4*>(a.residual_out) + base + j, rounded);
        h = unpack_bf16(rounded);
      }
      F8 w{};
      if (j < nvec) w = load_weight(a.weight, a.w_f32, j);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = __builtin_fmaf(h.v[e], h.v[e], sum);
        hw[i].v[e] = h.v[e] * w.v[e];
      }
      if constexpr (!BLOCKED) most = mag_max(hw[i], most);
    }
    float block_amax[NV];
    if constexpr (BLOCKED) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * TPR + lane;
        block_amax[i] = __uint_as_float(row16_reduce(mag_max(hw[i], 0), MaxU()));
        if (j < nvec) store_out(reinterpret_cast<u32x2*>(a.XQ) + base + j, codes_of(hw[i], inverse_scale(block_amax[i])));
      }
    }
    team_reduce<TPR>(sum, most, slot);
    slot ^= 1;
    float mean = __builtin_fmaf(sum, inv_k, a.eps), up = 1.0f;
    if (mean < kSmallMean) {                         // the same for the whole team
      mean = mean_of_small(a, base, lane, inv_k);
      up = 0x1p96f;
    }
    // a row of zeros without eps: 0, so that neither its output nor its gradient is NaN
    const float rstd = mean == 0.f ? 0.f : up / sqrtf(mean);
    if constexpr (BLOCKED) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * TPR + lane;
        if (j < nvec && (lane & 15) == 0)
          a.x_scale[row * (nvec / 16) + j / 16] = block_amax[i] == 0.f ? 1.f : rstd * scale_of(block_amax[i]);
      }
    } else {
      const float amax = __uint_as_float(most);
      const float inv = inverse_scale(amax);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * TPR + lane;
        if (j < nvec) store_out(reinterpret_cast<u32x2*>(a.XQ) + base + j, codes_of(hw[i], inv));
      }
      if (lane == 0) a.x_scale[row] = amax == 0.f ? 1.f : rstd * scale_of(amax);
    }
    if (a.Y) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * TPR + lane;
        F8 y;
#pragma unroll
        for (int e = 0; e < 8; ++e) y.v[e] = hw[i].v[e] * rstd;
        if (j < nvec) store_out(reinterpret_cast<u32x4*>(a.Y) + base + j, pack_bf16(y));
      }
    }
    if (a.rstd && lane == 0) a.rstd[row] = rstd;
  }
}

// Eight columns of one row as they are loaded.
struct BackVec {
  u32x4 dy, h, dres;
};

__device__ __forceinline__ BackVec load_back(const NormBackwardArgs& a, int64_t row, int j) {
  const int nvec = a.K / 8;
  BackVec v{{0, 0, 0, 0}, {0, 0, 0, 0}, {0, 0, 0, 0}};
  if (j < nvec) {
    v.dy = reinterpret_cast<const u32x4*>(a.dY)[row * nvec + j];
    v.h = reinterpret_cast<const u32x4*>(a.H)[row * nvec + j];
    if (a.dresidual) v.dres = reinterpret_cast<const u32x4*>(a.dresidual)[row * nvec + j];
  }
  return v;
}

// What a thread keeps depends on the registers that its columns leave.  One vector (or two
// in small workgroups): the weights, and the next row, which is asked for before this one
// is reduced (1024 threads and 256 teams so, against 256 threads, four vectors and 512
// teams without: 54.4 -> 51.8 us at 4093 x 7184).  Two vectors of 1024 threads: the row.
// Four: nothing, the second pass over the row reads it again: 65 us at 1228 x 20480, 3.1 TB/s
// of what the call cannot do without (with the row kept, in scratch memory, 130).  Its sums of
// dweight alone take 32 of the 128 registers; 48 bytes per thread still go through scratch.
template <int TPR, int NV>
__global__ void __launch_bounds__(threads_of(TPR)) rmsnorm_backward_kernel(NormBackwardArgs a) {
  constexpr int kTeams = threads_of(TPR) / TPR;
  constexpr bool kAhead = NV == 1 || TPR == 64;
  constexpr bool kKept = NV <= 2;
  const int lane = threadIdx.x % TPR;
  const int team = blockIdx.x * kTeams + threadIdx.x / TPR, teams = a.parts * kTeams;
  const int nvec = a.K / 8;
  const float inv_k = 1.0f / (float)a.K;
  F8 held[kAhead ? NV : 1], dw[NV] = {};
  BackVec now[kKept ? NV : 1], next[kAhead ? NV : 1];
  const auto weight = [&](int i) {
    F8 w = {};
    if constexpr (kAhead) w = held[i];
    else if (i * TPR + lane < nvec) w = load_weight(a.weight, a.w_f32, i * TPR + lane);
    return w;
  };
  const auto vec = [&](int64_t row, int i) {
    if constexpr (kKept) return now[i];
    else return load_back(a, row, i * TPR + lane);
  };
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      held[i] = F8{};
      if (i * TPR + lane < nvec) held[i] = load_weight(a.weight, a.w_f32, i * TPR + lane);
      if (team < a.rows) now[i] = load_back(a, team, i * TPR + lane);
    }
  }
  int slot = 0;
  for (int64_t row = team; row < a.rows; row += teams) {
    const float rstd = a.rstd[row];
    if constexpr (kKept) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (!kAhead) now[i] = load_back(a, row, i * TPR + lane);
        else if (row + teams < a.rows) next[i] = load_back(a, row + teams, i * TPR + lane);
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const BackVec v = vec(row, i);
      const F8 w = weight(i), dy = unpack_bf16(v.dy), h = unpack_bf16(v.h);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = dy.v[e] * (h.v[e] * rstd);
        dot = __builtin_fmaf(w.v[e], g, dot);
        dw[i].v[e] += g;
      }
    }
    uint32_t unused = 0;
    team_reduce<TPR>(dot, unused, slot);
    slot ^= 1;
    const float c = dot * inv_k * rstd;   // times h: xhat * mean(w dY xhat)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * TPR + lane;
      const BackVec v = vec(row, i);
      const F8 w = weight(i), dy = unpack_bf16(v.dy), h = unpack_bf16(v.h), dr = unpack_bf16(v.dres);
      F8 dx;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        dx.v[e] = __builtin_fmaf(__builtin_fmaf(-h.v[e], c, w.v[e] * dy.v[e]), rstd, dr.v[e]);
      if (j < nvec) store_out(reinterpret_cast<u32x4*>(a.dX) + row * nvec + j, pack_bf16(dx));
    }
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < NV; ++i) now[i] = next[i];
    }
  }
  // The workgroup's sums, those of several teams joined first.
  __shared__ f32x4 joined[kTeams > 1 ? kTeams * TPR * NV * 2 : 1];
  f32x4* partial = reinterpret_cast<f32x4*>(a.partial + (int64_t)blockIdx.x * a.K);
  f32x4* own = kTeams > 1 ? joined + threadIdx.x / TPR * (TPR * NV * 2) : partial;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = i * TPR + lane;
    if (j < nvec) {
      own[2 * j] = f32x4{dw[i].v[0], dw[i].v[1], dw[i].v[2], dw[i].v[3]};
      own[2 * j + 1] = f32x4{dw[i].v[4], dw[i].v[5], dw[i].v[6], dw[i].v[7]};
    }
  }
  if constexpr (kTeams > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * nvec; c += threads_of(TPR)) {
      f32x4 sum = joined[c];
#pragma unroll
      for (int x = 1; x < kTeams; ++x) sum += joined[x * (TPR * NV * 2) + c];
      partial[c] = sum;
    }
  }
}

// dweight[k] = sum over the parts, in a fixed order: 8 lanes cover 32 columns, the
// workgroup's 32 rows of lanes take every 32nd part (eight loads in flight), then join
// through LDS.
constexpr int kSumCols = 32;
__global__ void __launch_bounds__(256) sum_parts_kernel(const float* __restrict__ partial, float* __restrict__ dweight,
                                                        int K, int parts) {
  __shared__ f32x4 joined[32][kSumCols / 4];
  const int lane = threadIdx.x % (kSumCols / 4), r = threadIdx.x / (kSumCols / 4);
  const int col = blockIdx.x * (kSumCols / 4) + lane;
  f32x4 s = {0.f, 0.f, 0.f, 0.f};
  if (col < K / 4) {
#pragma unroll 8
    for (int p = r; p < parts; p += 32) s += reinterpret_cast<const f32x4*>(partial + (int64_t)p * K)[col];
  }
  joined[r][lane] = s;
  __syncthreads();
  if (r == 0 && col < K / 4) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += joined[i][lane];
    reinterpret_cast<f32x4*>(dweight)[col] = s;
  }
}

template <int TPR, int NV>
hipError_t launch_norm(const NormArgs& a, int block, hipStream_t stream) {
  constexpr int kTeams = threads_of(TPR) / TPR;
  const int64_t want = (a.rows + kTeams - 1) / kTeams;
  const dim3 grid((uint32_t)(want < 65536 ? want : 65536)), threads(threads_of(TPR));
  if (block)
    hipLaunchKernelGGL((rmsnorm_quantize_kernel<TPR, NV, true>), grid, threads, 0, stream, a);
  else
    hipLaunchKernelGGL((rmsnorm_quantize_kernel<TPR, NV, false>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

template <int TPR, int NV>
hipError_t launch_back(const NormBackwardArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((rmsnorm_backward_kernel<TPR, NV>), dim3(a.parts), dim3(threads_of(TPR)), 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rmsnorm_quantize(const NormArgs& given, int block, hipStream_t stream) {
  NormArgs a = given;
  if (a.rows == 0) return hipSuccess;
  a.stream = a.rows * a.K * (a.residual ? 4 : 2) > kStreamBytes;
  // Threads and vectors per row, by K alone (a row's sums then come out the same in every
  // batch).  Measured with 24 M elements, us: K = 512: a wave per row 32.5, 256 threads
  // 61.5.  2048: 256 threads 31.2, a wave with four vectors 31.7 (16 rows: 3.0 and 4.0).
  // 4096: 512 threads 30.1, 256 with two vectors 31.2.  7168, row scales: 512 with two
  // 30.8, 256 with four 32.9, 1024 with one 32.2; block scales, which need no barrier
  // before their codes: 35.3, 34.3, 33.8, and at 16384 rows 183, 178, 187.  16384: 1024
  // with two 32.4, 512 with four 33.2, 1024 with four 41.3.
  const int nvec = a.K / 8;
  if (nvec <= 64) return launch_norm<64, 1>(a, block, stream);
  if (nvec <= 128) return launch_norm<64, 2>(a, block, stream);
  if (nvec <= 256) return launch_norm<256, 1>(a, block, stream);
  if (nvec <= 512) return launch_norm<512, 1>(a, block, stream);
  if (nvec <= 1024) return block ? launch_norm<256, 4>(a, block, stream) : launch_norm<512, 2>(a, block, stream);
  if (nvec <= 2048) return launch_norm<1024, 2>(a, block, stream);
  return launch_norm<1024, 4>(a, block, stream);
}

// One workgroup per compute unit of 1024 threads, two of 256 or 512; 2048 teams of one
// wave (K = 512, 24 M elements: 37.5 us, 1024 teams 49.8, 4096 40.6, 512 of 256 threads
// 101).  More teams read and write more partial sums (K = 2048: 512 teams 38.6, 1024
// 40.3, 256 59.8); the four one-wave teams of a workgroup join theirs
// first (2000 x 512: 12.5 -> 8.7; 16000 x 1024: 25.6 -> 21.0).
int norm_backward_parts(int64_t rows, int64_t K) {
  const int64_t nvec = K / 8, most = nvec <= 512 ? 512 : 256, teams = nvec <= 128 ? 4 : 1;
  const int64_t filled = (rows + teams - 1) / teams;
  return (int)(filled < most ? filled : most);
}

hipError_t launch_rmsnorm_backward(const NormBackwardArgs& a, hipStream_t stream) {
  const int nvec = a.K / 8;
  hipError_t e = hipSuccess;
  if (a.rows > 0) {
    // as for the forward pass; 4096: 512 threads 39.8 us, 256 with two vectors 43.1; 7168:
    // 1024 with one 39.9, 512 with two 44.2; 12288: 1024 with two 45.8, 512 with four 48.7
    if (nvec <= 64) e = launch_back<64, 1>(a, stream);
    else if (nvec <= 128) e = launch_back<64, 2>(a, stream);
    else if (nvec <= 256) e = launch_back<256, 1>(a, stream);
    else if (nvec <= 512) e = launch_back<512, 1>(a, stream);
    else if (nvec <= 1024) e = launch_back<1024, 1>(a, stream);
    else if (nvec <= 2048) e = launch_back<1024, 2>(a, stream);
    else e = launch_back<1024, 4>(a, stream);
  }
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(sum_parts_kernel, dim3((a.K + kSumCols - 1) / kSumCols), dim3(256), 0, stream, a.partial,
                     a.dweight, a.K, a.parts);
  return hipGetLastError();
}

}  // namespace fp8gg
