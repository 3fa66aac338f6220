// 8-bit activation checkpoints (gfx950): the gated activation with its fp8 output and
// the checkpoint of its input, its gradient from the checkpoint, and the weight
// gradient's operand (rows requantised per group and column, transposed).
//
// The checkpoint keeps the input of the gated activation as e4m3 codes with one scale
// per row, half and 128 columns: 1.03 bytes per value where bf16 takes 2.  The forward
// pass reads H once: a wave's 16 lanes x 8 columns are one scale block, so the block's
// largest magnitude is a reduction over 16 lanes; the activation itself stays in
// registers until the row's largest magnitude is known.  The backward pass is
// elementwise.  Both are bound by HBM: 16384 x 2048 with the checkpoint 38.5 us, 6.2 TB/s;
// backward, 5001 x 1000 7.8 us, 5.2 TB/s.
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

constexpr int threads_of(int tpr) { return tpr < 256 ? 256 : tpr; }

// 1 / (1 + exp(-g)) from the hardware's exp2 and reciprocal (a few units in the last
// place plus |g| 2^-23; what it feeds is rounded to 8 or 16 bits).
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

template <bool STREAM, int TPR, int NV>
__device__ __forceinline__ void load_halves(const SiluArgs& a, int64_t row, int lane, u32x4 (&rg)[NV], u32x4 (&ru)[NV]) {
  const int nvec = a.I / 8;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = i * TPR + lane;
    rg[i] = ru[i] = u32x4{0, 0, 0, 0};
    if (j < nvec) {
      rg[i] = load_in<STREAM>(reinterpret_cast<const u32x4*>(a.H) + 2 * row * nvec + j);
      ru[i] = load_in<STREAM>(reinterpret_cast<const u32x4*>(a.H) + (2 * row + 1) * nvec + j);
    }
  }
}

// A team of TPR threads works on one row, NV x 8 columns of each half per thread.
template <int TPR, int NV, bool BLOCKED>
__global__ void __launch_bounds__(threads_of(TPR)) silu_mul_quantize_kernel(SiluArgs a) {
  constexpr int kTeams = threads_of(TPR) / TPR;
  __shared__ uint32_t mosts[2][threads_of(TPR) / 64];
  const int lane = threadIdx.x % TPR;
  const int nvec = a.I / 8, nblocks = (a.I + 127) / 128;
  int slot = 0;
  for (int64_t row = (int64_t)blockIdx.x * kTeams + threadIdx.x / TPR; row < a.rows;
       row += (int64_t)gridDim.x * kTeams) {
    u32x4 rg[NV], ru[NV];
    if (a.stream) load_halves<true, TPR>(a, row, lane, rg, ru);
    else load_halves<false, TPR>(a, row, lane, rg, ru);
    F8 act[NV];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = i * TPR + lane;
      const F8 g = unpack_bf16(rg[i]), u = unpack_bf16(ru[i]);
      if (a.HQ) {
        const float ag = __uint_as_float(row16_reduce(mag_max(g, 0), MaxU()));
        const float au = __uint_as_float(row16_reduce(mag_max(u, 0), MaxU()));
        if (j < nvec) {
          store_out(reinterpret_cast<u32x2*>(a.HQ) + 2 * row * nvec + j, codes_of(g, inverse_scale(ag)));
          store_out(reinterpret_cast<u32x2*>(a.HQ) + (2 * row + 1) * nvec + j, codes_of(u, inverse_scale(au)));
          if ((lane & 15) == 0) {
            a.h_scale[2 * row * nblocks + j / 16] = scale_of(ag);
            a.h_scale[(2 * row + 1) * nblocks + j / 16] = scale_of(au);
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) act[i].v[e] = g.v[e] * sigmoid(g.v[e]) * u.v[e];
      if constexpr (BLOCKED) {
        const float amax = __uint_as_float(row16_reduce(mag_max(act[i], 0), MaxU()));
        if (j < nvec) {
          store_out(reinterpret_cast<u32x2*>(a.AQ) + row * nvec + j, codes_of(act[i], inverse_scale(amax)));
          if ((lane & 15) == 0) a.a_scale[row * nblocks + j / 16] = scale_of(amax);
        }
      } else {
        most = mag_max(act[i], most);
      }
    }
    if constexpr (!BLOCKED) {
      most = wave_reduce(most, MaxU());
      if constexpr (TPR > 64) {
        if ((threadIdx.x & 63) == 0) mosts[slot][threadIdx.x >> 6] = most;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 64; ++w) most = umax(most, mosts[slot][w]);
        slot ^= 1;   // rewritten only after the next row's barrier
      }
      const float amax = __uint_as_float(most), inv = inverse_scale(amax);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = i * TPR + lane;
        if (j < nvec) store_out(reinterpret_cast<u32x2*>(a.AQ) + row * nvec + j, codes_of(act[i], inv));
      }
      if (lane == 0) a.a_scale[row] = scale_of(amax);
    }
  }
}

// TX threads along the row (eight columns each), 256 / TX rows per workgroup.
template <int TX>
__global__ void __launch_bounds__(256) silu_mul_backward_kernel(SiluBackwardArgs a, int chunks, int64_t work) {
  constexpr int kRows = 256 / TX;
  const int nvec = a.I / 8, nblocks = (a.I + 127) / 128;
  for (int64_t i = blockIdx.x; i < work; i += gridDim.x) {
    const int64_t rows = i / chunks;
    const int64_t row = rows * kRows + threadIdx.x / TX;
    const int j = (int)(i - rows * chunks) * TX + threadIdx.x % TX;
    if (row >= a.rows || j >= nvec) continue;
    const F8 da = unpack_bf16(reinterpret_cast<const u32x4*>(a.dA)[row * nvec + j]);
    const F8 qg = values_of(reinterpret_cast<const u32x2*>(a.HQ)[2 * row * nvec + j]);
    const F8 qu = values_of(reinterpret_cast<const u32x2*>(a.HQ)[(2 * row + 1) * nvec + j]);
    const float sg = a.h_scale[2 * row * nblocks + j / 16];
    const float su = a.h_scale[(2 * row + 1) * nblocks + j / 16];
    F8 dg, du;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float g = qg.v[e] * sg, s = sigmoid(g), silu = g * s;
      du.v[e] = da.v[e] * silu;
      // sig (1 + g (1 - sig)) = sig + silu (1 - sig)
      dg.v[e] = da.v[e] * (qu.v[e] * su) * __builtin_fmaf(silu, 1.0f - s, s);
    }
    store_out(reinterpret_cast<u32x4*>(a.dH) + 2 * row * nvec + j, pack_bf16(dg));
    store_out(reinterpret_cast<u32x4*>(a.dH) + (2 * row + 1) * nvec + j, pack_bf16(du));
  }
}

// ---------------------------------------------------------------------------
// The weight gradient's operand
// ---------------------------------------------------------------------------
//
// Rows are cut into chunks of at most 128 rows of one group.  The first kernel writes
// each chunk's largest magnitude per column, and where the chunk lies; the second one
// joins the chunks of the group, requantises its own 128 rows x 128 columns and turns
// them through LDS, so that both sides are accessed in runs of at least 128 bytes.  The
// rows are read twice; the second time the Infinity Cache holds them unless they pass
// 256 MB.  4096 x 7168 codes in 8 groups: 9.5 + 11.8 us, 20 in a loop.  One kernel whose
// workgroups take a whole group's 128 columns, the rows kept in registers between the two
// steps, reads them once but waits for its largest group: 25 us there, 91 against 27 in 64
// groups, 46 against 21 in one.

constexpr int kTile = 128;             // columns of the second kernel's tile
constexpr int kLdsStride = 33;         // words per column: 128 codes and one of padding

// 64 groups, one per lane: counts clamped as in the stacked layout (negative ones to 0,
// ends to R), and where each group's rows, columns and chunks end.  R, and with it every
// number here, is below 2^31.
struct GroupSpan {
  uint32_t begin, end;                 // rows
  uint32_t cols, cols_end;             // columns, a multiple of 16, and their end
  uint32_t chunks, chunks_end;
};

// Sums that stop at R: ends cut at R add up in any order.
struct AddUpTo {
  uint32_t most;
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return umin(a + b, most); }
};

// Calls visit(first group, the lane's span) for every 64 groups until it returns true;
// all lanes of the wave take part.  Returns the end of the last group's columns.
template <typename Visit>
__device__ __forceinline__ uint32_t scan_groups(const KOffsetsArgs& a, Visit visit) {
  const int lane = threadIdx.x & 63;
  const AddUpTo add{(uint32_t)a.R};
  uint32_t rows_before = 0, cols_before = 0, chunks_before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    int64_t m = g0 + lane < a.G ? a.M_sizes[g0 + lane] : 0;
    m = m < 0 ? 0 : (m > a.R ? a.R : m);
    const uint32_t sum = wave_scan((uint32_t)m, add);
    GroupSpan s;
    s.end = add(rows_before, sum);
    // the group before this one ends where this one begins (lane 0: the last one of the 64 before)
    const uint32_t prior = (uint32_t)__shfl_up((int)s.end, 1, 64);
    s.begin = lane == 0 ? rows_before : prior;
    const uint32_t size = s.end - s.begin;
    s.chunks = (size + kChunkRows - 1) / kChunkRows;
    s.cols = (size + 15) / 16 * 16;
    s.chunks_end = chunks_before + wave_scan(s.chunks, AddF());
    s.cols_end = cols_before + wave_scan(s.cols, AddF());
    if (visit(g0, s)) break;
    rows_before = (uint32_t)__builtin_amdgcn_readlane((int)s.end, 63);
    chunks_before = (uint32_t)__builtin_amdgcn_readlane((int)s.chunks_end, 63);
    cols_before = (uint32_t)__builtin_amdgcn_readlane((int)s.cols_end, 63);
  }
  return cols_before;
}

__device__ __forceinline__ int from_lane(uint32_t x, int lane) { return __builtin_amdgcn_readlane((int)x, lane); }

__device__ __forceinline__ KChunk find_chunk(const KOffsetsArgs& a, uint32_t c) {
  KChunk f{0, 0, -1, 0, 0, 0};
  scan_groups(a, [&](int g0, const GroupSpan& s) {
    const uint64_t hit = __ballot(c >= s.chunks_end - s.chunks && c < s.chunks_end);
    if (!hit) return false;
    const int src = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
    f.group = g0 + src;
    f.chunks = from_lane(s.chunks, src);
    f.first = from_lane(s.chunks_end, src) - f.chunks;
    const int at = ((int)c - f.first) * kChunkRows;
    f.row = from_lane(s.begin, src) + at;
    const int left = from_lane(s.end, src) - f.row;
    f.rows = left < kChunkRows ? left : kChunkRows;
    f.col = from_lane(s.cols_end, src) - from_lane(s.cols, src) + at;
    return true;
  });
  return f;
}

// One load of a row: 16 codes and their row's scale (E4M3), or 8 bf16 values.
template <bool E4M3>
struct Raw {
  u32x4 q;
  float scale;
};

template <bool E4M3>
__device__ __forceinline__ Raw<E4M3> load_raw(const KOffsetsArgs& a, int64_t row, int col) {
  Raw<E4M3> r;
  if constexpr (E4M3) {
    r.q = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(a.X) + row * a.K + col);
    r.scale = a.x_scale[row * a.scale_cols + (a.scale_cols > 1 ? col / 128 : 0)];
  } else {
    r.q = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.X) + row * a.K + col);
    r.scale = 1.f;
  }
  return r;
}

template <bool E4M3>
__device__ __forceinline__ void values(const Raw<E4M3>& r, float (&v)[E4M3 ? 16 : 8]) {
  if constexpr (E4M3) {
    const F8 lo = values_of(u32x2{r.q[0], r.q[1]}), hi = values_of(u32x2{r.q[2], r.q[3]});
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] = lo.v[e] * r.scale;
      v[8 + e] = hi.v[e] * r.scale;
    }
  } else {
    const F8 f = unpack_bf16(r.q);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = f.v[e];
  }
}

// partial[c][k]: largest magnitude of column k in chunk c.  The workgroups have the
// tiles of the second kernel, in the same order: what one reads here its XCD's L2 may
// still hold there (tiles of 512 columns: 9.0 + 13.5 us for the two kernels at 4096 x
// 7168 codes, of 128: 9.5 + 11.7).
template <bool E4M3>
__global__ void __launch_bounds__(256) column_amax_kernel(KOffsetsArgs a, int tiles) {
  constexpr int W = E4M3 ? 16 : 8;
  constexpr int kLanes = kTile / W, kRowLanes = 256 / kLanes, kRows = kChunkRows / kRowLanes;
  __shared__ uint32_t most[kRowLanes][kTile + 4];
  const int chunk = blockIdx.x / tiles, col0 = (int)(blockIdx.x % tiles) * kTile;
  const KChunk f = find_chunk(a, chunk);
  if (col0 == 0 && threadIdx.x == 0) a.table[chunk] = f;
  if (f.group < 0) return;
  const int lx = threadIdx.x % kLanes, ly = threadIdx.x / kLanes;
  const int col = col0 + lx * W;
  Raw<E4M3> raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    raw[i] = Raw<E4M3>{{0, 0, 0, 0}, 0.f};
    if (ly + i * kRowLanes < f.rows && col < a.K) raw[i] = load_raw<E4M3>(a, f.row + ly + i * kRowLanes, col);
  }
  uint32_t m[W] = {};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float v[W];
    values<E4M3>(raw[i], v);
#pragma unroll
    for (int e = 0; e < W; ++e) m[e] = umax(m[e], mag(v[e]));
  }
#pragma unroll
  for (int e = 0; e < W; ++e) most[ly][lx * W + e] = m[e];
  __syncthreads();
  if (threadIdx.x < kTile && col0 + (int)threadIdx.x < a.K) {
    uint32_t top = most[0][threadIdx.x];
#pragma unroll
    for (int y = 1; y < kRowLanes; ++y) top = umax(top, most[y][threadIdx.x]);
    a.partial[(int64_t)chunk * a.K + col0 + threadIdx.x] = __uint_as_float(top);
  }
}

// After the chunks comes one more row of workgroups, which writes k_offsets, the scales
// of empty groups and the columns past the last group.
template <bool E4M3>
__global__ void __launch_bounds__(256) transpose_quantize_kernel(KOffsetsArgs a, int tiles, int chunks) {
  constexpr int W = E4M3 ? 16 : 8;
  constexpr int kLanes = kTile / W, kRowLanes = 256 / kLanes;
  __shared__ uint32_t turned[kTile * kLdsStride];
  __shared__ float inverse[kTile];
  const int chunk = blockIdx.x / tiles, col0 = (int)(blockIdx.x % tiles) * kTile;
  if (chunk == chunks) {
    const int64_t used = scan_groups(a, [&](int g0, const GroupSpan& s) {
      if (threadIdx.x >= 64) return false;
      const int lane = threadIdx.x;
      if (col0 == 0 && g0 + lane < a.G) a.k_offsets[g0 + lane] = (int32_t)s.cols_end;
      for (uint64_t empty = __ballot(g0 + lane < a.G && s.chunks == 0); empty; empty &= empty - 1) {
        float* scales = a.t_scale + (int64_t)(g0 + __ffsll((unsigned long long)empty) - 1) * a.K;
        for (int k = col0 + lane; k < col0 + kTile && k < a.K; k += 64) scales[k] = 1.f;
      }
      return false;
    });
    const int64_t tail = (a.cap - used) / 16;
    for (int64_t i = threadIdx.x; i < tail * kTile; i += 256) {
      const int k = col0 + (int)(i / tail);
      if (k < a.K) *reinterpret_cast<u32x4*>(a.XT + k * a.cap + used + (i % tail) * 16) = u32x4{0, 0, 0, 0};
    }
    return;
  }
  const KChunk f = a.table[chunk];
  if (f.group < 0) return;
  const int lx = threadIdx.x % kLanes, ly = threadIdx.x / kLanes;
  const int col = col0 + lx * W;
  // four neighbouring rows per thread: their codes of one column are one LDS word.  The
  // rows are asked for before the scales are put together.
  constexpr int kPasses = kChunkRows / (kRowLanes * 4);
  Raw<E4M3> raw[kPasses][4];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = (p * kRowLanes + ly) * 4 + i;
      raw[p][i] = Raw<E4M3>{{0, 0, 0, 0}, 0.f};
      if (r < f.rows && col < a.K) raw[p][i] = load_raw<E4M3>(a, f.row + r, col);
    }
  if (threadIdx.x < kTile) {
    const int k = col0 + threadIdx.x;
    uint32_t m = 0;
    if (k < a.K) {
#pragma unroll 4
      for (int c = f.first; c < f.first + f.chunks; ++c) m = umax(m, __float_as_uint(a.partial[(int64_t)c * a.K + k]));
    }
    const float amax = __uint_as_float(m);
    inverse[threadIdx.x] = inverse_scale(amax);
    if (k < a.K && chunk == f.first) a.t_scale[(int64_t)f.group * a.K + k] = scale_of(amax);
  }
  __syncthreads();
  float inv[W];
#pragma unroll
  for (int e = 0; e < W; ++e) inv[e] = inverse[lx * W + e];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    float v[4][W];
#pragma unroll
    for (int i = 0; i < 4; ++i) values<E4M3>(raw[p][i], v[i]);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      int q = __builtin_amdgcn_cvt_pk_fp8_f32(v[0][e] * inv[e], v[1][e] * inv[e], 0, false);
      q = __builtin_amdgcn_cvt_pk_fp8_f32(v[2][e] * inv[e], v[3][e] * inv[e], q, true);
      turned[(lx * W + e) * kLdsStride + p * kRowLanes + ly] = (uint32_t)q;
    }
  }
  __syncthreads();
  const int runs = (f.rows + 15) / 16;
  for (int i = threadIdx.x; i < kTile * 8; i += 256) {
    const int k = i / 8, s = i % 8;
    if (col0 + k < a.K && s < runs) {
      const uint32_t* w = turned + k * kLdsStride + s * 4;
      // through the caches: a run of 128 bytes starts anywhere, and the workgroups beside
      // this one write the rest of its lines (13.5 against 21.8 us past the caches)
      *reinterpret_cast<u32x4*>(a.XT + (col0 + k) * a.cap + f.col + s * 16) = u32x4{w[0], w[1], w[2], w[3]};
    }
  }
}

template <int TPR, int NV>
hipError_t launch_silu(const SiluArgs& a, int block, hipStream_t stream) {
  constexpr int kTeams = threads_of(TPR) / TPR;
  const int64_t want = (a.rows + kTeams - 1) / kTeams;
  const dim3 grid((uint32_t)(want < 65536 ? want : 65536)), threads(threads_of(TPR));
  if (block) hipLaunchKernelGGL((silu_mul_quantize_kernel<TPR, NV, true>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((silu_mul_quantize_kernel<TPR, NV, false>), grid, threads, 0, stream, a);
  return hipGetLastError();
}

template <int TX>
hipError_t launch_silu_back(const SiluBackwardArgs& a, hipStream_t stream) {
  const int chunks = (a.I / 8 + TX - 1) / TX;
  const int64_t work = (a.rows + 256 / TX - 1) / (256 / TX) * chunks;
  hipLaunchKernelGGL((silu_mul_backward_kernel<TX>), dim3((uint32_t)(work < (1 << 20) ? work : (1 << 20))), dim3(256), 0,
                     stream, a, chunks, work);
  return hipGetLastError();
}

template <bool E4M3>
hipError_t launch_k_offsets(const KOffsetsArgs& a, hipStream_t stream) {
  const int chunks = (int)k_offsets_chunks(a.R, a.G);
  const int tiles = (a.K + kTile - 1) / kTile;
  if (chunks > 0) {
    hipLaunchKernelGGL((column_amax_kernel<E4M3>), dim3(chunks * tiles), dim3(256), 0, stream, a, tiles);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((transpose_quantize_kernel<E4M3>), dim3((chunks + 1) * tiles), dim3(256), 0, stream, a, tiles,
                     chunks);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_silu_mul_quantize(const SiluArgs& given, int block, hipStream_t stream) {
  SiluArgs a = given;
  if (a.rows == 0) return hipSuccess;
  a.stream = a.rows * a.I * 4 > kStreamBytes;
  // Threads and vectors per row, with 12 M elements, us: I = 512: a wave per row 15.8, 256
  // threads 33.4.  2048: 256 threads 14.9, a wave with four vectors 16.3.  4096: 512
  // threads 14.9, 256 with two vectors 15.6.  7168: 512 with two 15.6, 256 with four 16.5,
  // 1024 with one 15.7.  14336: 1024 with two 16.0, with four 25.8.
  const int nvec = a.I / 8;
  if (nvec <= 64) return launch_silu<64, 1>(a, block, stream);
  if (nvec <= 128) return launch_silu<64, 2>(a, block, stream);
  if (nvec <= 256) return launch_silu<256, 1>(a, block, stream);
  if (nvec <= 512) return launch_silu<512, 1>(a, block, stream);
  if (nvec <= 1024) return launch_silu<512, 2>(a, block, stream);
  if (nvec <= 2048) return launch_silu<1024, 2>(a, block, stream);
  return launch_silu<1024, 4>(a, block, stream);
}

hipError_t launch_silu_mul_backward(const SiluBackwardArgs& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  // 12 M elements, us, with 64 / 128 / 256 threads along the row: I = 512: 16.5 / - / 17.7,
  // 1000: 17.9 / 16.4 / 17.3, 2048: - / 16.0 / 15.8, 7168: - / 16.2 / 17.4.
  return a.I / 8 <= 64 ? launch_silu_back<64>(a, stream) : launch_silu_back<128>(a, stream);
}

hipError_t launch_quantize_k_offsets(const KOffsetsArgs& a, hipStream_t stream) {
  if (a.K == 0 || a.G == 0) return hipSuccess;
  return a.x_scale ? launch_k_offsets<true>(a, stream) : launch_k_offsets<false>(a, stream);
}

}  // namespace fp8gg
