// Routing of tokens to experts, its plan (rows per expert, places of the pairs) and
// its gradient (gfx950).
//
// Choice.  A team of 16 lanes (E <= 256; else the wave's 64) holds one token's keys in
// registers, up to 16 per lane.  Each of the k rounds takes the largest key (a scan of
// the lane's own, then moves inside the row of 16 lanes, no LDS) and, among equal ones,
// the lowest index, and takes it out.
//
// What has to be compared exactly.  Scores rise with their logits, so without a bias
// and with groups ranked by their best expert the logits themselves are the keys: exact
// and no exponential.  Otherwise keys are p + bias or sums of two of them in fp32, off
// by a few units in the last place; every pair of neighbours in the order taken (and the
// border between kept and dropped groups) is checked, and where two are nearer than the
// error bound the token is decided again in fp64.  With scores spread like a router's
// that is one token in a few hundred.
//
// Plan.  A stable counting sort of the pairs by expert: each workgroup counts its
// tokens' experts, the second kernel adds up the counts before its own block and ranks
// the block's pairs by comparing expert numbers within a wave (ballots over their bits)
// and counting across waves.  Integer sums only, so the order is fixed.
#include "fp8gg_layer_internal.h"

namespace fp8gg {

namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kMaxExperts = 1024;
constexpr int kMaxChosen = 16;
constexpr int kMaxBlocks = 256;        // workgroups whose counts the second kernel adds up

struct MaxK {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a > b ? a : b; }
};

template <int L, typename T, typename Op>
__device__ __forceinline__ T team_reduce(T x, Op op) {
  if constexpr (L == 16) return row16_reduce(x, op);
  else return wave_reduce(x, op);
}

// Whether any lane of the token's team says so.
template <int L>
__device__ __forceinline__ bool team_any(bool p, int tok) {
  const uint64_t b = __ballot(p);
  if constexpr (L == 64) return b != 0;
  else return ((b >> (tok * L)) & ((uint64_t(1) << (L & 63)) - 1)) != 0;
}

// The expert of the lane's v-th key.  From four keys per lane on, four neighbouring
// experts sit in one lane, so that a row is read with 16-byte (bf16: 8-byte) loads.
// Expert numbers rise with v within a lane.
template <int L, int V>
__device__ __forceinline__ int expert_of(int v, int l) {
  if constexpr (V >= 4) return (v >> 2) * (4 * L) + l * 4 + (v & 3);
  else return v * L + l;
}

template <typename T>
__device__ __forceinline__ T none() { return -__builtin_huge_valf(); }

// A logit or bias as it counts: NaN and -infinity take the expert out, +infinity is the
// largest finite value, -0 is 0.
__device__ __forceinline__ float counted(float x) {
  const float y = x + 0.0f;
  return !(y > -__builtin_huge_valf()) ? -__builtin_huge_valf() : (y > 3.402823466e38f ? 3.402823466e38f : y);
}

__device__ __forceinline__ float logit_at(const void* logits, int bf16, int64_t i) {
  return counted(bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(logits)[i] << 16)
                      : reinterpret_cast<const float*>(logits)[i]);
}

template <int L, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int l, float (&x)[V]) {
  const int64_t base = t * a.E;
  if constexpr (V >= 4) {
    if (a.E % 4 == 0) {
#pragma unroll
      for (int v = 0; v < V; v += 4) {
        const int e = expert_of<L, V>(v, l);
        f32x4 w = {none<float>(), none<float>(), none<float>(), none<float>()};
        if (e < a.E) {
          if (a.bf16) {
            const u32x2 q = *reinterpret_cast<const u32x2*>(reinterpret_cast<const uint16_t*>(a.logits) + base + e);
            w = f32x4{__uint_as_float(q[0] << 16), __uint_as_float(q[0] & 0xFFFF0000u), __uint_as_float(q[1] << 16),
                      __uint_as_float(q[1] & 0xFFFF0000u)};
          } else {
            w = *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(a.logits) + base + e);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) x[v + i] = counted(w[i]);
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L, V>(v, l);
    x[v] = e < a.E ? logit_at(a.logits, a.bf16, base + e) : none<float>();
  }
}

// exp and 1 / x as the precision of the key asks for.  fp32: the hardware's exp2 and
// reciprocal, whose error kMargin covers.
__device__ __forceinline__ float key_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }
__device__ __forceinline__ double key_exp(double x) { return exp(x); }
__device__ __forceinline__ float key_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double key_rcp(double x) { return 1.0 / x; }

// fp64 keys are compared as multiples of 2^-44: sums of two scores that are equal in
// exact arithmetic, as sigmoid(x) + sigmoid(-x) for every x, then tie, and adding two
// such keys rounds nothing more.
__device__ __forceinline__ float on_grid(float key) { return key; }
__device__ __forceinline__ double on_grid(double key) { return rint(key * 0x1p44) * 0x1p-44; }

// Keys p + bias.  Error of the fp32 ones, with u = 2^-24: the rounded exponent makes
// exp(x) off by 2 u |x| relative to itself, exp2 and the reciprocal by 2 u each.
// Sigmoid: p (1 - p) |x| <= 0.23 and p (1 - p) <= 0.25, so p is off by at most 5 u and
// the key by u more per unit of its size.  Softmax: p |x - max| <= 0.37, and the sum of
// E <= 1024 positive terms (16 per lane, then 6 steps) adds at most 22 u.  So a key is
// within 8 u (sigmoid) or 32 u (softmax), and two sums of two keys are told apart by
// more than four times that: 2^-19 and 2^-17.
template <typename K, int L, int V>
__device__ __forceinline__ void make_keys(const RouteArgs& a, int l, const float (&x)[V], K (&key)[V]) {
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = key_rcp(K(1) + key_exp(-K(x[v])));
  } else {
    float m = none<float>();
#pragma unroll
    for (int v = 0; v < V; ++v) m = MaxK()(m, x[v]);
    m = team_reduce<L>(m, MaxK());
    const K most = m > none<float>() ? K(m) : K(0);
    K sum = K(0);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = key_exp(K(x[v]) - most);
      sum += key[v];
    }
    const K r = key_rcp(team_reduce<L>(sum, AddF()));
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] *= r;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float b = 0.f;
    const int e = expert_of<L, V>(v, l);
    if (a.bias && e < a.E) b = counted(a.bias[e]);
    key[v] = x[v] > none<float>() && b > none<float>() ? on_grid(key[v] + K(b)) : none<K>();
  }
}

template <typename K>
__device__ __forceinline__ K margin_of(const RouteArgs& a, K s) {
  const K size = s > K(1) ? s : (s < K(-1) ? -s : K(1));
  return size * (a.sigmoid ? K(0x1p-19) : K(0x1p-17));
}

// Keeps the keys of the topk_group best groups.  `buf`: the token's own LDS, E + n_group
// keys (one word of padding per group keeps the lanes that scan the groups on different
// banks) and n_group scores; only this wave touches it.
template <typename K, int L, int V, bool CHECK>
__device__ __forceinline__ void keep_groups(const RouteArgs& a, int l, int tok, K* buf, K (&key)[V], bool& close) {
  const int per = a.E / a.n_group;
  const uint32_t magic = ((1u << 22) + per - 1) / per;   // e / per for e < 1024
  K* score = buf + a.E + a.n_group;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L, V>(v, l);
    if (e < a.E) buf[e + (int)((e * magic) >> 22)] = key[v];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (l < a.n_group) {
    K m1 = none<K>(), m2 = none<K>();
    for (int i = 0; i < per; ++i) {
      const K x = buf[l * (per + 1) + i];
      const K low = x < m1 ? x : m1;
      m2 = low > m2 ? low : m2;
      m1 = x > m1 ? x : m1;
    }
    score[l] = a.group_top == 2 && m2 > none<K>() ? m1 + m2 : m1;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  bool keep = false, near = false;
  if (l < a.n_group) {
    const K s = score[l];
    int rank = 0;
    K gap = K(3.0e38f);
    for (int o = 0; o < a.n_group; ++o) {
      const K other = score[o];
      const bool ahead = other > s || (other == s && o < l);
      rank += ahead;
      gap = ahead && other - s < gap ? other - s : gap;
    }
    keep = rank < a.topk_group && s > none<K>();
    // the first group dropped against the last one kept
    near = rank == a.topk_group && s > none<K>() && gap <= margin_of(a, s + gap);
  }
  uint32_t kept = (uint32_t)(__ballot(keep) >> (L == 64 ? 0 : tok * L)) & 0xFFFFu;   // n_group <= 16
  if (CHECK) close |= team_any<L>(near, tok);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L, V>(v, l);
    if (e < a.E && !((kept >> ((e * magic) >> 22)) & 1)) key[v] = none<K>();
  }
}

// The k largest keys: lane j of the team gets the j-th expert (-1: none left).  CHECK:
// `close` tells that two neighbours of the order are too near for fp32, the first one
// left out among them.  Two keys made of the same logit and bias are a true tie; where
// the first ones left out tie with the last one taken, the one after them counts too.
template <typename K, int L, int V, bool CHECK>
__device__ __forceinline__ void choose(const RouteArgs& a, int64_t t, int l, K (&key)[V], int& id, bool& close) {
  K last = K(0);
  int last_e = -1;
  bool open = CHECK;                               // the border is not settled yet
  for (int j = 0; j < a.k || (CHECK && __any(open)); ++j) {
    K m = key[0];
    int mv = 0;
#pragma unroll
    for (int v = 1; v < V; ++v) {
      const bool c = key[v] > m;
      m = c ? key[v] : m;
      mv = c ? v : mv;
    }
    const K top = team_reduce<L>(m, MaxK());
    const bool any = top > none<K>();
    const int e = (int)team_reduce<L>(any && m == top ? (uint32_t)expert_of<L, V>(mv, l) : 0xFFFFFFFFu, MinU());
    if (CHECK && j > 0 && open) {
      bool same = false;
      if (any && last - top <= margin_of(a, last)) {
        if (last == top)
          same = logit_at(a.logits, a.bf16, t * a.E + e) == logit_at(a.logits, a.bf16, t * a.E + last_e) &&
                 (!a.bias || counted(a.bias[e]) == counted(a.bias[last_e]));
        close |= !same;
      }
      open = any && !close && (j < a.k || same);
    }
    if (l == j && j < a.k) id = e;
    // d equals the lane's v-th expert number less the lane's share for the taken one only
    const int d = V >= 4 ? e - l * 4 : e - l;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (d == expert_of<L, V>(v, 0)) key[v] = none<K>();
    last = top;
    last_e = e;
  }
}

// Places of the pairs of one workgroup's tokens.  base[e]: the place of the block's
// first pair of expert e.  Every wave walks a run of 64-pair pieces: first to count,
// then, from the counts of the waves before it, to rank.
template <typename Ids>
__device__ __forceinline__ void place_pairs(Ids ids, int n, int E, const int* base, int* counts, int32_t* dst) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int pieces = (n + 63) / 64;
  const int per_wave = (pieces + kWaves - 1) / kWaves;
  const int bits = 32 - __clz(E);                    // E itself marks a slot without an expert
  int* own = counts + wave * E;
  for (int i = threadIdx.x; i < kWaves * E; i += kThreads) counts[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int p = wave * per_wave; p < (wave + 1) * per_wave && p < pieces; ++p) {
      const int i = p * 64 + lane;
      int e = i < n ? ids(i) : E;
      if (e < 0) e = E;
      uint64_t same = ~uint64_t(0);
      for (int b = 0; b < bits; ++b) {
        const bool one = (e >> b) & 1;
        const uint64_t with = __ballot(one);
        same &= one ? with : ~with;
      }
      const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
      if (e < E) {
        const int at = own[e];
        if (pass) dst[i] = at + before;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (before == 0) own[e] = at + __popcll(same);
      } else if (pass && i < n) {
        dst[i] = -1;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    if (pass == 0) {
      if ((int)threadIdx.x < E) {
        int at = base[threadIdx.x];
        for (int w = 0; w < kWaves; ++w) {
          const int c = counts[w * E + threadIdx.x];
          counts[w * E + threadIdx.x] = at;
          at += c;
        }
      }
      __syncthreads();
    }
  }
}

// Exclusive prefix sum over the workgroup's threads.
__device__ __forceinline__ int prefix_before(int x, int* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int s = x;
  for (int off = 1; off < 64; off <<= 1) {
    const int y = __shfl_up(s, off, 64);
    if (lane >= off) s += y;
  }
  if (lane == 63) waves[wave] = s;
  __syncthreads();
  for (int w = 0; w < wave; ++w) s += waves[w];
  return s - x;
}

// sigmoid(x) exp(-min(most, 0)), most being the row's largest chosen logit: a factor that
// renormalising takes out again, and with it the largest term is at least 1/2.
__device__ __forceinline__ float shifted_sigmoid(float x, float most, bool mine) {
  if (!mine) return 0.f;
  return most > 0.f ? 1.0f / (1.0f + expf(-x)) : expf(x - most) / (1.0f + expf(x));
}

template <int L, int V, bool ARITH>
__global__ void __launch_bounds__(kThreads) route_kernel(RouteArgs a) {
  constexpr int kTokens = kWaves * (64 / L);       // tokens of one pass over the workgroup's waves
  extern __shared__ double dynamic_lds[];
  __shared__ int count[kMaxExperts];
  __shared__ int chosen[64 * kMaxChosen];
  __shared__ int wave_sums[kWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int l = lane % L, tok = lane / L;
  const bool plan = a.M_sizes != nullptr;
  const bool alone = gridDim.x == 1 && a.block_tokens == 64;
  if (plan) {
    count[threadIdx.x] = 0;
    chosen[threadIdx.x] = -1;
    __syncthreads();
  }
  const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
  for (int at = wave * (64 / L); at < a.block_tokens; at += kTokens) {
    if (first + at >= a.T) break;                  // uniform over the wave
    const bool live = first + at + tok < a.T;
    const int64_t t = live ? first + at + tok : a.T - 1;
    float x[V];
    load_row<L, V>(a, t, l, x);
    int id = -1;
    bool close = false;
    if constexpr (ARITH) {
      const int region = a.E + 2 * a.n_group + 1;
      float key[V];
      make_keys<float, L, V>(a, l, x, key);
      if (a.n_group > 1)
        keep_groups<float, L, V, true>(a, l, tok, reinterpret_cast<float*>(dynamic_lds + (wave * (64 / L) + tok) * region),
                                       key, close);
      choose<float, L, V, true>(a, t, l, key, id, close);
      if (__any(close)) {
        double exact[V];
        int exact_id = -1;
        bool unused = false;
        make_keys<double, L, V>(a, l, x, exact);
        if (a.n_group > 1)
          keep_groups<double, L, V, false>(a, l, tok, dynamic_lds + (wave * (64 / L) + tok) * region, exact, unused);
        choose<double, L, V, false>(a, t, l, exact, exact_id, unused);
        if (close) id = exact_id;
      }
    } else {
      bool unused = false;
      float key[V];
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v];
      if (a.n_group > 1)
        keep_groups<float, L, V, false>(
            a, l, tok, reinterpret_cast<float*>(dynamic_lds) + (wave * (64 / L) + tok) * (a.E + 2 * a.n_group + 1), key,
            unused);
      choose<float, L, V, false>(a, t, l, key, id, unused);
    }
    // Weights: lane j has the j-th expert; all of them lie in the team's first 16 lanes.
    const bool mine = l < a.k && id >= 0;
    const float lx = mine ? logit_at(a.logits, a.bf16, t * a.E + id) : none<float>();
    float p;
    if (a.sigmoid) {
      if (a.renormalize) {
        p = shifted_sigmoid(lx, row16_reduce(lx, MaxK()), mine);
        p = p / row16_reduce(p, AddF());
      } else {
        p = mine ? 1.0f / (1.0f + expf(-lx)) : 0.f;
      }
    } else if (a.renormalize) {
      // softmax over the chosen: the other experts cancel
      const float most = row16_reduce(lx, MaxK());
      p = mine ? expf(lx - most) : 0.f;
      p = p / row16_reduce(p, AddF());
    } else {
      float most = none<float>(), sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) most = MaxK()(most, x[v]);
      most = team_reduce<L>(most, MaxK());
#pragma unroll
      for (int v = 0; v < V; ++v) sum += x[v] > none<float>() ? expf(x[v] - most) : 0.f;
      sum = team_reduce<L>(sum, AddF());
      p = mine ? expf(lx - most) / sum : 0.f;
    }
    if (live && l < a.k) {
      a.weights[t * a.k + l] = mine ? p * a.scale : 0.f;
      a.ids[t * a.k + l] = id;
      if (plan) {
        if (id >= 0) atomicAdd(&count[id], 1);
        if (alone) chosen[(at + tok) * a.k + l] = id;
      }
    }
  }
  if (!plan) return;
  __syncthreads();
  if (!alone) {
    if ((int)threadIdx.x < a.E) a.hist[(int64_t)blockIdx.x * a.E + threadIdx.x] = count[threadIdx.x];
    return;
  }
  const int c = count[threadIdx.x];                // 0 beyond E
  const int before = prefix_before(c, wave_sums);
  if ((int)threadIdx.x < a.E) a.M_sizes[threadIdx.x] = c;
  __syncthreads();
  count[threadIdx.x] = before;
  __syncthreads();
  place_pairs([&](int i) { return chosen[i]; }, (int)a.T * a.k, a.E, count, reinterpret_cast<int*>(dynamic_lds),
              a.dst_row);
}

// Second kernel of the plan: block b adds up the counts of all blocks and of those
// before it, then places its own pairs.
__global__ void __launch_bounds__(kThreads) place_kernel(RouteArgs a, int blocks) {
  extern __shared__ double dynamic_lds[];
  __shared__ int total[kMaxExperts];
  __shared__ int earlier[kMaxExperts];
  __shared__ int wave_sums[kWaves];
  total[threadIdx.x] = 0;
  earlier[threadIdx.x] = 0;
  __syncthreads();
  // lanes of experts side by side, as many rows of counts at once as fit
  const int width = a.E <= 64 ? 64 : (a.E <= 128 ? 128 : (a.E <= 256 ? 256 : (a.E <= 512 ? 512 : 1024)));
  const int e = threadIdx.x % width, step = kThreads / width;
  if (e < a.E) {
    int all = 0, prior = 0;
    for (int b = threadIdx.x / width; b < blocks; b += step) {
      const int c = a.hist[(int64_t)b * a.E + e];
      all += c;
      prior += b < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&earlier[e], prior);
  }
  __syncthreads();
  const int c = total[threadIdx.x];
  const int before = prefix_before(c, wave_sums);
  if (blockIdx.x == 0 && (int)threadIdx.x < a.E) a.M_sizes[threadIdx.x] = c;
  earlier[threadIdx.x] += before;
  __syncthreads();
  const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
  const int64_t left = a.T - first;
  const int n = (int)(left < a.block_tokens ? left : a.block_tokens) * a.k;
  const int32_t* ids = a.ids + first * a.k;
  place_pairs([&](int i) { return ids[i]; }, n, a.E, earlier, reinterpret_cast<int*>(dynamic_lds),
              a.dst_row + first * a.k);
}

template <int L, int V, bool ARITH>
hipError_t launch(const RouteArgs& a, int blocks, hipStream_t stream) {
  const size_t keys = a.n_group > 1 ? (size_t)kWaves * (64 / L) * (a.E + 2 * a.n_group + 1) * (ARITH ? 8 : 4) : 0;
  const size_t counts = a.M_sizes && blocks == 1 ? (size_t)kWaves * a.E * sizeof(int) : 0;
  const size_t lds = keys > counts ? keys : counts;
  hipLaunchKernelGGL((route_kernel<L, V, ARITH>), dim3(blocks), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

template <bool ARITH>
hipError_t launch_by_width(const RouteArgs& a, int blocks, hipStream_t stream) {
  if (a.E <= 16) return launch<16, 1, ARITH>(a, blocks, stream);
  if (a.E <= 32) return launch<16, 2, ARITH>(a, blocks, stream);
  if (a.E <= 64) return launch<16, 4, ARITH>(a, blocks, stream);
  if (a.E <= 128) return launch<16, 8, ARITH>(a, blocks, stream);
  if (a.E <= 256) return launch<16, 16, ARITH>(a, blocks, stream);
  if (a.E <= 512) return launch<64, 8, ARITH>(a, blocks, stream);
  return launch<64, 16, ARITH>(a, blocks, stream);
}

// One wave per token.  Only the chosen logits matter, except for softmax weights that
// are not renormalised, whose gradient reaches every expert.  The row is put together in
// LDS, so that it leaves in whole vectors.
__global__ void __launch_bounds__(256) route_backward_kernel(RouteBackwardArgs a) {
  __shared__ float rows[4][kMaxExperts];
  const int lane = threadIdx.x & 63;
  float* row = rows[threadIdx.x >> 6];
  for (int e = lane; e < a.E; e += 64) row[e] = 0.f;
  const bool every = !a.sigmoid && !a.renormalize;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += (int64_t)gridDim.x * 4) {
    const int64_t base = t * a.E;
    const int id = lane < a.k ? a.ids[t * a.k + lane] : -1;
    const bool inside = id >= 0 && id < a.E;
    const float x = inside ? logit_at(a.logits, a.bf16, base + id) : none<float>();
    const bool mine = inside && x > none<float>();
    const float g = mine ? a.dweights[t * a.k + lane] * a.scale : 0.f;
    float dx = 0.f;
    if (every) {
      float most = none<float>(), sum = 0.f;
      for (int e = lane; e < a.E; e += 64) most = MaxK()(most, logit_at(a.logits, a.bf16, base + e));
      most = wave_reduce(most, MaxK());
      most = most > none<float>() ? most : 0.f;
      for (int e = lane; e < a.E; e += 64) {
        row[e] = expf(logit_at(a.logits, a.bf16, base + e) - most);
        sum += row[e];
      }
      sum = wave_reduce(sum, AddF());
      const float r = sum > 0.f ? 1.0f / sum : 0.f;
      const float p = mine ? expf(x - most) * r : 0.f;
      const float dot = row16_reduce(p * g, AddF());   // the chosen lie in the first 16 lanes
      const float d = __shfl(dot, 0, 64);
      for (int e = lane; e < a.E; e += 64) row[e] = -d * (row[e] * r);
      dx = p * (g - d);
    } else if (a.sigmoid) {
      const float s = 1.0f / (1.0f + expf(-x)), rest = 1.0f / (1.0f + expf(x));
      if (a.renormalize) {
        const float p = shifted_sigmoid(x, row16_reduce(x, MaxK()), mine);
        const float sum = row16_reduce(p, AddF());
        const float q = mine ? p / sum : 0.f;
        const float dot = row16_reduce(q * g, AddF());
        dx = q * rest * (g - dot);
      } else {
        dx = g * s * rest;
      }
    } else {
      const float most = row16_reduce(x, MaxK());
      const float p = mine ? expf(x - most) : 0.f;
      const float sum = row16_reduce(p, AddF());
      const float q = sum > 0.f ? p / sum : 0.f;
      const float dot = row16_reduce(q * g, AddF());
      dx = q * (g - dot);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (mine) row[id] = dx;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (a.bf16) {
      uint16_t* out = reinterpret_cast<uint16_t*>(a.dlogits) + base;
      if (a.E % 8 == 0) {
        for (int j = lane; j < a.E / 8; j += 64) {
          F8 f;
#pragma unroll
          for (int i = 0; i < 8; ++i) f.v[i] = row[8 * j + i];
          reinterpret_cast<u32x4*>(out)[j] = pack_bf16(f);
        }
      } else {
        for (int e = lane; e < a.E; e += 64) out[e] = (uint16_t)pack_bf16(row[e], 0.f);
      }
    } else {
      float* out = reinterpret_cast<float*>(a.dlogits) + base;
      if (a.E % 4 == 0) {
        for (int j = lane; j < a.E / 4; j += 64)
          reinterpret_cast<f32x4*>(out)[j] = f32x4{row[4 * j], row[4 * j + 1], row[4 * j + 2], row[4 * j + 3]};
      } else {
        for (int e = lane; e < a.E; e += 64) out[e] = row[e];
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (mine) row[id] = 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

}  // namespace

int route_block_tokens(int64_t T) {
  const int64_t n = (T + 64 * kMaxBlocks - 1) / (64 * kMaxBlocks);
  return (int)(64 * (n > 0 ? n : 1));
}

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.T == 0 && !a.M_sizes) return hipSuccess;
  // T == 0 with a plan: one workgroup writes zero counts
  const int blocks = a.T == 0 ? 1 : (int)((a.T + a.block_tokens - 1) / a.block_tokens);
  const bool arith = a.bias || (a.n_group > 1 && a.group_top == 2);
  hipError_t e = arith ? launch_by_width<true>(a, blocks, stream) : launch_by_width<false>(a, blocks, stream);
  if (e != hipSuccess || !a.M_sizes || blocks == 1) return e;
  hipLaunchKernelGGL(place_kernel, dim3(blocks), dim3(kThreads), (size_t)kWaves * a.E * sizeof(int), stream, a, blocks);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const int64_t want = (a.T + 3) / 4;
  hipLaunchKernelGGL(route_backward_kernel, dim3((uint32_t)(want < 8192 ? want : 8192)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8gg
