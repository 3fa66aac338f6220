// Routing of tokens to experts, its plan (rows per expert, places of the pairs) and
// its gradient (gfx950).
//
// Choice.  A team of 16 or 64 lanes holds one token's keys in registers, up to 32 per
// lane.  The k-th largest of the lanes' own maxima bounds the k-th largest key from
// below; the keys that reach it, a dozen or so of 256, go to LDS,
// and each of them finds its rank by comparing itself with the others.  That is about a
// third of the instructions of k rounds of a maximum over the team (48 us at 16384
// tokens, 256 experts in 8 groups, k = 8, against 18).
//
// What has to be compared exactly.  Scores rise with their logits, so without a bias the
// logits themselves rank the experts, and the groups where their best expert stands for
// them: exact and no exponential.  Otherwise keys are p + bias or sums of two of them in
// fp32, off by a few units in the last place; where two of the ranked keys (or the last
// group kept and the first one dropped) are nearer than the error bound, those keys are
// computed again in fp64 and ranked by that.
//
// Plan.  A stable counting sort of the pairs by expert: each workgroup counts its
// tokens' experts, the second kernel adds up the counts before its own block and ranks
// the block's pairs by comparing expert numbers within a wave (ballots over their bits)
// and counting across waves.  Integer sums only, so the order is fixed.  A few tokens are
// planned by the workgroup that chooses, up to 4096 pairs by a second one that counts
// them itself.
//
// 16384 tokens, 256 experts in 8 groups, k = 8, sigmoid and bias: 18 us for the choice (15
// alone in a loop), 8.5 for the plan.  The logits (16.8 MB) take 3.2 us at a copy's rate.
// The choice's 1350 vector instructions per four tokens are 9 us of issue, 4 waves on each
// SIMD; the rest is waiting: a workgroup of 64 tokens has 84 KB of LDS and a CU to itself, so
// that all waves load, rank and finish in step, and the few tokens decided in fp64 end up to
// 4 us after the others.
//
// What rows hold matters.  Rows with more candidates than the list has places go through
// choose_in_rounds, and their wave waits.  16384 x 256, us, and with spread logits and k = 8:
// k = 16, where 16 lanes give too low a bound, 104 and 19; one row in four of equal logits,
// as padding leaves them, 73 and 19, in groups with a zero bias 170 and 27 (with a bias that
// tells the experts apart 26); softmax with a bias, whose fp32 keys are told apart by 2^-16
// alone, 30.
//
// 16 tokens, 8 experts: one launch, 4.9 us.  64 tokens of the 256 experts: 9.9 us, 6.4 of
// them the choice, which is one wave's chain of instructions from the load of a row to its
// weights.
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

// The expert of the lane's v-th key: neighbouring experts lie in neighbouring lanes, so
// that every lane has its share of each group of experts.  (With four neighbours per
// lane, for wider loads, kept groups may leave half the lanes without a key: the
// bound below falls and the list of candidates grows, to 60 of them now and then.)
template <int L>
__device__ __forceinline__ int expert_of(int v, int l) { return v * L + l; }

template <typename T>
__device__ __forceinline__ T none() { return -__builtin_huge_valf(); }

// A logit or bias as it counts: NaN and -infinity take the expert out, +infinity is the
// largest finite value.
__device__ __forceinline__ float counted(float x) {
  return __builtin_fminf(__builtin_fmaxf(x, -__builtin_huge_valf()), 3.402823466e38f);
}

__device__ __forceinline__ float logit_at(const void* logits, int bf16, int64_t i) {
  return counted(bf16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(logits)[i] << 16)
                      : reinterpret_cast<const float*>(logits)[i]);
}

template <int L, int V>
__device__ __forceinline__ void load_row(const RouteArgs& a, int64_t t, int l, float (&x)[V]) {
  const int64_t base = t * a.E;
  if (a.E == L * V) {   // no lane past the last expert
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = logit_at(a.logits, a.bf16, base + expert_of<L>(v, l));
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = expert_of<L>(v, l);
      x[v] = e < a.E ? logit_at(a.logits, a.bf16, base + e) : none<float>();
    }
  }
}

// The hardware's exp2 and reciprocal, whose error margin_of covers.
__device__ __forceinline__ float fast_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504088896341f); }

// fp32 keys p + bias.  Their error, with u = 2^-24: the rounded exponent makes exp(x)
// off by 2 u |x| relative to itself, exp2 and the reciprocal by 2 u each.  Sigmoid:
// p (1 - p) |x| <= 0.23 and p (1 - p) <= 0.25, so p is off by at most 5 u and the key by
// u more per unit of its size.  Softmax: p |x - max| <= 0.37, and the sum of positive
// terms (32 per lane, then 4 steps; or 16, then 6) adds at most 36 u.  So a key is within
// 8 u (sigmoid) or 44 u (softmax), and two sums of two keys are told apart by more than
// four times that: 2^-19 = 32 u and 2^-16 = 256 u cover both.
template <int L, int V>
__device__ __forceinline__ void make_keys(const RouteArgs& a, int l, const float (&x)[V], float (&key)[V]) {
  if (a.sigmoid) {
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = __builtin_amdgcn_rcpf(1.0f + fast_exp(-x[v]));
  } else {
    float m = none<float>(), sum = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) m = MaxK()(m, x[v]);
    m = team_reduce<L>(m, MaxK());
    m = m > none<float>() ? m : 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      key[v] = fast_exp(x[v] - m);
      sum += key[v];
    }
    const float r = __builtin_amdgcn_rcpf(team_reduce<L>(sum, AddF()));
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] *= r;
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L>(v, l);
    const float b = a.bias ? counted(a.bias[e < a.E ? e : a.E - 1]) : 0.f;
    key[v] = x[v] > none<float>() && b > none<float>() ? key[v] + b : none<float>();
  }
}

template <typename K>
__device__ __forceinline__ K margin_of(const RouteArgs& a, K s) {
  const K size = s > K(1) ? s : (s < K(-1) ? -s : K(1));
  return size * (a.sigmoid ? K(0x1p-19) : K(0x1p-16));
}

// The key of one expert in fp64, from its logit in memory (taken seldom, so nothing is
// kept in registers for it).  Not rounded further: scores far below the row's largest, and
// sigmoids near 1, keep their order.  Without arith: the logit itself.
//
// A call, not inlined: the polynomials of exp would otherwise be kept in registers
// through the whole kernel and push its own values out.
__device__ __attribute__((noinline)) double exact_exp(double x) { return exp(x); }

struct ExactKey {
  const RouteArgs& a;
  int64_t base;
  bool arith;
  double most, sum;      // softmax
  __device__ __forceinline__ double operator()(int e) const {
    const double x = logit_at(a.logits, a.bf16, base + e);
    if (!arith) return x;
    const double b = a.bias ? (double)counted(a.bias[e]) : 0.0;
    const double w = exact_exp(a.sigmoid ? -x : x - most);
    const double p = a.sigmoid ? 1.0 / (1.0 + w) : w / sum;
    return x > none<double>() && b > none<double>() ? p + b : none<double>();
  }
};

template <int L>
__device__ __forceinline__ ExactKey exact_key(const RouteArgs& a, int64_t t, int l, bool arith) {
  ExactKey k{a, t * a.E, arith, 0.0, 1.0};
  if (arith && !a.sigmoid) {
    float m = none<float>();
#pragma unroll 1
    for (int e = l; e < a.E; e += L) m = MaxK()(m, logit_at(a.logits, a.bf16, k.base + e));
    m = team_reduce<L>(m, MaxK());
    k.most = m > none<float>() ? m : 0.f;
    double sum = 0.0;
#pragma unroll 1
    for (int e = l; e < a.E; e += L) sum += exact_exp((double)logit_at(a.logits, a.bf16, k.base + e) - k.most);
    k.sum = team_reduce<L>(sum, AddF());
  }
  return k;
}

// e / (E / n_group) for e < 1024.
struct GroupOf {
  uint32_t magic;
  __device__ __forceinline__ explicit GroupOf(int per) : magic(((1u << 22) + per - 1) / per) {}
  __device__ __forceinline__ int operator()(int e) const { return (int)(__umul24((uint32_t)e, magic) >> 22); }
};

constexpr int kMaxGroups = 16;

// x to 44 significant bits (halves away from zero): sums of two keys that are equal in exact
// arithmetic, as sigmoid(x) + sigmoid(-x) for every x, are the same then, whatever their
// last bits in fp64.
__device__ __forceinline__ double significant(double x) {
  return __builtin_bit_cast(double, (__builtin_bit_cast(uint64_t, x) + 0x100) & ~uint64_t(0x1FF));
}

// The groups kept, as a mask, from lane g's (g < n_group) score and its rank.
template <typename K, int L>
__device__ __forceinline__ uint32_t groups_within(const RouteArgs& a, int l, int tok, K s, int rank) {
  const bool real = l < a.n_group && s > none<K>();
  return (uint32_t)(__ballot(real && rank < a.topk_group) >> (L == 64 ? 0 : tok * L)) & 0xFFFFu;
}

// Group l's score in fp64, one lane per group, from the experts whose fp32 key reaches
// `least` (the second one's less the error bound): nearly always the two that count, so
// they are listed first and their scores computed side by side.
template <int L>
__device__ __forceinline__ uint32_t keep_groups_exactly(const RouteArgs& a, int l, int tok, const float* buf, float least,
                                                        const ExactKey& key) {
  constexpr int kListed = 4;
  const int per = a.E / a.n_group;
  const float* own = buf + l * (per + 1);
  int list[kListed] = {}, n = 0;
  if (l < a.n_group) {
    for (int i = 0; i < per; ++i) {
      if (own[i] < least || !(own[i] > none<float>())) continue;
#pragma unroll
      for (int u = 0; u < kListed; ++u)
        if (u == n) list[u] = i;
      ++n;
    }
  }
  double m1 = none<double>(), m2 = none<double>();
  const auto take = [&](double x) {
    const double low = x < m1 ? x : m1;
    m2 = low > m2 ? low : m2;
    m1 = x > m1 ? x : m1;
  };
#pragma unroll
  for (int u = 0; u < kListed; ++u)
    if (u < n && n <= kListed) take(key(l * per + list[u]));
  if (n > kListed) {
#pragma unroll 1
    for (int i = 0; i < per; ++i)
      if (own[i] >= least) take(key(l * per + i));
  }
  if (a.group_top == 2 && m1 > none<double>()) m1 = significant(m2 > none<double>() ? m1 + m2 : m1);
  int rank = 0;
  for (int o = 0; o < a.n_group; ++o) {
    const double other = __shfl(m1, (L == 64 ? 0 : tok * L) + o, 64);
    rank += other > m1 || (other == m1 && o < l);
  }
  return groups_within<double, L>(a, l, tok, m1, rank);
}

// The groups kept, by way of the token's own LDS: kMaxGroups best and second keys and E +
// n_group keys (one word of padding per group keeps the lanes that scan the groups on
// different banks).  Only this wave touches it.  Up to eight lanes scan a group where there
// are enough.  ARITH: the keys are fp32 sums, and a border too close is decided in fp64.
// With group_top 2 a score is half the sum: the halves are exact, and no sum of two finite
// keys leaves fp32 (biases of the type's lowest value would take a group out).
template <int L, int V, bool ARITH>
__device__ __forceinline__ uint32_t keep_groups(const RouteArgs& a, int64_t t, int l, int tok, float* lds,
                                                const float (&key)[V]) {
  const int per = a.E / a.n_group;
  const GroupOf group(per);
  float *best = lds, *second = lds + kMaxGroups, *buf = lds + 2 * kMaxGroups;
  if (a.E == L * V) {
#pragma unroll
    for (int v = 0; v < V; ++v) buf[expert_of<L>(v, l) + group(expert_of<L>(v, l))] = key[v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (expert_of<L>(v, l) < a.E) buf[expert_of<L>(v, l) + group(expert_of<L>(v, l))] = key[v];
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const int shift = 8 * a.n_group <= L ? 3 : 4 * a.n_group <= L ? 2 : 2 * a.n_group <= L ? 1 : 0;
  const int g = l >> shift, step = 1 << shift;
  float m1 = none<float>(), m2 = none<float>();
  const auto take = [&](float x) {
    const float low = x < m1 ? x : m1;
    m2 = low > m2 ? low : m2;
    m1 = x > m1 ? x : m1;
  };
  if (g < a.n_group) {
#pragma unroll 8
    for (int i = l & (step - 1); i < per; i += step) take(buf[g * (per + 1) + i]);
  }
  const auto join = [&](float o1, float o2) {
    take(o1);
    m2 = o2 > m2 ? o2 : m2;
  };
  if (shift > 0) join(dpp<0xB1>(m1), dpp<0xB1>(m2));       // lanes 1 0 3 2
  if (shift > 1) join(dpp<0x4E>(m1), dpp<0x4E>(m2));       // lanes 2 3 0 1
  if (shift > 2) join(dpp<0x141>(m1), dpp<0x141>(m2));     // mirror in each half row
  // A sum may be far smaller than what was added: its error goes by the largest key.
  float largest = 0.f;
  if (ARITH && g < a.n_group) {
    if (m1 > none<float>()) largest = fabsf(m1);
    if (m2 > none<float>()) largest = MaxK()(largest, fabsf(m2));
  }
  const float part = a.group_top == 2 ? 0.5f : 1.0f;
  if (g < a.n_group) {
    best[g] = a.group_top == 2 && m2 > none<float>() ? part * m1 + part * m2 : part * m1;
    second[g] = a.group_top == 2 && m2 > none<float>() ? m2 : m1;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const float mine = l < a.n_group ? best[l] : none<float>();
  // all scores at once: a read per step of the loop would wait for LDS each time
  f32x4 all[kMaxGroups / 4];
#pragma unroll
  for (int i = 0; i < kMaxGroups / 4; ++i) all[i] = reinterpret_cast<const f32x4*>(best)[i];
  int rank = 0;
  float gap = 3.0e38f;
#pragma unroll
  for (int o = 0; o < kMaxGroups; ++o) {
    if (o >= a.n_group) break;
    const float other = all[o / 4][o % 4];
    const bool ahead = other > mine || (other == mine && o < l);
    rank += ahead;
    const float above = ahead ? other - mine : gap;
    gap = above < gap ? above : gap;
  }
  uint32_t kept = groups_within<float, L>(a, l, tok, mine, rank);
  if constexpr (ARITH) {
    // is the first group dropped too close to the last one kept for fp32?
    const float margin = part * margin_of(a, team_reduce<L>(largest, MaxK()));
    if (__any(l < a.n_group && mine > none<float>() && rank == a.topk_group && gap <= margin)) {
      const float low = l < a.n_group ? second[l] : none<float>();
      kept = keep_groups_exactly<L>(a, l, tok, buf, low - margin_of(a, low), exact_key<L>(a, t, l, true));
    }
  }
  return kept;
}

template <int L, int V>
__device__ __forceinline__ void drop_groups(const RouteArgs& a, int l, uint32_t kept, float (&key)[V]) {
  const GroupOf group(a.E / a.n_group);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = expert_of<L>(v, l);
    if (e < a.E && !((kept >> group(e)) & 1)) key[v] = none<float>();
  }
}

// The k largest keys in k rounds of a maximum over the team, each round among those that
// come after the last one taken: lane j gets the j-th expert (-1: none left).  For rows
// with more candidates than the LDS list holds, as where many logits are equal.
template <int L>
__device__ __forceinline__ int choose_in_rounds(const RouteArgs& a, int l, uint32_t kept, const ExactKey& key) {
  const GroupOf group(a.E / a.n_group);
  int id = -1, last_e = -1;
  double last = __builtin_huge_val();
  for (int j = 0; j < a.k; ++j) {
    double m = none<double>();
    int me = 0;
#pragma unroll 1
    for (int e = l; e < a.E; e += L) {
      const double x = (kept >> group(e)) & 1 ? key(e) : none<double>();
      if (x > m && (x < last || (x == last && e > last_e))) {
        m = x;
        me = e;
      }
    }
    const double top = team_reduce<L>(m, MaxK());
    const bool any = top > none<double>();
    last_e = (int)team_reduce<L>(any && m == top ? (uint32_t)me : 0xFFFFFFFFu, MinU());
    last = top;
    if (l == j) id = last_e;
  }
  return id;
}

// One token's candidates in LDS.
constexpr int kCandidates = 64;
struct alignas(16) Candidates {
  float key[kCandidates];
  int expert[kCandidates];
  double exact[kCandidates];
  int chosen[kMaxChosen];
};

// Lower bound of the k-th largest key: the k-th largest of the team's lanes' maxima.
// -infinity where fewer than k lanes hold a key.
template <int N>
__device__ __forceinline__ int count_reaching(float m, float other_than) {
  // lanes N, N - 1, ... 1 further along the row
  const int here = dpp<0x120 + N>(m) >= other_than;   // row_ror N
  if constexpr (N > 1) return here + count_reaching<N - 1>(m, other_than);
  else return here;
}
template <int L, int V>
__device__ __forceinline__ float bound_of(int k, const float (&key)[V]) {
  float m = key[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = MaxK()(m, key[v]);
  int reaching;
  if constexpr (L == 16) {
    reaching = 1 + count_reaching<15>(m, m);
  } else {
    uint32_t rows[4], a, b;                        // the maxima of the wave's four rows
    swapped<false>(__float_as_uint(m), a, b);
    swapped<true>(a, rows[0], rows[1]);
    swapped<true>(b, rows[2], rows[3]);
    reaching = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = __uint_as_float(rows[i]);
      reaching += (x >= m) + count_reaching<15>(x, m);
    }
  }
  return team_reduce<L>(reaching >= k ? m : none<float>(), MaxK());
}

template <int L>
__device__ __forceinline__ uint32_t team_scan(uint32_t x) {
  if constexpr (L == 64) {
    return wave_scan(x, AddF());
  } else {
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);
    x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);
    return x + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);
  }
}

// Puts the keys that reach `least` into the list; returns how many there are (they fit
// when that is at most kCandidates).
template <int L, int V>
__device__ __forceinline__ int gather(const RouteArgs& a, int l, float least, const float (&key)[V], Candidates& c) {
  uint32_t own = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) own += key[v] >= least && key[v] > none<float>();
  const uint32_t end = team_scan<L>(own);
  const int n = (int)team_reduce<L>(end, MaxU());
  uint32_t at = end - own;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (key[v] >= least && key[v] > none<float>()) {
      if (at < kCandidates) {
        c.key[at] = key[v];
        c.expert[at] = expert_of<L>(v, l);
      }
      ++at;
    }
  }
  if (l < 4 && n + l < kCandidates) {              // read four at a time
    c.key[n + l] = none<float>();
    c.expert[n + l] = a.E;
  }
  if (l < kMaxChosen) c.chosen[l] = -1;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  return n;
}

// Ranks the n candidates of the token by their fp32 keys and writes down the k first.
// CHECK: `near` tells that two keys are too close (equal ones among them: their order is
// left open).  Else ties go to the lowest expert.
template <int L, bool CHECK>
__device__ __forceinline__ void rank(const RouteArgs& a, int l, int n, Candidates& c, bool& near) {
  for (int base = 0; __any(base < n); base += L) {
    const int s = base + l;
    const bool mine = s < n;
    const float own = mine ? c.key[s] : none<float>();
    const int e = mine ? c.expert[s] : 0;
    const float close = margin_of(a, own);
    int ahead = 0, around = 0;
    for (int i = 0; i < n; i += 4) {
      const f32x4 other = *reinterpret_cast<const f32x4*>(c.key + i);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (CHECK) {
          ahead += other[u] > own;
          around += fabsf(other[u] - own) <= close;
        } else {
          ahead += other[u] > own || (other[u] == own && c.expert[i + u] < e);
        }
      }
    }
    if (CHECK) near |= mine && around > 1;
    if (mine && ahead < a.k) c.chosen[ahead] = e;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The same by their fp64 keys.
template <int L>
__device__ __forceinline__ void rank_exactly(const RouteArgs& a, int l, int n, Candidates& c, const ExactKey& key) {
  for (int i = l; i < n; i += L) c.exact[i] = key(c.expert[i]);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  for (int s = l; s < n; s += L) {
    const double own = c.exact[s];
    const int e = c.expert[s];
    int ahead = 0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) ahead += c.exact[i] > own || (c.exact[i] == own && c.expert[i] < e);
    if (ahead < a.k) c.chosen[ahead] = e;
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// Places of the pairs of one workgroup's tokens.  Every wave takes a run of 64-pair
// pieces; it counts its pairs by expert and ranks them from the counts of the waves
// before it.
struct Pieces {
  int n, first, end;   // pairs of the workgroup; the wave's pieces
};
__device__ __forceinline__ Pieces pieces_of(int n) {
  const int pieces = (n + 63) / 64, per_wave = (pieces + kWaves - 1) / kWaves;
  const int first = (int)(threadIdx.x >> 6) * per_wave;
  return {n, first, first + per_wave < pieces ? first + per_wave : pieces};
}

// The expert of the lane's pair in piece p (-1: none), from memory.
template <typename Ids>
__device__ __forceinline__ int pair_of(const Pieces& w, int p, Ids ids) {
  const int i = p * 64 + (threadIdx.x & 63);
  return p < w.end && i < w.n ? ids(i) : -1;
}

// The first kHeld pieces' experts are held in registers (given), the others read again.
constexpr int kHeld = 4;
template <typename Ids>
__device__ __forceinline__ void count_pairs(const Pieces& w, Ids ids, const int (&held)[kHeld], int* own) {
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (held[u] >= 0) atomicAdd(&own[held[u]], 1);
  for (int p = w.first + kHeld; p < w.end; ++p) {
    const int e = pair_of(w, p, ids);
    if (e >= 0) atomicAdd(&own[e], 1);
  }
}

// counts[wave][e]: from the number of pairs to the place of the first one; base[e]: the
// place of the workgroup's first pair of expert e.
__device__ __forceinline__ void start_places(int E, int base, int* counts) {
  if ((int)threadIdx.x < E) {
    int c[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) c[w] = counts[w * E + threadIdx.x];
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      counts[w * E + threadIdx.x] = base;
      base += c[w];
    }
  }
  __syncthreads();
}

template <typename Ids>
__device__ __forceinline__ void place_pairs(const Pieces& w, Ids ids, const int (&held)[kHeld], int E, int* own,
                                            int32_t* dst) {
  const int lane = threadIdx.x & 63;
  const int bits = 32 - __clz(E);                    // E itself marks a slot without an expert
  const auto piece = [&](int p, int id) {
    const int i = p * 64 + lane;
    const int e = id < 0 ? E : id;
    uint64_t same = ~uint64_t(0);
    for (int b = 0; b < bits; ++b) {
      const bool one = (e >> b) & 1;
      const uint64_t with = __ballot(one);
      same &= one ? with : ~with;
    }
    const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
    if (e < E) {
      const int at = own[e];
      dst[i] = at + before;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      if (before == 0) own[e] = at + __popcll(same);
    } else if (i < w.n) {
      dst[i] = -1;
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (w.first + u < w.end) piece(w.first + u, held[u]);
  for (int p = w.first + kHeld; p < w.end; ++p) piece(p, pair_of(w, p, ids));
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
  const int pass = a.threads / L;                  // tokens of one pass over the workgroup's waves
  extern __shared__ double dynamic_lds[];
  __shared__ int count[kMaxExperts];
  __shared__ int chosen[64 * kMaxChosen];
  __shared__ int wave_sums[kWaves];
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int tok = lane / L;
  const bool alone = a.alone;
  const bool plan = a.M_sizes && (alone || a.hist);   // else the second kernel counts
  if (plan) {
    for (int e = threadIdx.x; e < a.E; e += a.threads) count[e] = 0;
    if (alone) chosen[threadIdx.x] = -1;
    __syncthreads();
  }
  const int64_t first = (int64_t)blockIdx.x * a.block_tokens;
  for (int at = wave * (64 / L); at < a.block_tokens; at += pass) {
    if (first + at >= a.T) break;                  // uniform over the wave
    // Opaque to the compiler in each pass: it would keep what follows from the lane for
    // every v (expert, group, addresses) in registers across the passes, of which there
    // is seldom more than one.
    int l = lane % L;
    asm volatile("" : "+v"(l));
    const bool live = first + at + tok < a.T;
    const int64_t t = live ? first + at + tok : a.T - 1;
    float x[V];
    load_row<L, V>(a, t, l, x);
    char* own_lds = reinterpret_cast<char*>(dynamic_lds) + (wave * (64 / L) + tok) * a.token_lds;
    Candidates& list = *reinterpret_cast<Candidates*>(own_lds);
    float key[V];
    uint32_t kept = 0xFFFFu;
    if constexpr (ARITH) {
      make_keys<L, V>(a, l, x, key);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) key[v] = x[v];
    }
    if (a.n_group > 1) {
      kept = keep_groups<L, V, ARITH>(a, t, l, tok, reinterpret_cast<float*>(own_lds), key);
      if (ARITH && !a.bias) {                        // the experts themselves in order of their logits
#pragma unroll
        for (int v = 0; v < V; ++v) key[v] = x[v];
      }
      drop_groups<L, V>(a, l, kept, key);
    }
    const float bound = bound_of<L, V>(a.k, key);
    const bool sums = ARITH && a.bias;
    const int n = gather<L, V>(a, l, sums ? bound - margin_of(a, bound) : bound, key, list);
    const int listed = n < kCandidates ? n : kCandidates;
    bool near = false;
    if (sums) {
      rank<L, true>(a, l, listed, list, near);
      if (__any(near && n <= kCandidates)) rank_exactly<L>(a, l, listed, list, exact_key<L>(a, t, l, true));
    } else {
      rank<L, false>(a, l, listed, list, near);
    }
    int id = -1;
    if (l < a.k) id = list.chosen[l];
    if (__any(n > kCandidates)) {
      const int in_rounds = choose_in_rounds<L>(a, l, kept, exact_key<L>(a, t, l, sums));
      if (n > kCandidates) id = in_rounds;
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
      // In the order of a team of 64 lanes, whichever the team: the weights do not depend
      // on how many tokens a call has.
      constexpr int kRows = L == 16 && V >= 4 ? 4 : 1;
      float part[kRows] = {};
#pragma unroll
      for (int v = 0; v < V; ++v) part[v % kRows] += x[v] > none<float>() ? expf(x[v] - most) : 0.f;
      if constexpr (kRows == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) part[i] = row16_reduce(part[i], AddF());
        sum = (part[0] + part[1]) + (part[2] + part[3]);
      } else {
        sum = team_reduce<L>(part[0], AddF());
      }
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
    for (int e = threadIdx.x; e < a.E; e += a.threads) a.hist[(int64_t)blockIdx.x * count_row(a.E) + e] = count[e];
    return;
  }
  const int c = (int)threadIdx.x < a.E ? count[threadIdx.x] : 0;
  const int before = prefix_before(c, wave_sums);
  if ((int)threadIdx.x < a.E) a.M_sizes[threadIdx.x] = c;
  int* counts = reinterpret_cast<int*>(dynamic_lds);
  int* own = counts + wave * a.E;
  for (int i = threadIdx.x; i < kWaves * a.E; i += kThreads) counts[i] = 0;
  __syncthreads();
  const Pieces w = pieces_of((int)a.T * a.k);      // at most one per wave
  const auto ids = [&](int i) { return chosen[i]; };
  const int held[kHeld] = {pair_of(w, w.first, ids), -1, -1, -1};
  count_pairs(w, ids, held, own);
  __syncthreads();
  start_places(a.E, before, counts);
  place_pairs(w, ids, held, a.E, own, a.dst_row);
}

// Second kernel of the plan: each workgroup takes the pairs of `span` neighbouring blocks
// of the first one; it adds up the counts of all blocks and of those before its own,
// then places its pairs.  At most 64 workgroups, because each of them reads all counts
// (256 x 256 of them at 16384 tokens and 256 experts: one workgroup per block took 21 us).
// Up to kLonePairs pairs, what its registers hold, a single workgroup counts them all
// itself: many workgroups that read the same few lines of counts wait 3 to 5 us for them
// (route with plan, one workgroup against many: 6.4 and 10.7 us at 256 tokens, 8 experts,
// k = 2; 13.7 and 14.8 us at 256 tokens, 256 experts in groups, k = 8, with 16 lanes per
// token).  Fewer workgroups
// of more pairs beyond that are slower (1024 tokens, 256 experts: 16.9 us, and 19.3 with
// 4096 pairs each; 4096 tokens, 8 experts: 12.6 and 14.0).
constexpr int kPlaceGroups = 64;

// LDS of the second kernel: the waves' counts, and for each of the kThreads / width sets
// of lanes that read the first kernel's counts side by side their two sums.
__host__ __device__ inline int place_width(int E) {
  const int lanes = E % 4 == 0 ? E / 4 : E;
  int width = 64;
  while (width < lanes) width *= 2;
  return width;
}
inline size_t place_lds(int E) { return (size_t)(kWaves + 2 * (kThreads / place_width(E))) * E * sizeof(int); }

// Sums of the counts of all blocks and of those before `first_block`; four experts per
// lane where the rows allow 16-byte loads, sixteen loads in flight.
template <typename V>
__device__ __forceinline__ void add_counts(const V* hist, int row, int lanes, int width, int blocks, int first_block,
                                           V* sums) {
  const int lane = threadIdx.x % width, set = threadIdx.x / width, sets = kThreads / width;
  if (lane >= lanes) return;
  V all = {}, prior = {};
  for (int b = set; b < blocks; b += 16 * sets) {
    V c[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      c[i] = V{};
      if (b + i * sets < blocks) c[i] = hist[(int64_t)(b + i * sets) * row + lane];
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      all += c[i];
      if (b + i * sets < first_block) prior += c[i];
    }
  }
  sums[set * lanes + lane] = all;
  sums[(sets + set) * lanes + lane] = prior;
}

__global__ void __launch_bounds__(kThreads) place_kernel(RouteArgs a, int blocks, int span) {
  extern __shared__ double dynamic_lds[];
  __shared__ int wave_sums[kWaves];
  int* counts = reinterpret_cast<int*>(dynamic_lds);
  int* own = counts + (threadIdx.x >> 6) * a.E;
  int* sums = counts + kWaves * a.E;
  const int first_block = blockIdx.x * span;
  const int64_t first = (int64_t)first_block * a.block_tokens, most = (int64_t)span * a.block_tokens;
  const Pieces w = pieces_of((int)(a.T - first < most ? a.T - first : most) * a.k);
  const int32_t* block_ids = a.ids + first * a.k;
  const auto ids = [&](int i) { return block_ids[i]; };
  // The pairs are asked for first, so that counting them does not wait for the counts.
  int held[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u) held[u] = pair_of(w, w.first + u, ids);
  for (int i = threadIdx.x; i < kWaves * a.E; i += kThreads) counts[i] = 0;
  __syncthreads();
  const int width = place_width(a.E), sets = kThreads / width;
  count_pairs(w, ids, held, own);
  if (a.hist && a.E % 4 == 0)
    add_counts(reinterpret_cast<const u32x4*>(a.hist), count_row(a.E) / 4, a.E / 4, width, blocks, first_block,
               reinterpret_cast<u32x4*>(sums));
  else if (a.hist)
    add_counts(reinterpret_cast<const uint32_t*>(a.hist), count_row(a.E), a.E, width, blocks, first_block,
               reinterpret_cast<uint32_t*>(sums));
  __syncthreads();
  int total = 0, earlier = 0;
  if ((int)threadIdx.x < a.E) {
    if (a.hist) {
      for (int s = 0; s < sets; ++s) {
        total += sums[s * a.E + threadIdx.x];
        earlier += sums[(sets + s) * a.E + threadIdx.x];
      }
    } else {
      for (int x = 0; x < kWaves; ++x) total += counts[x * a.E + threadIdx.x];
    }
    if (blockIdx.x == 0) a.M_sizes[threadIdx.x] = total;
  }
  earlier += prefix_before(total, wave_sums);
  start_places(a.E, earlier, counts);
  place_pairs(w, ids, held, a.E, own, a.dst_row + first * a.k);
}

template <int L, int V, bool ARITH>
hipError_t launch(const RouteArgs& a, int blocks, hipStream_t stream) {
  // a token's candidates, and before them its keys by group, in the same place
  const int keys = a.n_group > 1 ? (2 * kMaxGroups + a.E + a.n_group) * (int)sizeof(float) : 0;
  RouteArgs b = a;
  b.token_lds = ((keys > (int)sizeof(Candidates) ? keys : (int)sizeof(Candidates)) + 15) / 16 * 16;
  const size_t tokens = (size_t)(a.threads / L) * b.token_lds;
  const size_t counts = a.alone ? (size_t)kWaves * a.E * sizeof(int) : 0;
  hipLaunchKernelGGL((route_kernel<L, V, ARITH>), dim3(blocks), dim3(a.threads), tokens > counts ? tokens : counts, stream,
                     b);
  return hipGetLastError();
}

template <bool ARITH>
hipError_t launch_by_width(const RouteArgs& a, bool wide, int blocks, hipStream_t stream) {
  if (wide) {
    if (a.E <= 128) return launch<64, 2, ARITH>(a, blocks, stream);
    if (a.E <= 256) return launch<64, 4, ARITH>(a, blocks, stream);
    if (a.E <= 512) return launch<64, 8, ARITH>(a, blocks, stream);
    return launch<64, 16, ARITH>(a, blocks, stream);
  }
  if (a.E <= 16) return launch<16, 1, ARITH>(a, blocks, stream);
  if (a.E <= 32) return launch<16, 2, ARITH>(a, blocks, stream);
  if (a.E <= 64) return launch<16, 4, ARITH>(a, blocks, stream);
  if (a.E <= 128) return launch<16, 8, ARITH>(a, blocks, stream);
  if (a.E <= 256) return launch<16, 16, ARITH>(a, blocks, stream);
  return launch<16, 32, ARITH>(a, blocks, stream);
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

// How the tokens are shared out.  16 lanes per token take the fewest instructions; 64 lanes
// have the shorter chain of them and are the faster ones until the SIMDs are full.  Graph of
// calls with 256 experts in 8 groups, k = 8, sigmoid and bias, us, against 16 lanes and 16
// (up to 64 tokens: all) tokens per workgroup:
//   1 token         one launch, 64 lanes          8.1 against 10.3
//   8               one launch, 64 lanes          9.1 against 9.5 in two launches
//   16 to 512       4 tokens per workgroup of 256 threads, then one workgroup that counts:
//                   16: 9.8 against 11.0; 64: 9.9 and 15.0; 200: 10.9 and 13.8
//   1024 (4096)     16 tokens of 64 lanes per workgroup: 15.5 (17.6) against 16.6 (21.8)
//   16384           16 lanes: 24.6, and 40.2 with 64
// 344 experts: 16 tokens 11.2 against 19.4.  One launch while T E is small: 128 experts,
// sigmoid and bias, 64 tokens take 8.6 in one and 7.6 in two.  Up to 128 experts 16 lanes stay the better ones
// where counts are handed on (4096 tokens, 128 experts: 12.8 and 14.2 with 64), and up to 64
// experts everywhere.  Without a plan 4 tokens per workgroup up to 2048 (8.3 against 9.4).
//
// Tokens of one workgroup where there are counts to hand on, at most kMaxBlocks rows: each
// place workgroup reads all of them, so where the choice is quick half as many rows are
// better (4096 tokens, k = 2, 8 experts: 10.8 us with 32 tokens, 12.7 with 16; 128 experts,
// k = 8: 12.9 and 13.9; but 256 experts: 17.0 and 14.6).
static int counted_tokens(int64_t T, int64_t E) {
  if (T <= (E <= 128 ? 8 : 16) * kMaxBlocks) return 16;
  if (T <= 16 * kMaxBlocks) return 32;
  return (int)(64 * ((T + 64 * kMaxBlocks - 1) / (64 * kMaxBlocks)));
}

int64_t route_count_rows(int64_t T, int64_t E) {
  const int tokens = counted_tokens(T, E);
  return (T + tokens - 1) / tokens;
}

hipError_t launch_route(const RouteArgs& given, hipStream_t stream) {
  RouteArgs a = given;
  if (a.T == 0 && !a.M_sizes) return hipSuccess;
  a.alone = a.M_sizes && a.T <= 64 && a.T * a.E <= (a.E <= 128 ? 4096 : 2048);
  bool wide;
  if (a.alone) {
    a.block_tokens = 64;
    wide = a.E > 128;
    a.threads = kThreads;
  } else if (!a.hist && a.E > 64 && a.T <= 8 * kMaxBlocks) {
    a.block_tokens = 4;
    wide = true;
    a.threads = 256;
  } else {
    a.block_tokens = counted_tokens(a.T, a.E);
    wide = a.E > (a.block_tokens == 16 ? 128 : 512);
    if (wide || a.block_tokens > 32) a.threads = kThreads;
    else a.threads = 16 * a.block_tokens;
  }
  // T == 0 with a plan: one workgroup writes zero counts
  const int blocks = a.T == 0 ? 1 : (int)((a.T + a.block_tokens - 1) / a.block_tokens);
  const bool arith = a.bias || (a.n_group > 1 && a.group_top == 2);
  hipError_t e = arith ? launch_by_width<true>(a, wide, blocks, stream)
                       : launch_by_width<false>(a, wide, blocks, stream);
  if (e != hipSuccess || !a.M_sizes || a.alone) return e;
  const int span = a.hist ? (blocks + kPlaceGroups - 1) / kPlaceGroups : blocks;
  hipLaunchKernelGGL(place_kernel, dim3((blocks + span - 1) / span), dim3(kThreads), place_lds(a.E), stream, a,
                     blocks, span);
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteBackwardArgs& a, hipStream_t stream) {
  if (a.T == 0) return hipSuccess;
  const int64_t want = (a.T + 3) / 4;
  hipLaunchKernelGGL(route_backward_kernel, dim3((uint32_t)(want < 8192 ? want : 8192)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8gg
