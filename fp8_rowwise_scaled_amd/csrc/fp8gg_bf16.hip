// Products of bf16 matrices by group for gfx950: the forward product of the experts, the gradient
// of its input and that of its weights.
//
//     Y[m, n]  = sum_k X[m, k] W[g, n, k]        both operands run along the contraction
//     dX[m, k] = sum_n dY[m, n] W[g, n, k]       W runs across it
//     dW[g, n, k] = sum_m dY[m, n] X[m, k]       both run across it, over the rows of a group
//
// One tile serves all three: an operand that runs along the contraction is read from LDS sixteen
// bytes a lane, one that runs across it with the transposing read (ds_read_b64_tr_b16), so no
// transposed copy of anything is made.  v_mfma_f32_16x16x32_bf16 with the output's columns as its rows,
// fp32 accumulators; tiles go global -> LDS without registers.
//
// What bounds it: on data as it comes the card's power.  A product of 4096 x 4096 x 7168 in one group takes
// 129 us on zeros and 168 on normal values (a library's product 110 and 151; each alone, in a captured graph;
// in turn with others 141 and 176 against 118 and 158), so what moves fewer bits counts as much as what waits
// less.  Steps on the way, each timed against the one before: 16 x 16 x 32 instead of 32 x 32 x 16
// instructions, which write half the sums per product, 198 -> 176 us; copies addressed by a scalar base and a
// fixed offset per lane (no vector arithmetic in the loop), 169 -> 164; neighbouring instructions that share an
// operand, 164 -> 163.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8gg_lds.h"
#include "fp8gg_layer_internal.h"
#include "fp8gg_train_internal.h"

namespace fp8gg {

namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

// ---------------------------------------------------------------------------
// Groups: rows of each, from the counts on the device
// ---------------------------------------------------------------------------

struct SatAdd {
  uint32_t cap;
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return umin(a + b, cap); }
};
struct AddU {
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return a + b; }
};

__device__ __forceinline__ uint32_t lane_value(uint32_t x, int lane) {
  return (uint32_t)__builtin_amdgcn_readlane((int)x, lane);
}

// Rows [start, end) of the 64 groups from g0 on, one per lane; `rows`: the rows before them.
__device__ __forceinline__ void group_rows(const ProductArgs& a, int g0, uint32_t rows, uint32_t& start, uint32_t& end) {
  const int lane = threadIdx.x & 63;
  const int64_t n = g0 + lane < a.G ? a.M_sizes[g0 + lane] : 0;
  const uint32_t M = (uint32_t)a.M;
  const uint32_t c = n <= 0 ? 0u : n >= a.M ? M : (uint32_t)n;
  end = umin(wave_scan(c, SatAdd{M}) + rows, M);
  const uint32_t before = (uint32_t)__shfl_up((int)end, 1, 64);
  start = lane ? before : rows;
}

// The stores' cache policy: written once, past the caches.
constexpr int kPastCaches = 2;

struct RowTile {
  int g;
  int64_t row0, row_end;
};

// Tiles of BM rows over all groups: first those with more than BM / 2 rows, then the others (at
// most one per group).
struct RowTiles {
  uint32_t tall, all;
  uint32_t start, end;           // the first 64 groups' rows, one group per lane
};

template <int BM>
__device__ __forceinline__ RowTiles count_row_tiles(const ProductArgs& a) {
  uint32_t rows = 0;
  RowTiles n = {0, 0, 0, 0};
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    uint32_t start, end;
    group_rows(a, g0, rows, start, end);
    if (g0 == 0) n.start = start, n.end = end;
    n.tall += lane_value(wave_scan((end - start + BM / 2 - 1) / BM, AddU{}), 63);
    n.all += lane_value(wave_scan((end - start + BM - 1) / BM, AddU{}), 63);
    rows = lane_value(end, 63);
  }
  return n;
}

template <int BM>
__device__ __forceinline__ RowTile find_row_tile(const ProductArgs& a, const RowTiles& n, uint32_t tile) {
  const bool tall = tile < n.tall;
  tile -= tall ? 0 : n.tall;
  uint32_t rows = 0, tiles = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    uint32_t start = n.start, end = n.end;
    if (g0 > 0) group_rows(a, g0, rows, start, end);
    const uint32_t high = (end - start + BM / 2 - 1) / BM;
    const uint32_t mine = tall ? high : (end - start + BM - 1) / BM - high;
    const uint32_t upto = tiles + wave_scan(mine, AddU{});
    const uint64_t hit = __ballot(tile < upto);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const uint32_t nth = tile - lane_value(upto - mine, l) + (tall ? 0 : lane_value(high, l));
      return {g0 + l, lane_value(start, l) + (int64_t)nth * BM, (int64_t)lane_value(end, l)};
    }
    tiles = lane_value(upto, 63);
    rows = lane_value(end, 63);
  }
  return {0, 0, 0};
}

// xcd_slot in 32 bits (the launcher's bound on the tiles).
__device__ __forceinline__ uint32_t xcd_slot32(uint32_t w, uint32_t P) {
  const uint32_t x = w % 8, q = P / 8, r = P % 8;
  return x * q + (x < r ? x : r) + w / 8;
}

// Tiles of a rows x cols grid in strips of four rows, column by column: the 32 tiles that an XCD works on
// at a time are four rows by eight columns (12 panels of the operands to read), not one row or two
// (18 to 30).  Input's gradient of 4096 rows in 8 even groups, N = 4096, K = 7168: 225 us in strips of one row, 218 of four.
__device__ __forceinline__ void in_strips(uint32_t tile, uint32_t rows, uint32_t cols, uint32_t& row, uint32_t& col) {
  constexpr uint32_t H = 4;
  const uint32_t strip = tile / (H * cols), at = tile - strip * H * cols, left = rows - strip * H, h = left < H ? left : H;
  col = __builtin_amdgcn_readfirstlane(at / h);
  row = __builtin_amdgcn_readfirstlane(strip * H + at - col * h);
}

// The row and column of a tile over all groups: the tall row tiles' first, so that a persistent grid
// meets its cheap tiles last.
__device__ __forceinline__ void tile_place(const RowTiles& n, uint32_t cols, uint32_t tile, uint32_t& row, uint32_t& col) {
  const uint32_t tall = n.tall * cols;
  if (tile < tall) {
    in_strips(tile, n.tall, cols, row, col);
  } else {
    in_strips(tile - tall, n.all - n.tall, cols, row, col);
    row += n.tall;
  }
}

// ---------------------------------------------------------------------------
// One output tile
// ---------------------------------------------------------------------------

// A pointer that all lanes hold alike, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t u = (uint64_t)p;
  return (const uint8_t*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u) |
                          (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32);
}

// An operand of the tile in LDS: R rows (or columns) of the output by BK of the contraction.
// ALONG: the contraction runs along memory; LDS rows are BK values, read 16 bytes a lane.
// Else it runs across memory; LDS rows are the R values of one place in the contraction, and the
// matrix instruction's operand is read transposed (ds_read_b64_tr_b16: sixteen lanes read four
// places of sixteen values, lane i gets value i of the four).
template <int R, int BK, int NT, bool ALONG>
struct Operand {
  static constexpr int CHUNKS = R * BK / 8;
  static constexpr int LOADS = CHUNKS / NT;
  static constexpr int BYTES = R * BK * 2;
  static constexpr int CPR = (ALONG ? BK : R) / 8;
  static_assert(CHUNKS % NT == 0, "every thread copies as much");
  int tid;                       // thread of the tile
  const uint8_t* base;           // of the tile's part of the operand, the same in all lanes
  uint32_t off[LOADS];           // this lane's chunks from there, in bytes

  // 16-byte chunk c of LDS row `row` lies at c ^ swz(row): sixteen lanes meet no bank twice in either kind of
  // read (across: the four places that they read lie in four different 64-byte columns.  Others read with them
  // may meet theirs: the counter of bank conflicts has 1% of the cycles of LDS in kernels that read along, 30 to 46% where
  // an operand is read across).
  static __device__ __forceinline__ int swz(int row) {
    if constexpr (ALONG) return lds_swz<BK * 2>(row);
    else if constexpr (R >= 128) return (row & 3) << 2;
    else if constexpr (R == 64) return ((row >> 1) & 1) << 2;
    else return 0;
  }

  // The contraction starts at `from`; rows (columns) [first, first + count) of the matrix exist, the
  // tile's other ones repeat the last and their results are dropped.  Offsets stay below 2^32: ld is at
  // most 2^22, rows of the tile 256.
  __device__ __forceinline__ void setup(int thread, const uint16_t* from, int64_t ld, int64_t first, int64_t count) {
    tid = thread;
    base = (const uint8_t*)(from + (ALONG ? first * ld : first));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int q = i * NT + tid;
      const int row = q / CPR;
      const int c = (q % CPR) ^ swz(row);
      int64_t r = ALONG ? row : c * 8;
      if (r >= count) r = ALONG ? count - 1 : count - 8;
      off[i] = (uint32_t)((ALONG ? r * ld + c * 8 : row * ld + r) * 2);
    }
  }

  // Copy i of contraction [k, k + BK) of n, WHOLE if that ends within n; else zeros from n on (for both
  // operands, so that nothing that lies there, a NaN included, reaches a sum).
  template <bool WHOLE>
  __device__ __forceinline__ void issue(int i, uint8_t* lds, int64_t k, int64_t n, int64_t ld) const {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint8_t* s = base + (ALONG ? k : k * ld) * 2;
    const uint32_t to = lds_addr(lds + (i * NT + wave * 64) * 16);
    if constexpr (WHOLE) {
      copy16_to_lds(uniform(s), off[i], to);
    } else {
      const int q = i * NT + tid, row = q / CPR, at = ALONG ? (q % CPR ^ swz(row)) * 8 : row;
      copy16_to_lds(k + at < n ? s + off[i] : g_zero16, to);
    }
  }

  // The instruction's operand: block b of 16, step ks of 32 along the contraction.
  __device__ __forceinline__ v8bf frag(const uint8_t* lds, int b, int ks) const {
    const int r = tid & 15, q = (tid & 63) >> 4;
    if constexpr (ALONG) {
      const int row = 16 * b + r;
      return *(const v8bf*)(lds + row * (BK * 2) + (((4 * ks + q) ^ swz(row)) * 16));
    } else {
      const int piece = 4 * b + (r & 3);                 // four neighbouring values
      const int k = 32 * ks + 8 * q + (r >> 2);
      const uint8_t* p = lds + k * (R * 2) + ((piece >> 1) ^ swz(k)) * 16 + (piece & 1) * 8;
      const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p));
      const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * R * 2));
      return __builtin_bit_cast(v8bf, (v8s)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }
};

// A BM x BN tile of the output by WM x WN waves.  P: the operand of the output's rows, in a ring of
// SP slots of LDS; Q: of its columns, in SQ slots.
template <bool P_ALONG, bool Q_ALONG, int BM, int BN, int BK, int WM, int WN, int SP, int SQ>
struct ProductTile {
  static constexpr int NT = WM * WN * 64;
  static constexpr int FM = BM / WM / 16, FN = BN / WN / 16, KS = BK / 32;
  typedef Operand<BM, BK, NT, P_ALONG> P;
  typedef Operand<BN, BK, NT, Q_ALONG> Q;
  static constexpr int SMEM = SP * P::BYTES + SQ * Q::BYTES;
  static_assert(SP >= 2 && (SQ == SP || (SP == 2 && SQ == 3)), "the wait counts below");
  static_assert(KS % 2 == 0, "operands alternate between two sets of registers");
  typedef v4f Acc[FM][FN];   // lane (q, r) = (lane / 16, lane % 16): row r, columns 4 q .. 4 q + 3 of a block

  uint8_t* smem;
  P p;
  Q q;

  // This thread's number in the tile, opaque: what follows from it is worked out for each tile, where a
  // persistent kernel would else keep it in registers that the loop has no room for.
  static __device__ __forceinline__ int thread() {
    int tid = threadIdx.x % NT;
    asm volatile("" : "+v"(tid));
    __builtin_assume(tid >= 0 && tid < NT);
    return tid;
  }

  __device__ __forceinline__ uint8_t* pslot(int i) const { return smem + i * P::BYTES; }
  __device__ __forceinline__ uint8_t* qslot(int i) const { return smem + SP * P::BYTES + i * Q::BYTES; }
  __device__ __forceinline__ int wave_id() const { return __builtin_amdgcn_readfirstlane(p.tid >> 6); }
  // A single wave orders its own copies and reads by its waits.
  static __device__ __forceinline__ void barrier() {
    if constexpr (NT > 64) block_barrier();
    else asm volatile("" ::: "memory");
  }
  static __device__ __forceinline__ void publish() {
    if constexpr (NT > 64) publish_barrier();
    else asm volatile("" ::: "memory");
  }

  // Where stage s of nk lies in the contraction of n: from stage `start` on, and round; past the last, n.
  // start > 0: n % BK == 0.
  template <bool WHOLE = false>
  static __device__ __forceinline__ int64_t from(int s, int nk, int start, int64_t n) {
    if (!WHOLE && s >= nk) return n;
    const int at = s + start;
    return (int64_t)(at < nk ? at : at - nk) * BK;
  }

  // Copies of the first stages of a contraction of n: all that the loop starts with, or in two parts, HEAD (all
  // of P's, Q's first) and REST.  No wave reads their slots any more.
  enum Part { ALL, HEAD, REST };
  template <Part PART = ALL>
  __device__ __forceinline__ void prologue(int64_t n, int64_t ldp, int64_t ldq, int start = 0) const {
    if (n <= 0) return;
    const int nk = (int)((n + BK - 1) / BK);
    constexpr int Q0 = PART == REST ? 1 : 0, Q1 = PART == HEAD ? 1 : SQ - 1;
#pragma unroll
    for (int s = 0; s < (SP > SQ - 1 ? SP : SQ - 1); ++s) {
#pragma unroll
      for (int i = 0; PART != REST && s < SP && i < P::LOADS; ++i) p.template issue<false>(i, pslot(s), from(s, nk, start, n), n, ldp);
#pragma unroll
      for (int i = 0; s >= Q0 && s < Q1 && i < Q::LOADS; ++i) q.template issue<false>(i, qslot(s), from(s, nk, start, n), n, ldq);
    }
  }

  // acc += the products over a contraction of n, after its prologue.  YOUNGER: only its HEAD is under way, and
  // behind it, if `younger`, so many stores of each wave, which read from the slots of the REST.
  template <int YOUNGER = 0>
  __device__ __forceinline__ void loop(int64_t n, int64_t ldp, int64_t ldq, bool younger, Acc& acc, int start = 0) const {
    constexpr bool HEADED = YOUNGER > 0;
    const int wm = wave_id() / WN, wn = wave_id() % WN;
    const int nk = (int)((n + BK - 1) / BK);
    asm volatile("" ::: "memory");               // whatever came before is issued before the waits below
    if (nk == 0) {
      barrier();                                 // the waves part here as after the loop
      return;
    }
    constexpr int FIRST = (SP - 1) * P::LOADS + (HEADED ? 0 : (SQ - 2) * Q::LOADS);
    constexpr int NEXT = SP == SQ ? (SP - 2) * (P::LOADS + Q::LOADS) : Q::LOADS;
    static_assert(!HEADED || (SP == 2 && SQ == 3), "HEAD: P's two stages and Q's first");
    if (younger) wait_vmcnt_le(FIRST + YOUNGER);
    else wait_vmcnt_le(FIRST);
    barrier();
    if constexpr (HEADED) prologue<REST>(n, ldp, ldq, start);
    v8bf pf[2][FM], qf[2][FN];
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) pf[0][fm] = p.frag(pslot(0), wm * FM + fm, 0);
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) qf[0][fn] = q.frag(qslot(0), wn * FN + fn, 0);
    constexpr int NM = FM * FN, NR = FM + FN;    // instructions and operands of a step
    constexpr int QS = KS - 1 < 2 ? KS - 1 : 2;  // steps over which Q's copies are spread
    int sp = 0, sq = 0;
    const auto stage = [&](int kt, auto whole) __attribute__((always_inline)) {
      constexpr bool WHOLE = decltype(whole)::value;
      const int np = sp == SP - 1 ? 0 : sp + 1, nq = sq == SQ - 1 ? 0 : sq + 1, bq = sq == 0 ? SQ - 1 : sq - 1;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const int c = ks & 1, d = c ^ 1;
        const bool last = ks == KS - 1;
        if (last) {
          // this wave has read its last operands of stage kt, and stage kt + 1 has landed once only
          // the younger copies are outstanding; the barrier says so of all waves
          __builtin_amdgcn_s_waitcnt(0xC07F);    // lgkmcnt 0
          wait_vmcnt_le(NEXT);
          barrier();
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const int fm = i / FN, fn = fm & 1 ? FN - 1 - i % FN : i % FN;
          acc[fm][fn] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(qf[c][fn], pf[c][fm], acc[fm][fn], 0, 0, 0);
          // the next step's operands (of the next stage in the last step; past the end they are read
          // from the ring all the same and not used)
#pragma unroll
          for (int r = i * NR / NM; r < (i + 1) * NR / NM; ++r) {
            const int rk = last ? 0 : ks + 1;
            if (r < FN) qf[d][r] = q.frag(qslot(last ? nq : sq), wn * FN + r, rk);
            else pf[d][r - FN] = p.frag(pslot(last ? np : sp), wm * FM + r - FN, rk);
          }
          // P's copies into the slot that the last step has freed, Q's in the first steps after it
          if (last) {
#pragma unroll
            for (int r = i * P::LOADS / NM; r < (i + 1) * P::LOADS / NM; ++r)
              p.template issue<WHOLE>(r, pslot(sp), from<WHOLE>(kt + SP, nk, start, n), n, ldp);
          } else if (ks < QS) {
#pragma unroll
            for (int r = (ks * NM + i) * Q::LOADS / (QS * NM); r < (ks * NM + i + 1) * Q::LOADS / (QS * NM); ++r)
              q.template issue<WHOLE>(r, qslot(bq), from<WHOLE>(kt + SQ - 1, nk, start, n), n, ldq);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      sp = np;
      sq = nq;
    };
    // the copies that a stage issues are of whole stages while they lie before n
    const int full = (int)(n / BK) - (SP > SQ - 1 ? SP : SQ - 1);
    int kt = 0;
    for (; kt < full; ++kt) stage(kt, std::true_type{});
    for (; kt < nk; ++kt) stage(kt, std::false_type{});
    // No copy is in flight, of any wave's, when the ring is used again.  (Past the end a wave may still be
    // reading operands that nothing uses.)
    wait_vmcnt_le(0);
    barrier();
  }

  __device__ __forceinline__ void run(int64_t n, int64_t ldp, int64_t ldq, Acc& acc, int start = 0) const {
    prologue(n, ldp, ldq, start);
    loop(n, ldp, ldq, false, acc, start);
  }

  // Rows [row0, row_end) and columns [col0, cols) of a bf16 output, rounded to nearest even from the fp32
  // sums, through the idle ring, so that every store covers whole rows of the tile.
  __device__ __forceinline__ void store(uint16_t* out, int64_t ldo, int64_t row0, int64_t row_end, int64_t col0, int64_t cols,
                                        const Acc& acc) const {
    constexpr int CPR = BN / 8, MASK = (CPR < 16 ? CPR : 16) - 1;
    static_assert(BM * BN * 2 <= SMEM, "the tile fits the ring");
    const int tid = p.tid, r16 = tid & 15, q4 = (tid & 63) >> 4;
    const int wm = wave_id() / WN, wn = wave_id() % WN;
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int r = (wm * FM + fm) * 16 + r16;
#pragma unroll
      for (int fn = 0; fn < FN; ++fn) {
        const v4f& x = acc[fm][fn];
        const int col = (wn * FN + fn) * 16 + 4 * q4;
        *(v2i*)(smem + (r * CPR + (col / 8 ^ (r & MASK))) * 16 + col % 8 * 2) =
            v2i{(int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3])};
      }
    }
    publish();
#pragma unroll 4
    for (int i = tid; i < BM * CPR; i += NT) {
      const int r = i / CPR, c = i % CPR;
      if (row0 + r < row_end && col0 + 8 * c < cols)
        store_out((v4i*)(out + (row0 + r) * ldo + col0 + 8 * c), *(const v4i*)(smem + (r * CPR + (c ^ (r & MASK))) * 16));
    }
    barrier();                                   // the ring is free again
  }

  // The same while the HEAD of the next tile's prologue is under way, through the rest of the ring (Q's last two
  // slots), as many rows at a time as that holds.  Whole rows count: each wave by itself, without barriers but
  // 256 bytes of a row at a time, takes 357 us instead of 342 for the gate and up weights' gradient.  F32: the output's type, else
  // bf16.  What lies outside is sent past the buffer's end, which drops it, so that every wave issues the same
  // number of stores, STORES.
  template <bool F32>
  static constexpr int PASSES = BM * BN * (F32 ? 4 : 2) / (2 * Q::BYTES);
  template <bool F32>
  static constexpr int STORES = BM * BN * (F32 ? 4 : 2) / 16 / NT;
  template <bool F32>
  __device__ __forceinline__ void store_behind(void* out, int64_t ldo, int64_t row0, int64_t row_end, int64_t col0, int64_t cols,
                                               bool accumulate, const Acc& acc) const {
    constexpr int SIZE = F32 ? 4 : 2, PER = 16 / SIZE;   // values of a 16-byte chunk
    constexpr int CPR = BN / PER, MASK = (CPR < 16 ? CPR : 16) - 1;
    constexpr int ROWS = BM / PASSES<F32>, FP = FM / PASSES<F32>, PART = ROWS * CPR / NT;
    static_assert(FM % PASSES<F32> == 0 && ROWS * CPR % NT == 0, "whole blocks a pass, as much for every thread");
    constexpr uint32_t kEnd = 0xFFFFFFF0u;       // past every offset within 256 rows of 2^22 values
    uint8_t* const lds = qslot(SQ - 2);
    const int tid = p.tid, r16 = tid & 15, q4 = (tid & 63) >> 4;
    const int wm = wave_id() / WN, wn = wave_id() % WN;
    const auto rsrc = __builtin_amdgcn_make_buffer_rsrc((uint8_t*)out + (row0 * ldo + col0) * SIZE, 0, kEnd, 0x00020000);
    const int64_t rows_left = row_end - row0, cols_left = cols - col0;
#pragma unroll
    for (int ps = 0; ps < PASSES<F32>; ++ps) {
      if (ps > 0) barrier();
#pragma unroll
      for (int f = 0; f < FP; ++f) {
        const int r = (wm * FP + f) * 16 + r16;
#pragma unroll
        for (int fn = 0; fn < FN; ++fn) {
          const v4f& x = acc[ps * FP + f][fn];
          const int col = (wn * FN + fn) * 16 + 4 * q4;
          uint8_t* to = lds + (r * CPR + (col / PER ^ (r & MASK))) * 16;
          if constexpr (F32) *(v4f*)to = x;
          else *(v2i*)(to + col % PER * 2) = v2i{(int)pack_bf16x2(x[0], x[1]), (int)pack_bf16x2(x[2], x[3])};
        }
      }
      publish();
#pragma unroll
      for (int i = 0; i < PART; ++i) {
        const int at = i * NT + tid, r = at / CPR, c = at % CPR;
        const int row = r / (16 * FP) * (16 * FM) + ps * FP * 16 + r % (16 * FP), col = PER * c;
        const uint32_t off = row < rows_left && col < cols_left ? (uint32_t)((row * ldo + col) * SIZE) : kEnd;
        u32x4 v = *(const u32x4*)(lds + (r * CPR + (c ^ (r & MASK))) * 16);
        if constexpr (F32)
          if (accumulate)
            v = __builtin_bit_cast(u32x4, __builtin_bit_cast(v4f, v) +
                                              __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0)));
        __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, off, 0, kPastCaches);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Forward and the input's gradient: the output's rows are grouped
// ---------------------------------------------------------------------------

template <typename E, bool Q_ALONG>
__device__ __forceinline__ void product_tile(const ProductArgs& a, uint8_t* smem, const RowTile& t, int64_t col0, int start = 0) {
  E e;
  e.smem = smem;
  const int tid = E::thread();
  e.p.setup(tid, a.P, a.L, t.row0, t.row_end - t.row0);
  const int64_t ldq = Q_ALONG ? a.L : a.C;
  e.q.setup(tid, a.Q + t.g * a.L * a.C, ldq, col0, a.C - col0);
  typename E::Acc acc = {};
  e.run(a.L, a.L, ldq, acc, start);
  e.store((uint16_t*)a.out, a.C, t.row0, t.row_end, col0, a.C, acc);
}

// One workgroup per compute unit: rounds of whole tiles, and the tiles that do not fill one as halves or
// quarters where the rounds of these take less.  The matrix units under the power limit are the bound:
// 4096 rows in 8 groups from 0 to 1400, N = 4096, K = 7168, forward 252 us (950 TFLOP/s; 52% of the cycles of
// the matrix units busy, the rest mostly rows that tiles of 256 have and groups do not, and the last round), input's gradient 245; in 8 even groups 194 and 212;
// in one group 168 to 184 (1310 to 1430 TFLOP/s; a library's product in turn 151 to 164).
template <bool Q_ALONG>
__global__ void __launch_bounds__(512, 2) product_persistent_kernel(ProductArgs a) {
  constexpr int BM = 256, BN = 256;
  typedef ProductTile<true, Q_ALONG, BM, BN, 64, 2, 4, 2, 3> E;
  typedef ProductTile<true, Q_ALONG, BM / 2, BN, 64, 2, 4, 2, 3> Half;
  typedef ProductTile<true, Q_ALONG, BM / 2, BN / 2, 64, 2, 4, 5, 5> Quarter;
  static_assert(Half::SMEM <= E::SMEM && Quarter::SMEM <= E::SMEM, "parts share the ring");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[E::SMEM];
  const uint32_t P = gridDim.x, w = xcd_slot32(blockIdx.x, P);
  const RowTiles n = count_row_tiles<BM>(a);
  const uint32_t T = n.all * a.col_tiles, tall = n.tall * a.col_tiles;
  // Rounds of whole tiles: as many as the tall ones fill, as all fill, or all.  Of the tiles behind them the tall
  // ones have two halves, the others one.  A round of halves counts as 0.6 of one of whole tiles, of quarters as 0.4
  // (4096 rows in one group, N = 2048, K = 4096, whose 128 tiles fill half a round: 100 us whole, 68 to 70 as halves,
  // 83 as two rounds of quarters; 4096 rows in 8 groups from 0 to 1400, N = 4096, K = 7168: 335, 292, 258 forward and
  // 300, 256, 262 for the input's gradient).
  uint32_t whole = T, rest = 0, halves = 0, parts = 1, least = (T + P - 1) / P * 10;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const uint32_t full = (c ? T : tall) / P, at = full * P, r = tall > at ? tall - at : 0, h = T - at + r;
    const uint32_t by_half = (h + P - 1) / P * 6, by_quarter = (2 * h + P - 1) / P * 4;
    const uint32_t cost = full * 10 + (by_half < by_quarter ? by_half : by_quarter);
    if (cost < least) least = cost, whole = at, rest = r, halves = h, parts = by_quarter < by_half ? 2 : 1;
  }
  uint32_t row, col;
  for (uint32_t tile = w; tile < whole; tile += P) {
    tile_place(n, a.col_tiles, tile, row, col);
    product_tile<E, Q_ALONG>(a, smem, find_row_tile<BM>(a, n, row), (int64_t)col * BN);
  }
  for (uint32_t i = w; i < halves * parts; i += P) {
    const uint32_t half = i / parts;
    const bool in_tall = half < 2 * rest;
    tile_place(n, a.col_tiles, whole + (in_tall ? half / 2 : half - rest), row, col);
    RowTile t = find_row_tile<BM>(a, n, row);
    t.row0 += in_tall ? half % 2 * (BM / 2) : 0;
    const int64_t col0 = (int64_t)col * BN + i % parts * (BN / 2);
    if (parts == 1) product_tile<Half, Q_ALONG>(a, smem, t, col0);
    else if (col0 < a.C) product_tile<Quarter, Q_ALONG>(a, smem, t, col0);
  }
}

// The same with tiles of half the rows, for groups whose weights' way from memory is the bound (1537 rows in 16
// uneven groups, N = 1000, K = 7184, input's gradient: 70 us, 3.7 TB/s; 1536 in 16, N = K = 4096: 130 us, 4.3 TB/s, in even
// groups 95, 5.9 TB/s): a tile's first
// copies are under way before the last tile's output is stored, and these stores while it is computed.  Forward, groups start at
// different places of the contraction: rows that lie a power of two apart and are read at the same place keep
// only some of the memory's channels busy.  Neighbouring groups, which are read at the same time, are five stages apart:
// with one stage, 128 bytes, most of their reads still meet; 3, 5 and 7 are alike, and an odd number gives the groups as many
// places as the contraction has (us for 0 / 1 / 3 / 5 / 7 stages, in a captured graph: 256 rows in 32 groups, N = K = 2048,
// 67 / 48 / 49 / 49 / 49; 1536 in 16, N = K = 4096, 127 / 107 / 95 / 95 / 94; 1536 in 16, N = 7168, K = 2048, 106 / 99 / 92 / 91 / 90;
// 1537 in 16, N = 1000, K = 7184, whose rows are not a power of two apart, 98 with any).  Different places for a group's own
// tiles gain less, as these share the rows of its input, and the input's gradient, whose reads run along the rows of W, nothing.
template <bool Q_ALONG>
__global__ void __launch_bounds__(512, 2) product_stream_kernel(ProductArgs a) {
  constexpr int BM = 128, BN = 256, BK = 64;
  typedef ProductTile<true, Q_ALONG, BM, BN, BK, 2, 4, 2, 3> E;
  typedef ProductTile<true, Q_ALONG, BM, BN / 2, BK, 2, 4, 5, 5> H;
  static_assert(H::SMEM >= E::SMEM, "both share the ring");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[H::SMEM];
  const uint32_t P = gridDim.x, w = xcd_slot32(blockIdx.x, P);
  const RowTiles n = count_row_tiles<BM>(a);
  const uint32_t T = n.all * a.col_tiles;
  uint32_t whole = T / P * P;
  if (2 * (T - whole) > P) whole = T;
  const int64_t ldq = Q_ALONG ? a.L : a.C;
  struct Item {
    RowTile rows;
    int64_t col0;
    int start;
  };
  const auto find = [&](uint32_t tile, Item& t) __attribute__((always_inline)) {
    uint32_t row, col;
    tile_place(n, a.col_tiles, tile, row, col);
    t.rows = find_row_tile<BM>(a, n, row);
    t.col0 = (int64_t)col * BN;
    t.start = Q_ALONG && a.L > 0 && a.L % BK == 0 ? (uint32_t)t.rows.g * 5u % (uint32_t)(a.L / BK) : 0;
  };
  E e;
  e.smem = smem;
  const auto place = [&](uint32_t tile, Item& t) __attribute__((always_inline)) {
    find(tile, t);
    const int tid = E::thread();
    e.p.setup(tid, a.P, a.L, t.rows.row0, t.rows.row_end - t.rows.row0);
    e.q.setup(tid, a.Q + t.rows.g * a.L * a.C, ldq, t.col0, a.C - t.col0);
    e.template prologue<E::HEAD>(a.L, a.L, ldq, t.start);
  };
  Item t;
  uint32_t tile = w;
  if (tile < whole) {
    place(tile, t);
    for (bool stored = false;; stored = true) {
      typename E::Acc acc = {};
      e.template loop<E::template STORES<false>>(a.L, a.L, ldq, stored, acc, t.start);
      const Item done = t;
      tile += P;
      if (tile < whole) place(tile, t);
      e.template store_behind<false>(a.out, a.C, done.rows.row0, done.rows.row_end, done.col0, a.C, false, acc);
      if (tile >= whole) break;
    }
    E::barrier();
  }
  for (uint32_t i = w; i < 2 * (T - whole); i += P) {
    find(whole + i / 2, t);
    const int64_t col0 = t.col0 + i % 2 * (BN / 2);
    if (col0 < a.C) product_tile<H, Q_ALONG>(a, smem, t.rows, col0, t.start);
  }
}

// Few tiles: latency is the bound, and the bytes that are under way at a time (one row, N = 7168, K = 2048, forward 8.1 us,
// of which 3 a launch's; 29 MB).  The W waves of a workgroup take a part of the contraction each, in rings of their own,
// and their sums are added in the order of the waves.
template <bool Q_ALONG, int BN, int BK, int W, int SLOTS>
__global__ void __launch_bounds__(W * 64) product_split_kernel(ProductArgs a) {
  constexpr int BM = 32, FM = 2, FN = BN / 16;
  typedef ProductTile<true, Q_ALONG, BM, BN, BK, 1, 1, SLOTS, SLOTS> E;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[W * E::SMEM];
  static_assert(BM * BN * 4 <= E::SMEM, "a wave's sums fit its ring");
  const RowTiles n = count_row_tiles<BM>(a);
  const uint32_t T = n.all * a.col_tiles;
  if (blockIdx.x >= T) return;
  uint32_t row_tile, col_tile;
  tile_place(n, a.col_tiles, xcd_slot32(blockIdx.x, T), row_tile, col_tile);
  const RowTile t = find_row_tile<BM>(a, n, row_tile);
  const int64_t col0 = (int64_t)col_tile * BN;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int64_t per = ((a.L + W - 1) / W + BK - 1) / BK * BK;
  const int64_t k0 = wave * per, k1 = k0 + per < a.L ? k0 + per : a.L;
  E e;
  e.smem = smem + wave * E::SMEM;
  const int64_t ldq = Q_ALONG ? a.L : a.C;
  typename E::Acc acc = {};
  if (k0 < k1) {
    const int tid = E::thread();
    e.p.setup(tid, a.P + k0, a.L, t.row0, t.row_end - t.row0);
    e.q.setup(tid, a.Q + t.g * a.L * a.C + (Q_ALONG ? k0 : k0 * a.C), ldq, col0, a.C - col0);
    e.run(k1 - k0, a.L, ldq, acc);
  }
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) *((v4f*)e.smem + (fm * FN + fn) * 64 + lane) = acc[fm][fn];
  __syncthreads();
  // a thread: eight neighbouring columns of one row
  for (int i = threadIdx.x; i < BM * BN / 8; i += W * 64) {
    const int r = i / (BN / 8), c = i % (BN / 8);
    const int64_t row = t.row0 + r, col = col0 + 8 * c;
    if (row >= t.row_end || col >= a.C) continue;
    const int from = (r / 16 * FN + c / 2) * 64 + c % 2 * 32 + r % 16;   // its first four columns; the others 16 lanes on
    v4f lo = {0.f, 0.f, 0.f, 0.f}, hi = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const v4f* s = (const v4f*)(smem + w * E::SMEM) + from;
      lo += s[0];
      hi += s[16];
    }
    store_out((v4i*)((uint16_t*)a.out + row * a.C + col),
              v4i{(int)pack_bf16x2(lo.x, lo.y), (int)pack_bf16x2(lo.z, lo.w), (int)pack_bf16x2(hi.x, hi.y),
                  (int)pack_bf16x2(hi.z, hi.w)});
  }
}

// ---------------------------------------------------------------------------
// The weights' gradient: the contraction runs over a group's rows
// ---------------------------------------------------------------------------

// The groups' rows, one group per lane, kept over a workgroup's tiles: up to 64 groups by size, the largest
// first, else the 64 from g0 on in their own order.
struct GroupTable {
  uint32_t g, first, count;      // of this lane's group
  int64_t g0;
  uint32_t rows;                 // before group g0

  __device__ __forceinline__ void load(const ProductArgs& a) {
    uint32_t end;
    group_rows(a, (int)g0, rows, first, end);
    g = (uint32_t)g0 + (threadIdx.x & 63);
    count = end - first;
  }
  __device__ __forceinline__ void start(const ProductArgs& a) {
    g0 = 0;
    rows = 0;
    load(a);
    if (a.G > 64) return;
    const int lane = threadIdx.x & 63;
    int rank = 0;
    for (int o = 0; o < 64; ++o) {
      const uint32_t other = lane_value(count, o);
      rank += other > count || (other == count && o < lane);
    }
    g = (uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)g);
    first = (uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)first);
    count = (uint32_t)__builtin_amdgcn_ds_permute(rank * 4, (int)count);
  }
  // The nth group; n never falls from one call to the next.
  __device__ __forceinline__ void nth(const ProductArgs& a, int64_t n, int64_t& group, int64_t& from, int64_t& many) {
    while (n >= g0 + 64) {
      rows = lane_value(first + count, 63);
      g0 += 64;
      load(a);
    }
    const int l = (int)(n - g0);
    group = lane_value(g, l);
    from = lane_value(first, l);
    many = lane_value(count, l);
  }
};

// One workgroup per compute unit.  Every XCD takes an eighth of each group's tiles (groups differ in size),
// the groups one after the other, the largest first.  A tile's first copies are under way before the last
// tile's sums are stored, and these stores while it is computed: 6143 rows in 64 groups, N = 1024, K = 1536, bf16
// 60 us against 75 with a workgroup per tile (201 MB out; 46 us at a copy's rate).  8 groups of 4096 rows in all,
// N = 4096, K = 7168, fp32 343 to 350 us: the stores alone take 185 (940 MB), the products alone 189, and a wave waits
// for its stores before the copies behind them, which the counter of both reports in order.  Added to what dW holds:
// 565 us (1.97 GB, 390 at a copy's rate), as each old value is waited for behind the stores before it.
// a.splits > 1: the group's rows in so many parts, each part's sums to a.partial.
template <bool F32>
__global__ void __launch_bounds__(512, 2) wgrad_kernel(ProductArgs a) {
  constexpr int BM = 256, BN = 256, BK = 64;
  typedef ProductTile<false, false, BM, BN, BK, 2, 4, 2, 3> E;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[E::SMEM];
  const uint32_t per = a.row_tiles * a.col_tiles * a.splits, share = (per + 7) / 8;
  const uint32_t x = blockIdx.x % 8, step = gridDim.x / 8;
  // An eighth of a group's tiles, neighbours, is the XCD's; where a group has too few for even eighths, every
  // eighth of all tiles is.
  const bool eighths = per >= 64;
  const uint32_t mine = !eighths ? per : per > x * share ? (per - x * share < share ? per - x * share : share) : 0;
  const uint64_t items = eighths ? (uint64_t)mine * a.G : ((uint64_t)per * a.G + 7 - x) / 8;
  GroupTable groups;
  groups.start(a);
  struct Item {
    int64_t count, row0, col0;
    uint8_t* out;
  };
  E e;
  e.smem = smem;
  const auto place = [&](uint64_t i, Item& t) __attribute__((always_inline)) {
    int64_t g, first;
    const uint64_t at = eighths ? i : i * 8 + x;
    groups.nth(a, (int64_t)(at / mine), g, first, t.count);
    const uint32_t tile = (eighths ? x * share : 0) + (uint32_t)(at % mine), part = tile % a.splits;
    uint32_t row, col;
    in_strips(tile / a.splits, a.row_tiles, a.col_tiles, row, col);
    t.row0 = (int64_t)row * BM;
    t.col0 = (int64_t)col * BN;
    t.out = (uint8_t*)a.out + g * a.L * a.C * (F32 ? 4 : 2);
    if (a.splits > 1) {
      const int64_t rows = ((t.count + a.splits - 1) / a.splits + BK - 1) / BK * BK;
      const int64_t from = part * rows < t.count ? part * rows : t.count;
      first += from;
      t.count = rows < t.count - from ? rows : t.count - from;
      t.out = (uint8_t*)(a.partial + (part * a.G + g) * a.L * a.C);
    }
    const int tid = E::thread();
    e.p.setup(tid, a.P + first * a.L, a.L, t.row0, a.L - t.row0);
    e.q.setup(tid, a.Q + first * a.C, a.C, t.col0, a.C - t.col0);
    e.template prologue<E::HEAD>(t.count, a.L, a.C);
  };
  const bool add = F32 && a.splits == 1 && a.accumulate;
  // Every second round of the XCD's workgroups is taken from the other end, so that nobody has the larger
  // groups' tiles in every one.
  const uint32_t w = blockIdx.x / 8;
  uint64_t round = 0;
  const auto item = [&]() { return round * step + (round % 2 ? step - 1 - w : w); };
  uint64_t i = item();
  if (i >= items) return;
  Item t;
  place(i, t);
  for (bool stored = false;;) {
    typename E::Acc acc = {};
    e.template loop<E::template STORES<F32>>(t.count, a.L, a.C, stored, acc);
    const Item done = t;
    ++round;
    i = item();
    if (i < items) place(i, t);
    // (nothing is added to a group without rows)
    stored = !(add && done.count == 0);
    if (stored) e.template store_behind<F32>(done.out, a.C, done.row0, a.L, done.col0, a.C, add, acc);
    if (i >= items) return;
  }
}

// The parts' sums added in their order.
template <bool F32>
__global__ void __launch_bounds__(256) wgrad_join_kernel(ProductArgs a) {
  const int64_t n = a.G * a.L * a.C / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    v4f lo = {0.f, 0.f, 0.f, 0.f}, hi = {0.f, 0.f, 0.f, 0.f};
    for (int64_t s = 0; s < a.splits; ++s) {
      const v4f* p = (const v4f*)a.partial + (s * n + i) * 2;
      lo += p[0];
      hi += p[1];
    }
    if constexpr (F32) {
      v4f* o = (v4f*)a.out + 2 * i;
      if (a.accumulate) {
        lo += o[0];
        hi += o[1];
      }
      o[0] = lo;
      o[1] = hi;
    } else {
      store_out((v4i*)a.out + i, v4i{(int)pack_bf16x2(lo.x, lo.y), (int)pack_bf16x2(lo.z, lo.w), (int)pack_bf16x2(hi.x, hi.y),
                                     (int)pack_bf16x2(hi.z, hi.w)});
    }
  }
}

}  // namespace

namespace {

constexpr int64_t kWgradRows = 256, kWgradCols = 256;

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles of the grouped output, whatever the groups' sizes.
int64_t most_row_tiles(const ProductArgs& a, int64_t BM) { return a.M / BM + (a.G < a.M ? a.G : a.M); }

enum Variant { kSplit, kStream, kPersistent };

// By the sizes that the host knows: the rows of an average group.  Few tiles of 32 x 128 leave compute units idle unless
// the contraction is split (us in captured graphs, even groups, split and by tiles of 128 x 256: one row of 4096 x 7168,
// 17 / 56 forward, 23 / 38 input's gradient; 128 rows in 2 groups, N = 2048, K = 4096, 14 / 36 and 16 / 23; 24 rows in 4,
// N = 4096, K = 2048, 20 / 22 and 23 / 39; 16 in 8, N = 4096, K = 7168, 86 / 83 forward, N = 7168, K = 2048, 53 / 66 input's
// gradient; with more such tiles, 16 in 8, N = 7168, K = 2048 forward, 57 / 45).  Uneven groups: 68 and 60 rows,
// N = 2048, K = 4096, 24 / 36 and 25 / 24.  Groups of few rows are bound by the weights' way from memory, which tiles of
// 128 rows with their stores behind the next tile keep busiest; large ones by the matrix units, which tiles of 256 x 256
// feed with half the reads (at 128 / 256 rows, forward and input's gradient: 8 groups of 512, N = 4096, K = 7168, 237 / 201
// and 252 / 217; 8 of 350, N = 4096, K = 2048, 64 / 66 and 67 / 70, uneven 78 / 64 and 73 / 70; 8 of 187, N = K = 4096,
// 86 / 81 and 93 / 79; 16 of 156, N = K = 2048, 46 / 44 forward, uneven 41 / 43; 16 of 96, N = K = 4096, 96 / 127 forward).
Variant variant_of(const ProductArgs& a) {
  if (most_row_tiles(a, 32) * cdiv(a.C, 128) <= 256) return kSplit;
  return a.M / a.G < 192 ? kStream : kPersistent;
}

template <bool Q_ALONG>
hipError_t launch_rows(ProductArgs a, int cus, hipStream_t stream) {
  switch (variant_of(a)) {
    case kSplit: {
      constexpr int BN = Q_ALONG ? 32 : 64;
      a.col_tiles = cdiv(a.C, BN);
      const dim3 grid((uint32_t)(most_row_tiles(a, 32) * a.col_tiles));
      if constexpr (Q_ALONG) hipLaunchKernelGGL((product_split_kernel<true, 32, 64, 4, 4>), grid, dim3(256), 0, stream, a);
      else hipLaunchKernelGGL((product_split_kernel<false, 64, 64, 4, 3>), grid, dim3(256), 0, stream, a);
      break;
    }
    case kStream:
      a.col_tiles = cdiv(a.C, 256);
      hipLaunchKernelGGL((product_stream_kernel<Q_ALONG>), dim3((uint32_t)cus), dim3(512), 0, stream, a);
      break;
    case kPersistent:
      a.col_tiles = cdiv(a.C, 256);
      hipLaunchKernelGGL((product_persistent_kernel<Q_ALONG>), dim3((uint32_t)cus), dim3(512), 0, stream, a);
      break;
  }
  return hipGetLastError();
}

}  // namespace

int64_t product_grid(const ProductArgs& a) {
  // tiles, or the quarters of the last ones, are counted in 32 bits
  return 2 * most_row_tiles(a, variant_of(a) == kStream ? 128 : 256) * cdiv(a.C, 256);
}

hipError_t launch_product(bool transposed, ProductArgs a, int cus, hipStream_t stream) {
  return transposed ? launch_rows<false>(a, cus, stream) : launch_rows<true>(a, cus, stream);
}

// A group's rows in parts where its tiles do not fill the compute units: up to two tiles for each, of 256 rows
// at least, and no more than 32 partial sums a value.  Fewer rows cost more for the parts' sums than they gain (us with
// parts of 128 / 256 / 512 rows at least: 256 rows in one group, N = K = 1024, 19 / 15 / 15; 1024 in 4, 31 / 16 / 16; 4096
// in 4, 66 / 42 / 35); more leave units idle where there is one tile (1024 rows, N = K = 256, 19 / 19 / 23).
int wgrad_splits(int64_t G, int64_t M, int64_t N, int64_t K) {
  if (G <= 0 || M <= 0 || N <= 0 || K <= 0) return 1;
  const int64_t tiles = G * cdiv(N, kWgradRows) * cdiv(K, kWgradCols);
  int64_t s = cdiv(512, tiles);
  const int64_t most = M / G / 256;
  s = s < most ? s : most;
  s = s < 32 ? s : 32;
  return tiles >= 256 || s < 1 ? 1 : (int)s;
}

int64_t wgrad_tiles(const ProductArgs& a) {
  return cdiv(a.L, kWgradRows) * cdiv(a.C, kWgradCols) * wgrad_splits(a.G, a.M, a.L, a.C);
}

hipError_t launch_wgrad(bool f32, ProductArgs a, int cus, hipStream_t stream) {
  a.row_tiles = cdiv(a.L, kWgradRows);
  a.col_tiles = cdiv(a.C, kWgradCols);
  a.splits = wgrad_splits(a.G, a.M, a.L, a.C);
  const int64_t tiles = a.G * cdiv(wgrad_tiles(a), 8) * 8, most = cus / 8 > 0 ? cus / 8 * 8 : 8;
  const dim3 grid((uint32_t)(tiles < most ? tiles : most));
  if (f32 || a.splits > 1) hipLaunchKernelGGL((wgrad_kernel<true>), grid, dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((wgrad_kernel<false>), grid, dim3(512), 0, stream, a);
  if (a.splits > 1) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int64_t blocks = cdiv(a.G * a.L * a.C / 8, 256);
    const dim3 join((uint32_t)(blocks < 2048 ? blocks : 2048));
    if (f32) hipLaunchKernelGGL((wgrad_join_kernel<true>), join, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((wgrad_join_kernel<false>), join, dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace fp8gg
