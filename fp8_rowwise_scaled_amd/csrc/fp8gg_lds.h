// Device helpers that the matrix products share: vector types, copies from global memory
// straight into LDS with their waits, and the order of tiles across the XCDs.
#ifndef FP8GG_LDS_H_
#define FP8GG_LDS_H_

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8gg {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;
typedef __attribute__((address_space(1))) void* gbl_ptr_t;

// Sixteen zero bytes.  K-tail chunks at or past K are fetched from here, so the
// last K tile is zero-padded without a masked load.
static __device__ __attribute__((aligned(64))) const uint8_t g_zero16[64] = {0};

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  // v_cvt_pk_bf16_f32: round to nearest even.
  const __bf16 l = (__bf16)lo;
  const __bf16 h = (__bf16)hi;
  return (uint32_t)__builtin_bit_cast(uint16_t, l) | ((uint32_t)__builtin_bit_cast(uint16_t, h) << 16);
}

// s_waitcnt immediate with only the vector-memory counter constrained to <= n
// (gfx9 encoding: vmcnt[3:0] in bits 3:0, vmcnt[5:4] in bits 15:14; expcnt (bits
// 6:4) and lgkmcnt (bits 11:8) left at their maxima).
constexpr int vmcnt_imm(int n) { return (n & 15) | ((n >> 4) << 14) | 0x0F70; }

__device__ __forceinline__ void wait_vmcnt_le(int n) {
  // The instruction takes an immediate: a switch over the counts the kernels use
  // (every count a compile-time constant folds to one instruction).
  switch (n) {
#define FP8GG_WAIT_CASE(k) \
  case k: __builtin_amdgcn_s_waitcnt(vmcnt_imm(k)); break;
    FP8GG_WAIT_CASE(1) FP8GG_WAIT_CASE(2) FP8GG_WAIT_CASE(3) FP8GG_WAIT_CASE(4) FP8GG_WAIT_CASE(5)
    FP8GG_WAIT_CASE(6) FP8GG_WAIT_CASE(7) FP8GG_WAIT_CASE(8) FP8GG_WAIT_CASE(9) FP8GG_WAIT_CASE(10)
    FP8GG_WAIT_CASE(11) FP8GG_WAIT_CASE(12) FP8GG_WAIT_CASE(13) FP8GG_WAIT_CASE(14) FP8GG_WAIT_CASE(15)
    FP8GG_WAIT_CASE(16) FP8GG_WAIT_CASE(18) FP8GG_WAIT_CASE(20) FP8GG_WAIT_CASE(24) FP8GG_WAIT_CASE(30)
    FP8GG_WAIT_CASE(32) FP8GG_WAIT_CASE(36) FP8GG_WAIT_CASE(40) FP8GG_WAIT_CASE(42) FP8GG_WAIT_CASE(48)
#undef FP8GG_WAIT_CASE
    default: __builtin_amdgcn_s_waitcnt(vmcnt_imm(0)); break;  // 0, or a count not listed: wait for all
  }
}

// LDS rows are BK bytes (BK/16 chunks of 16 bytes); chunk c of row p is stored at
// chunk c ^ lds_swz<BK>(p).  gfx950 serves a ds_read_b128 sixteen lanes (256 bytes,
// 64 banks) at a time, and rows p and p + 256/BK share banks, so XOR-ing with
// (p / (256/BK)) mod (BK/16) spreads the 16 consecutive rows that 16 lanes read at
// one logical chunk over all 16 bank groups.
template <int BK>
__device__ __forceinline__ int lds_swz(int p) { return (p / (256 / BK)) & (BK / 16 - 1); }

// One 16-byte-per-lane copy from global memory straight into LDS: lane l's 16 bytes
// land at LDS byte lds_base + 16*l.  lds_base is wave-uniform by construction; the
// readfirstlane states it, so that it always reaches M0 through a scalar register
// even where the compiler cannot prove the uniformity itself.  Written as inline
// assembly so that the compiler's wait-count pass does not track it: the pass
// cannot tell LDS slots apart when the slot index is a run-time value and would
// otherwise drain every copy in flight before each LDS read.  The callers order
// copies and reads themselves (wait_vmcnt_le, then a workgroup barrier).
__device__ __forceinline__ void copy16_to_lds(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :: "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds_base)) : "memory");
}

// Same from a base that all lanes share and a byte offset per lane.
__device__ __forceinline__ void copy16_to_lds(const void* base, uint32_t off, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(off), "s"(base), "s"(__builtin_amdgcn_readfirstlane(lds_base)) : "memory");
}

// Same with the non-temporal hint, for data that one workgroup reads once (the
// weights of a small-M call): it streams past the caches instead of displacing
// what other workgroups reuse.
__device__ __forceinline__ void copy16_to_lds_stream(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt"
               :: "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds_base)) : "memory");
}

// Same, 4 bytes per lane: lane l's 4 bytes land at LDS byte lds_base + 4*l.
__device__ __forceinline__ void copy4_to_lds(const void* src, uint32_t lds_base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :: "v"(src), "s"(__builtin_amdgcn_readfirstlane(lds_base)) : "memory");
}

__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(lds_ptr_t)p;
}

// Orders the waves of a workgroup, and waits for nothing: what they have copied or written they wait for
// themselves before it.
__device__ __forceinline__ void block_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ... after each wave's own LDS operations are done: what one has written, the others read after it.
__device__ __forceinline__ void publish_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);   // lgkmcnt 0, the other counters left alone
  block_barrier();
}

// Tile order across the XCDs.  MI355X dispatches consecutive workgroups of a grid
// to its eight XCDs in turn, and each XCD has its own L2, so workgroup w runs on
// XCD w % 8.  xcd_slot only reorders work (every tile is still computed by one
// workgroup in the same K order, so results do not depend on it): of a grid of P
// workgroups, XCD x runs workgroups x, x + 8, ..., ceil((P - x) / 8) of them, and
// xcd_slot gives them the contiguous positions that follow those of XCDs
// 0 .. x-1 (a permutation of [0, P) for any P), so that the workgroups running
// together on one XCD share operands.
__device__ __forceinline__ int64_t xcd_slot(int64_t w, int64_t P) {
  const int64_t x = w % 8, q = P / 8, r = P % 8;
  return x * q + (x < r ? x : r) + w / 8;
}

}  // namespace fp8gg

#endif  // FP8GG_LDS_H_
