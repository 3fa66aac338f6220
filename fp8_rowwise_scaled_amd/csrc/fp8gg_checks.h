// Host-side checks that the layer and training operators share.  Every check runs before
// anything is enqueued; nothing here throws or allocates.
#ifndef FP8GG_CHECKS_H_
#define FP8GG_CHECKS_H_

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "fp8gg_layer.h"

namespace fp8gg {

// Leaves the message that f8f8bf16_layer_last_error() gives on this thread; ok() clears it.
fp8gg_status fail(fp8gg_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fp8gg_status ok();

inline fp8gg_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(FP8GG_ERR_HIP, "%s launch failed: %s", what, hipGetErrorString(e));
  return ok();
}

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 256;
constexpr int64_t kMaxRowWidth = 32768;   // columns that a team of threads holds in registers

// One tensor of a call.
struct Tensor {
  const char* name;
  const void* p;
  int64_t bytes;       // a lower bound is enough: it is compared for overlap
  uintptr_t align;
  bool out;
  bool optional;
};

// Pointers present, aligned, and no output sharing memory with another tensor, except
// the pairs (a, b) named in `same`, which may be one and the same buffer.
struct Same {
  const char* a;
  const char* b;
};

inline bool named(const Same& s, const Tensor& x, const Tensor& y) {
  const auto is = [](const char* p, const char* q) { return std::strcmp(p, q) == 0; };
  return (is(x.name, s.a) && is(y.name, s.b)) || (is(x.name, s.b) && is(y.name, s.a));
}

inline fp8gg_status check(std::initializer_list<Tensor> tensors, std::initializer_list<Same> same = {}) {
  for (const Tensor& t : tensors) {
    if (!t.p && !t.optional && t.bytes > 0) return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s is null", t.name);
    if (reinterpret_cast<uintptr_t>(t.p) % t.align)
      return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s must be %d-byte aligned", t.name, (int)t.align);
  }
  for (const Tensor& x : tensors) {
    if (!x.out || !x.p || x.bytes <= 0) continue;
    const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.p);
    for (const Tensor& y : tensors) {
      if (&x == &y || !y.p || y.bytes <= 0) continue;
      const uintptr_t y0 = reinterpret_cast<uintptr_t>(y.p);
      if (!(x0 < y0 + (uintptr_t)y.bytes && y0 < x0 + (uintptr_t)x.bytes)) continue;
      bool allowed = false;
      if (x0 == y0)
        for (const Same& s : same) allowed = allowed || named(s, x, y);
      if (!allowed) return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s overlaps %s", x.name, y.name);
    }
  }
  return FP8GG_OK;
}

// rows >= 0, 0 < width <= most, width % granule == 0 (the width's name in messages).
inline fp8gg_status check_width(int64_t rows, const char* rows_name, int64_t width, const char* name, int64_t granule,
                         int64_t most) {
  if (rows < 0 || width < 0)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "negative size (%s=%lld %s=%lld)", rows_name, (long long)rows, name,
                (long long)width);
  if (width == 0 || width % granule != 0)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "%s=%lld must be a positive multiple of %lld", name, (long long)width,
                (long long)granule);
  if (width > most) return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "%s=%lld exceeds %lld", name, (long long)width, (long long)most);
  if (rows > kMaxDim || rows > (int64_t(1) << 46) / width)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "%s=%lld is too large", rows_name, (long long)rows);
  return FP8GG_OK;
}

inline fp8gg_status check_block(int block, int64_t width, const char* name) {
  if (block != 0 && block != 128)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "block=%d must be 0 (one scale per row) or 128", block);
  if (block && width % 128 != 0)
    return fail(FP8GG_ERR_UNSUPPORTED_SHAPE, "block scaling needs %s=%lld to be a multiple of 128", name, (long long)width);
  return FP8GG_OK;
}

inline fp8gg_status check_float_type(int dtype, const char* name) {
  if (dtype != FP8GG_DTYPE_BF16 && dtype != FP8GG_DTYPE_F32)
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "%s=%d must be bf16 (0) or fp32 (1)", name, dtype);
  return FP8GG_OK;
}

inline fp8gg_status check_workspace(const void* ws, int64_t have, int64_t need) {
  if (have < need || (need > 0 && !ws))
    return fail(FP8GG_ERR_INVALID_ARGUMENT, "workspace of %lld bytes, %lld needed", ws ? (long long)have : 0,
                (long long)need);
  return FP8GG_OK;
}

#define FP8GG_TRY(call)                         \
  do {                                          \
    const fp8gg_status st_ = (call);            \
    if (st_ != FP8GG_OK) return st_;            \
  } while (0)

}  // namespace fp8gg

#endif  // FP8GG_CHECKS_H_
