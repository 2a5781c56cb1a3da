// What the C ABI's translation units share: the exported-function marker,
// the calling thread's error message and the argument checks.  Pure host
// code.
#pragma once

#include "../../include/fp8bw.h"

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#define FP8BW_API extern "C" __attribute__((visibility("default")))

namespace fp8bw {
namespace api {

// Sets the calling thread's message and returns `status`.
int fail(int status, const char* fmt, ...);
// Clears the message; FP8BW_OK.
int ok();
int hip_status(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

constexpr int64_t kMaxDim = (int64_t)1 << 30;   // int32 indexing inside the kernels
constexpr int64_t kMaxGridY = 65535;

// Every element offset a call can form stays below 2^48: no allocation is
// larger, and the bound keeps each product the host and the kernels form on
// offsets (tile and byte offsets) far from int64 overflow.
constexpr int64_t kMaxExtent = (int64_t)1 << 48;

// (rows - 1) * ld + cols < kMaxExtent for a [rows, cols] matrix with
// leading dimension ld (1 <= rows, cols <= 2^32; the product is not formed).
inline bool extent_ok(int64_t rows, int64_t ld, int64_t cols) {
  if (ld < 0) return false;
  if (rows <= 1) return cols < kMaxExtent;
  return cols < kMaxExtent && ld <= (kMaxExtent - 1 - cols) / (rows - 1);
}

// A strided 2-D scale grid [ni, nj] with strides (si, sj) must map distinct
// index pairs to distinct addresses, and its last element must lie below
// kMaxExtent.  The stride of a dimension of size 1 is never used.
inline bool strides_injective(int64_t ni, int64_t nj, int64_t si, int64_t sj) {
  if (si < 0 || sj < 0) return false;
  if (ni <= 1 && nj <= 1) return true;
  if (ni <= 1) return sj >= 1 && extent_ok(nj, sj, 1);
  if (nj <= 1) return si >= 1 && extent_ok(ni, si, 1);
  // sj >= si * ni (or si >= sj * nj) without forming the product
  const bool nested = (si >= 1 && sj / ni >= si) || (sj >= 1 && si / nj >= sj);
  if (!nested) return false;
  // (ni - 1) * si + (nj - 1) * sj < kMaxExtent
  if (!extent_ok(ni, si, 1)) return false;
  const int64_t rest = kMaxExtent - 1 - (ni - 1) * si;
  return sj <= rest / (nj - 1);
}

// The stride of a size-1 dimension is never used; pass 0 for it so that
// no later arithmetic sees an arbitrary value.
inline int64_t used_stride(int64_t n, int64_t s) { return n > 1 ? s : 0; }

// a * b * c in size_t, SIZE_MAX when it does not fit.
inline size_t mul_sat(size_t a, size_t b, size_t c) {
  size_t ab, abc;
  if (__builtin_mul_overflow(a, b, &ab) || __builtin_mul_overflow(ab, c, &abc)) return SIZE_MAX;
  return abc;
}

inline size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace api
}  // namespace fp8bw
