// Argument checks of matrices, vectors and codes that the entry points around
// the GEMM share.  Pure host code.
#pragma once

#include "api_common.h"

namespace fp8bw {
namespace api {

// A bf16 [rows, cols] matrix: 16-byte aligned rows of `ld` elements.
inline int check_bf16(const void* p, int64_t rows, int64_t cols, int64_t ld, const char* name) {
  if (!p) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  if (!aligned(p, 16)) return fail(FP8BW_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (rows > 1 && (ld < cols || ld % 8))
    return fail(FP8BW_ERR_LAYOUT, "leading dimension %lld of %s must be >= %lld and a multiple of 8",
                (long long)ld, name, (long long)cols);
  if (!extent_ok(rows, ld, cols)) return fail(FP8BW_ERR_LAYOUT, "%s reaches past 2^48 elements", name);
  return FP8BW_OK;
}

inline int check_f32(const void* p, const char* name) {
  if (!p) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  if (!aligned(p, 4)) return fail(FP8BW_ERR_ALIGN, "%s must be 4-byte aligned", name);
  return FP8BW_OK;
}

// E4M3 codes [rows, cols] and their scale grid [rows, blocks].
inline int check_codes(const void* q, int64_t rows, int64_t cols, int64_t ld, const float* recip, int64_t rs_row,
                       int64_t rs_kb, const char* name, int64_t blocks) {
  if (!aligned(q, 16)) return fail(FP8BW_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (rows > 1 && (ld < cols || ld % 16))
    return fail(FP8BW_ERR_LAYOUT, "leading dimension %lld of %s must be >= %lld and a multiple of 16",
                (long long)ld, name, (long long)cols);
  if (!extent_ok(rows, ld, cols)) return fail(FP8BW_ERR_LAYOUT, "%s reaches past 2^48 elements", name);
  const int st = check_f32(recip, "reciprocal scales");
  if (st != FP8BW_OK) return st;
  if (!strides_injective(rows, blocks, rs_row, rs_kb))
    return fail(FP8BW_ERR_LAYOUT, "scale strides (%lld, %lld) of %s alias or are negative", (long long)rs_row,
                (long long)rs_kb, name);
  return FP8BW_OK;
}
inline int check_codes(const void* q, int64_t rows, int64_t cols, int64_t ld, const float* recip, int64_t rs_row,
                       int64_t rs_kb, const char* name) {
  return check_codes(q, rows, cols, ld, recip, rs_row, rs_kb, name, cdiv(cols, 128));
}

inline int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return fail(FP8BW_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned(ws, 256)) return fail(FP8BW_ERR_ALIGN, "ws must be 256-byte aligned");
  return FP8BW_OK;
}

}  // namespace api
}  // namespace fp8bw
