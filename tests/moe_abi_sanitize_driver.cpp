// Host-side driver for the sanitizer build of the expert, gated activation and
// grouped weight-gradient entry points (see tests/test_moe_abi_sanitizers.py):
// argument validation, workspace queries and launch plans over extreme sizes,
// strides and leading dimensions.  Calls that pass validation reach a launch, which
// fails without a GPU (FP8BW_ERR_HIP); where a GPU is visible nothing is run (exit 77).
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>

#include "fp8bw.h"

namespace {

int failures = 0;
long checks = 0;
constexpr int64_t kMin = INT64_MIN, kMax = INT64_MAX;
alignas(256) unsigned char buf[8192];

void known(int st, int line) {
  ++checks;
  const bool ok = st >= FP8BW_OK && st <= FP8BW_ERR_HIP && (st == FP8BW_OK) == (fp8bw_last_error()[0] == 0);
  if (!ok) {
    std::fprintf(stderr, "status %d with message '%s' (line %d)\n", st, fp8bw_last_error(), line);
    ++failures;
  }
}
#define KNOWN(call) known((call), __LINE__)

}  // namespace

int main() {
  int n = 0;
  if (hipGetDeviceCount(&n) == hipSuccess && n > 0) {
    std::printf("a GPU is visible: not run\n");
    return 77;
  }
  const int64_t dims[] = {kMin, -1, 0, 1, 16, 64, 128, 4096, 16400, 65536, (int64_t)1 << 20, ((int64_t)1 << 24) - 1,
                          ((int64_t)1 << 27) - 128, (int64_t)1 << 27, (int64_t)1 << 48, kMax - 15, kMax};
  const int64_t few[] = {kMin, 0, 1, 128, 65536, (int64_t)1 << 20, kMax};
  const int64_t lds[] = {kMin, -8, 0, 1, 64, 4096, ((int64_t)1 << 24) - 16, (int64_t)1 << 31, ((int64_t)1 << 48) - 16,
                         (int64_t)1 << 62, kMax - 15};
  unsigned char* const p = buf;
  float* const f = (float*)buf;
  int32_t* const i = (int32_t*)buf;

  for (int64_t tokens : dims)
    for (int64_t topk : {kMin, (int64_t)0, (int64_t)1, (int64_t)2, (int64_t)64, (int64_t)65, kMax})
      for (int64_t experts : {kMin, (int64_t)0, (int64_t)1, (int64_t)16, (int64_t)1024, (int64_t)1025, kMax})
        for (int64_t align : {kMin, (int64_t)0, (int64_t)1, (int64_t)128, (int64_t)65536, kMax}) {
          const int64_t rows = fp8bw_moe_rows(tokens, topk, experts, align);
          const size_t ws = fp8bw_moe_sort_ws_bytes(tokens, topk, experts);
          if (rows < 0 || rows >= (int64_t)1 << 27) ++failures;
          for (int64_t r : {kMin, rows - 1, rows, kMax}) {
            KNOWN(fp8bw_moe_sort(p, 32, tokens, topk, experts, align, r, i, i, i, p, ws, nullptr));
            KNOWN(fp8bw_moe_sort(p, 64, tokens, topk, experts, align, r, i, i, i, nullptr, 0, nullptr));
          }
        }

  for (int64_t rows : dims)
    for (int64_t cols : dims)
      for (int64_t a : lds)
        for (int64_t s : lds) {
          const fp8bw_layouts all = {p, a, p, s, f, a, s, p, s, f, s, a}, q = {nullptr, 0, p, a, f, 1, s, nullptr, 0, nullptr, 0, 0};
          for (int64_t tokens : {kMin, (int64_t)0, (int64_t)1, ((int64_t)1 << 24) - 1, kMax}) {
            KNOWN(fp8bw_moe_gather(p, a, tokens, 2, i, i, rows, cols, &all, nullptr));
            KNOWN(fp8bw_moe_gather(p, s, tokens, 64, i, i, rows, cols, &q, nullptr));
            KNOWN(fp8bw_moe_combine(p, a, f, 1, tokens, 8, i, rows, cols, p, s, nullptr));
            KNOWN(fp8bw_moe_combine_bwd(p, a, p, s, f, 0, tokens, 2, i, i, rows, cols, &all, f, nullptr));
          }
          KNOWN(fp8bw_swiglu_fwd(p, a, rows, cols, &all, p, s, f, a, s, nullptr));
          KNOWN(fp8bw_swiglu_fwd(p, s, rows, cols, &q, p, a, f, 1, a, nullptr));
          KNOWN(fp8bw_swiglu_bwd(p, a, p, s, f, s, a, rows, cols, &all, p, a, f, a, s, nullptr));
          KNOWN(fp8bw_swiglu_bwd(p, a, p, s, nullptr, 0, 0, rows, cols, &q, nullptr, 0, nullptr, 0, 0, nullptr));
        }

  for (int64_t M : dims)
    for (int64_t N : dims)
      for (int64_t K : few)
        for (int groups : {INT32_MIN, 0, 1, 7, 1 << 20, INT32_MAX}) {
          const size_t ws = fp8bw_grouped_wgrad_ws_bytes(M, N, K, groups);
          for (int64_t a : {(int64_t)0, (int64_t)128, (int64_t)1 << 27, (int64_t)1 << 48, kMax - 15})
            for (size_t w : {(size_t)0, ws, (size_t)-1})
              KNOWN(fp8_scaled_grouped_gemm_blockwise_wgrad(p, a, f, 1, a, p, a, f, a, 1, groups, (const int*)i, M, N, K, p, a,
                                                            a, groups & 1, p, w, nullptr));
        }

  for (int64_t rows : dims)
    for (int64_t cols : dims)
      for (int64_t a : lds)
        for (int64_t s : {kMin, (int64_t)-8, (int64_t)0, (int64_t)128, (int64_t)1 << 48, kMax - 15})
          for (int groups : {-1, 1, 65535, INT32_MAX})
            for (int t = 0; t < 2; ++t)
              KNOWN(fp8_blockwise_quant_grouped(p, rows, cols, a, s, groups, t, p, a, s, f, a, s, s, nullptr));
  std::printf("%ld checks, %d failures\n", checks, failures);
  return failures ? 1 : 0;
}
