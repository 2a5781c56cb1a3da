// Host-side driver for the sanitizer build of the norm, cross entropy and
// AdamW entry points (see tests/test_train_abi_sanitizers.py): argument
// validation and workspace queries over extreme sizes, strides and leading
// dimensions.  Calls that pass validation reach a launch, which fails without a
// GPU (FP8BW_ERR_HIP); where a GPU is visible nothing is run (exit 77).
#include <hip/hip_runtime_api.h>

#include <cstdint>
#include <cstdio>
#include <vector>

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
  const int64_t dims[] = {kMin, -1, 0, 1, 15, 16, 64, 128, 4096, 16384, 16400, (int64_t)1 << 22, (int64_t)1 << 30,
                          (int64_t)1 << 48, kMax - 15, kMax};
  const int64_t lds[] = {kMin, -8, 0, 1, 64, 4096, (int64_t)1 << 31, ((int64_t)1 << 48) - 16, (int64_t)1 << 62, kMax - 15};
  unsigned char* const p = buf;
  float* const f = (float*)buf;
  for (int64_t rows : dims)
    for (int64_t cols : dims) {
      (void)fp8bw_rms_norm_bwd_ws_bytes(rows, cols);
      for (int64_t k : dims)
        for (int b = 0; b < 2; ++b) (void)fp8bw_linear_xent_ws_bytes(rows, cols, k, b);
      for (int64_t a : lds)
        for (int64_t s : lds) {
          KNOWN(fp8bw_rms_norm_fwd(p, a, p, s, p, 0, 1e-6f, rows, cols, p, a, f, p, s, p, a, f, s, a, p, s, f, a, s, nullptr));
          KNOWN(fp8bw_rms_norm_fwd(p, a, nullptr, 0, p, 1, 0.f, rows, cols, nullptr, 0, f, nullptr, 0, p, s, f, 1, s, nullptr,
                                   0, nullptr, 0, 0, nullptr));
          KNOWN(fp8bw_rms_norm_bwd(p, a, p, s, f, p, 0, p, a, rows, cols, p, s, p, p, sizeof(buf), nullptr));
          for (int64_t k : {(int64_t)0, (int64_t)64, (int64_t)100, (int64_t)1 << 20, kMax}) {
            KNOWN(fp8bw_linear_xent_fwd(p, a, p, s, (int64_t*)buf, -100, rows, cols, k, f, f, p, sizeof(buf), nullptr));
            KNOWN(fp8bw_linear_xent_bwd(f, p, a, p, s, (int64_t*)buf, kMin, f, rows, cols, k, p, a, p, s, p, sizeof(buf),
                                        nullptr));
          }
        }
    }
  for (int count : {-1, 0, 1, 41, 200})
    for (int64_t numel : dims)
      for (int state = -1; state < 3; ++state)
        for (int64_t step : {kMin, (int64_t)0, (int64_t)1, (int64_t)1 << 40, kMax}) {
          std::vector<fp8bw_adamw_tensor> t(count > 0 ? count : 1);
          for (auto& x : t)
            x = {p, p, p, p, state == 1 ? f : nullptr, state == 1 ? f : nullptr, nullptr, numel, 0, 1};
          KNOWN(fp8bw_adamw_step(t.data(), count, state, step, 1e300, 0.0, 0.999999999, 1e300, 1e300, f, 1,
                                 0xFFFFFFFFFFFFFFFFull, nullptr));
        }
  std::printf("%ld checks, %d failures\n", checks, failures);
  return failures ? 1 : 0;
}
