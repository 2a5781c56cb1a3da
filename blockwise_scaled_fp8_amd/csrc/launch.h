// Internal host-side launchers shared by the C ABI (api.cpp) and the kernel
// translation units.  Arguments are validated by the caller (api.cpp); the
// launchers only size grids and enqueue on `stream`.  Each returns the
// hipError_t of the launch.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

namespace fp8bw {

// ---- quantization (quant.hip) ----
// 1x128 blocks along columns: q[r, c], recip[r*rs_row + kb*rs_kb].
hipError_t launch_quant_1x128_rows(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                   void* q, int64_t ld_q, float* recip, int64_t rs_row,
                                   int64_t rs_kb, hipStream_t stream);
// 128x128 tiles; transpose=1 writes q = x^T [cols, rows] and indexes recip by
// (output row block, output column block).
hipError_t launch_quant_128x128(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                int transpose, void* q, int64_t ld_q, float* recip,
                                int64_t rs_row, int64_t rs_kb, hipStream_t stream);
// 1x128 blocks running down the rows; output transposed q = x^T [cols, rows],
// recip[c*rs_row + mb*rs_kb].
hipError_t launch_quant_1x128_cols_t(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                     void* q, int64_t ld_q, float* recip, int64_t rs_row,
                                     int64_t rs_kb, hipStream_t stream);
// Both layouts from one read: block_128 = 0 writes the 1x128 row-block codes
// (q, recip[r*rs_row + kb*rs_kb]) and the transposed 1x128 column-block codes
// (qt = x^T, recip_t[c*rst_row + mb*rst_kb]); block_128 = 1 writes the
// 128x128 codes and the transposed codes with the tile scale in both orders.
// stream_t: the transposed codes go out with nontemporal stores.
hipError_t launch_quant_dual(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int block_128,
                             void* q, int64_t ld_q, float* recip, int64_t rs_row, int64_t rs_kb,
                             void* qt, int64_t ld_qt, float* recip_t, int64_t rst_row,
                             int64_t rst_kb, bool stream_t, hipStream_t stream);
// Per-tensor: partial amax into ws (n_partials floats, at most
// kMaxTensorwisePartials), then quantize.
constexpr int kMaxTensorwisePartials = 1024;
constexpr int kMaxDevices = 64;
int tensorwise_partials(int64_t rows, int64_t cols);
hipError_t launch_quant_tensorwise(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                   void* q, int64_t ld_q, float* recip, float* ws,
                                   hipStream_t stream);
// The same with the partials in the library's own per-device array (no
// workspace; calls that overlap on one GPU race on it).
hipError_t launch_quant_tensorwise_noalloc(const void* x, int64_t rows, int64_t cols,
                                           int64_t ld_x, void* q, int64_t ld_q, float* recip,
                                           hipStream_t stream);

// ---- GEMM (gemm.hip) ----
enum ScaleMode { kBlockB128 = 0, kBlockB1x128 = 1, kTensorwise = 2 };
enum OutKind { kOutBf16 = 0, kOutF32 = 1 };

struct GemmProblem {
  const void* a; int64_t lda;
  const void* b; int64_t ldb;
  const float* ra; int64_t ra_s_row, ra_s_kb;
  const float* rb; int64_t rb_s_row, rb_s_kb;
  void* out; int64_t ldo;
  int64_t M, N, K;
  int mode;       // ScaleMode
  int out_kind;   // OutKind
  const void* bias = nullptr;   // optional bf16 [N] added before the output cast
  int b_kn = 0;                 // B given as [K, N] (b[k * ldb + n]) instead of [N, K]
};

// Tile configurations; the table lives in gemm.hip.
int gemm_num_configs();
// Whether config `cfg` accepts this problem.
bool gemm_config_ok(const GemmProblem& p, int cfg);

// How one GEMM call is run: the tile configuration, a whole-problem split-K
// count (fp32 partials [splits, M, N], then an ordered reduce), or a tail
// split (tiles_full tiles unsplit, the remaining tiles split tail_splits
// ways into tile-local partials, then reduced), and the workspace it needs.
struct GemmPlan {
  int cfg;
  int splits;
  int tail_splits;
  int64_t tiles;
  int64_t tiles_full;
  size_t ws_bytes;
};
// config < 0: built-in choice; splits > 0 forces a whole-problem split
// (no tail split); splits == 0 lets the plan choose when allow_split.
GemmPlan gemm_plan(const GemmProblem& p, int config, int splits, bool allow_split);
hipError_t launch_gemm(const GemmProblem& p, const GemmPlan& plan, void* ws, hipStream_t stream);
// Fill a contiguous bf16 [rows, cols] matrix with +0.
// Grouped blockwise GEMM: row groups of A / out ending at device int32
// group_end[g] (cumulative), each with B + g*b_s_group and rb + g*rb_s_group.
bool grouped_gemm_ok(const GemmProblem& p, int groups);
hipError_t launch_grouped_gemm(const GemmProblem& p, int groups, const int* group_end,
                               int64_t b_s_group, int64_t rb_s_group, hipStream_t stream);
hipError_t launch_zero_bf16(void* out, int64_t rows, int64_t cols, hipStream_t stream);

// ---- RMS norm (rmsnorm.hip) ----
struct NormWeight {
  const void* p;   // bf16 or fp32 [cols]
  int f32;
};
constexpr int64_t kNormMaxCols = 16384;   // 1024 threads x 2 chunks of 8 columns
struct NormFwdArgs {
  int64_t rows, cols;
  const uint16_t* x; int64_t ld_x;
  const uint16_t* residual; int64_t ld_res;   // nullptr: s = x
  uint16_t* sum; int64_t ld_sum;              // s, written with a residual (may be x or residual)
  NormWeight weight;
  float eps;
  float* rstd;
  uint16_t* y; int64_t ld_y;                                          // nullptr: not written
  uint8_t* q; int64_t ld_q; float* recip; int64_t rs_row, rs_kb;      // nullptr: not written
  uint8_t* qt; int64_t ld_qt; float* recip_t; int64_t rst_row, rst_kb;
};
struct NormBwdArgs {
  int64_t rows, cols;
  const uint16_t* dy; int64_t ld_dy;
  const uint16_t* s; int64_t ld_s;
  const float* rstd;
  NormWeight weight;
  const uint16_t* dres; int64_t ld_dres;      // nullptr: none
  uint16_t* dx; int64_t ld_dx;
  void* dweight;                              // the weight's type
  float* partial;                             // rms_norm_bwd_ws_bytes
};
hipError_t launch_rms_norm_fwd(const NormFwdArgs& p, hipStream_t stream);
size_t rms_norm_bwd_ws_bytes(int64_t rows, int64_t cols);
hipError_t launch_rms_norm_bwd(const NormBwdArgs& p, hipStream_t stream);

// ---- AdamW (adamw.hip) ----
enum AdamwFlags { kAdamwParamF32 = 1, kAdamwGradF32 = 2 };
struct AdamwTensor {
  void* param;
  const void* grad;
  void* m;             // fp32, or E4M3 codes
  void* v;             // fp32, or E4M3 codes of the root
  float* m_scale;      // 8-bit states: one per 128 elements
  float* root_scale;
  float* master;       // nullptr: none
  int64_t numel;
  uint32_t key;        // of the tensor's random bits
  int flags;
};
// One launch's tensors and constants, passed by value: 40 tensors keep the
// kernel's arguments below 4 KB.
constexpr int kAdamwTensors = 40;
struct AdamwLaunch {
  AdamwTensor t[kAdamwTensors];
  int first[kAdamwTensors];   // first workgroup of each tensor
  int count, iters;           // tensors; runs of 2048 elements per workgroup
  const float* grad_scale;    // device scalar or nullptr
  float beta1, one_minus_beta1, beta2, one_minus_beta2;
  float decay;                // 1 - lr * weight_decay
  float step_size;            // lr / (1 - beta1^t)
  float root_factor;          // 1 / sqrt(1 - beta2^t)
  float eps;
};
uint32_t adamw_key(uint64_t seed, int ordinal);
hipError_t launch_adamw(const AdamwLaunch& L, int workgroups, bool eight, bool random,
                        hipStream_t stream);

// ---- linear cross entropy (xent.hip) ----
struct XentArgs {
  int64_t T, V, K;
  const void* h; int64_t ld_h;        // bf16 [T, K]
  const void* w; int64_t ld_w;        // bf16 [V, K]
  const int64_t* target;              // [T]
  int64_t ignore_index;
  float* loss;                        // [T] (forward)
  float* lse;                         // [T] (forward writes, backward reads)
  const float* dloss;                 // [T] (backward)
  const float* nll;                   // [T] the forward's losses or nullptr (backward)
  void* dh; int64_t ld_dh;            // bf16 [T, K] or nullptr
  void* dw; int64_t ld_dw;            // bf16 [V, K] or nullptr
};
size_t xent_ws_bytes(int64_t T, int64_t V, int64_t K, bool backward);
hipError_t launch_xent_fwd(const XentArgs& p, void* ws, hipStream_t stream);
hipError_t launch_xent_bwd(const XentArgs& p, void* ws, hipStream_t stream);
// +0 in a bf16 [rows, cols] matrix of leading dimension ld.
hipError_t launch_zero_rows_bf16(void* out, int64_t rows, int64_t cols, int64_t ld, hipStream_t stream);

}  // namespace fp8bw
