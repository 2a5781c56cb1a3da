// C ABI of the operators around the linear in a training step: RMS norm,
// vocabulary cross entropy, AdamW.  Validation and dispatch only; the
// contracts are in include/fp8bw.h.

#include <cmath>

#include "api_common.h"
#include "launch.h"

using namespace fp8bw::api;

namespace {

// A bf16 [rows, cols] matrix: 16-byte aligned rows of `ld` elements.
int check_bf16(const void* p, int64_t rows, int64_t cols, int64_t ld, const char* name) {
  if (!p) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  if (!aligned(p, 16)) return fail(FP8BW_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (rows > 1 && (ld < cols || ld % 8))
    return fail(FP8BW_ERR_LAYOUT, "leading dimension %lld of %s must be >= %lld and a multiple of 8",
                (long long)ld, name, (long long)cols);
  if (!extent_ok(rows, ld, cols)) return fail(FP8BW_ERR_LAYOUT, "%s reaches past 2^48 elements", name);
  return FP8BW_OK;
}

int check_f32(const void* p, const char* name) {
  if (!p) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  if (!aligned(p, 4)) return fail(FP8BW_ERR_ALIGN, "%s must be 4-byte aligned", name);
  return FP8BW_OK;
}

// E4M3 codes [rows, cols] and their scale grid [rows, ceil(cols / 128)].
int check_codes(const void* q, int64_t rows, int64_t cols, int64_t ld, const float* recip, int64_t rs_row,
                int64_t rs_kb, const char* name) {
  if (!aligned(q, 16)) return fail(FP8BW_ERR_ALIGN, "%s must be 16-byte aligned", name);
  if (rows > 1 && (ld < cols || ld % 16))
    return fail(FP8BW_ERR_LAYOUT, "leading dimension %lld of %s must be >= %lld and a multiple of 16",
                (long long)ld, name, (long long)cols);
  if (!extent_ok(rows, ld, cols)) return fail(FP8BW_ERR_LAYOUT, "%s reaches past 2^48 elements", name);
  const int st = check_f32(recip, "reciprocal scales");
  if (st != FP8BW_OK) return st;
  if (!strides_injective(rows, cdiv(cols, 128), rs_row, rs_kb))
    return fail(FP8BW_ERR_LAYOUT, "scale strides (%lld, %lld) of %s alias or are negative", (long long)rs_row,
                (long long)rs_kb, name);
  return FP8BW_OK;
}

constexpr int64_t kNormMaxRows = (int64_t)1 << 22;

int check_norm(int64_t rows, int64_t cols, int weight_dtype) {
  if (rows < 0 || cols < 0) return fail(FP8BW_ERR_SHAPE, "negative dimension");
  if (weight_dtype != FP8BW_OUT_BF16 && weight_dtype != FP8BW_OUT_F32)
    return fail(FP8BW_ERR_UNSUPPORTED, "unknown weight type %d", weight_dtype);
  // A launch has fewer than 2^32 threads, at most 1024 a row.
  if (rows >= kNormMaxRows) return fail(FP8BW_ERR_SHAPE, "rows=%lld must be below 2^22", (long long)rows);
  if (cols % 16 || cols > fp8bw::kNormMaxCols)
    return fail(FP8BW_ERR_SHAPE, "cols=%lld must be a multiple of 16 and at most %lld", (long long)cols,
                (long long)fp8bw::kNormMaxCols);
  return FP8BW_OK;
}

int check_weight(const void* w) {
  if (!w) return fail(FP8BW_ERR_NULL, "weight must be non-null");
  if (!aligned(w, 16)) return fail(FP8BW_ERR_ALIGN, "weight must be 16-byte aligned");
  return FP8BW_OK;
}

}  // namespace

FP8BW_API int fp8bw_rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                                 const void* weight, int weight_dtype, float eps, int64_t rows,
                                 int64_t cols, void* sum, int64_t ld_sum, float* rstd, void* y,
                                 int64_t ld_y, void* q, int64_t ld_q, float* recip, int64_t rs_row,
                                 int64_t rs_kb, void* qt, int64_t ld_qt, float* recip_t,
                                 int64_t rst_row, int64_t rst_kb, void* stream) {
  int st = check_norm(rows, cols, weight_dtype);
  if (st != FP8BW_OK) return st;
  if (!(eps >= 0.f)) return fail(FP8BW_ERR_UNSUPPORTED, "eps must be >= 0");
  if (qt && rows % 16)
    return fail(FP8BW_ERR_SHAPE, "transposed codes need rows %% 16 == 0 (rows=%lld)", (long long)rows);
  if (rows == 0 || cols == 0) return ok();
  if ((st = check_bf16(x, rows, cols, ld_x, "x")) != FP8BW_OK) return st;
  if ((st = check_weight(weight)) != FP8BW_OK) return st;
  if ((st = check_f32(rstd, "rstd")) != FP8BW_OK) return st;
  if (residual) {
    if ((st = check_bf16(residual, rows, cols, ld_res, "residual")) != FP8BW_OK) return st;
    if ((st = check_bf16(sum, rows, cols, ld_sum, "sum")) != FP8BW_OK) return st;
    if (rows > 1 && ((sum == x && ld_sum != ld_x) || (sum == residual && ld_sum != ld_res)))
      return fail(FP8BW_ERR_LAYOUT, "sum in the place of an input needs that input's leading dimension");
  }
  if (y && (st = check_bf16(y, rows, cols, ld_y, "y")) != FP8BW_OK) return st;
  if (q && (st = check_codes(q, rows, cols, ld_q, recip, rs_row, rs_kb, "q")) != FP8BW_OK) return st;
  if (qt && (st = check_codes(qt, cols, rows, ld_qt, recip_t, rst_row, rst_kb, "qt")) != FP8BW_OK) return st;
  fp8bw::NormFwdArgs p = {};
  p.rows = rows; p.cols = cols;
  p.x = (const uint16_t*)x; p.ld_x = used_stride(rows, ld_x);
  p.residual = (const uint16_t*)residual; p.ld_res = used_stride(rows, ld_res);
  p.sum = (uint16_t*)sum; p.ld_sum = used_stride(rows, ld_sum);
  p.weight.p = weight; p.weight.f32 = weight_dtype == FP8BW_OUT_F32;
  p.eps = eps;
  p.rstd = rstd;
  p.y = (uint16_t*)y; p.ld_y = used_stride(rows, ld_y);
  p.q = (uint8_t*)q; p.ld_q = used_stride(rows, ld_q);
  p.recip = recip; p.rs_row = used_stride(rows, rs_row); p.rs_kb = used_stride(cdiv(cols, 128), rs_kb);
  p.qt = (uint8_t*)qt; p.ld_qt = ld_qt;
  p.recip_t = recip_t; p.rst_row = rst_row; p.rst_kb = used_stride(cdiv(rows, 128), rst_kb);
  return hip_status(fp8bw::launch_rms_norm_fwd(p, (hipStream_t)stream), "fp8bw_rms_norm_fwd");
}

FP8BW_API size_t fp8bw_rms_norm_bwd_ws_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows >= kNormMaxRows || cols > fp8bw::kNormMaxCols) return 0;
  return align_up(fp8bw::rms_norm_bwd_ws_bytes(rows, cols));
}

FP8BW_API int fp8bw_rms_norm_bwd(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s,
                                 const float* rstd, const void* weight, int weight_dtype,
                                 const void* dres, int64_t ld_dres, int64_t rows, int64_t cols,
                                 void* dx, int64_t ld_dx, void* dweight, void* ws, size_t ws_bytes,
                                 void* stream) {
  int st = check_norm(rows, cols, weight_dtype);
  if (st != FP8BW_OK) return st;
  if (rows == 0 || cols == 0) return ok();
  if ((st = check_bf16(dy, rows, cols, ld_dy, "dy")) != FP8BW_OK) return st;
  if ((st = check_bf16(s, rows, cols, ld_s, "s")) != FP8BW_OK) return st;
  if ((st = check_f32(rstd, "rstd")) != FP8BW_OK) return st;
  if ((st = check_weight(weight)) != FP8BW_OK) return st;
  if (dres && (st = check_bf16(dres, rows, cols, ld_dres, "dres")) != FP8BW_OK) return st;
  if ((st = check_bf16(dx, rows, cols, ld_dx, "dx")) != FP8BW_OK) return st;
  if (!dweight) return fail(FP8BW_ERR_NULL, "dweight must be non-null");
  if (!aligned(dweight, 4)) return fail(FP8BW_ERR_ALIGN, "dweight must be 4-byte aligned");
  const size_t need = fp8bw_rms_norm_bwd_ws_bytes(rows, cols);
  if (!ws || ws_bytes < need) return fail(FP8BW_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned(ws, 16)) return fail(FP8BW_ERR_ALIGN, "ws must be 16-byte aligned");
  fp8bw::NormBwdArgs p = {};
  p.rows = rows; p.cols = cols;
  p.dy = (const uint16_t*)dy; p.ld_dy = used_stride(rows, ld_dy);
  p.s = (const uint16_t*)s; p.ld_s = used_stride(rows, ld_s);
  p.rstd = rstd;
  p.weight.p = weight; p.weight.f32 = weight_dtype == FP8BW_OUT_F32;
  p.dres = (const uint16_t*)dres; p.ld_dres = used_stride(rows, ld_dres);
  p.dx = (uint16_t*)dx; p.ld_dx = used_stride(rows, ld_dx);
  p.dweight = dweight;
  p.partial = (float*)ws;
  return hip_status(fp8bw::launch_rms_norm_bwd(p, (hipStream_t)stream), "fp8bw_rms_norm_bwd");
}

// ---------------------------------------------------------------------------
// Linear cross entropy.

namespace {

// A launch has fewer than 2^32 threads, 512 a tile.
constexpr int64_t kXentMaxTiles = (int64_t)1 << 23;
constexpr int64_t kXentMaxT = (int64_t)1 << 24, kXentMaxV = (int64_t)1 << 28, kXentMaxK = (int64_t)1 << 20;

bool xent_dims_ok(int64_t T, int64_t V, int64_t K) {
  return T >= 0 && V >= 0 && T <= kXentMaxT && V <= kXentMaxV && K >= 64 && K <= kXentMaxK && K % 64 == 0 &&
         cdiv(T, 256) * cdiv(V, 256) < kXentMaxTiles && cdiv(T, 256) * cdiv(K, 256) < kXentMaxTiles &&
         cdiv(V, 256) * cdiv(K, 256) < kXentMaxTiles;
}

// The products address a tile of 256 rows with 32-bit byte offsets.
int check_xent_operand(const void* p, int64_t rows, int64_t K, int64_t ld, const char* name) {
  const int st = check_bf16(p, rows, K, ld, name);
  if (st != FP8BW_OK) return st;
  if (rows > 1 && ld > ((int64_t)1 << 22) - K / 128)
    return fail(FP8BW_ERR_LAYOUT, "leading dimension %lld of %s too large", (long long)ld, name);
  return FP8BW_OK;
}

int check_xent(const void* h, int64_t ld_h, const void* w, int64_t ld_w, const int64_t* target, int64_t T,
               int64_t V, int64_t K) {
  if (!xent_dims_ok(T, V, K))
    return fail(FP8BW_ERR_SHAPE,
                "T=%lld V=%lld K=%lld: K must be a multiple of 64 in [64, 2^20], V <= 2^28, T <= 2^24, "
                "ceil(a / 256) ceil(b / 256) < 2^23 for any two of them",
                (long long)T, (long long)V, (long long)K);
  if (T == 0) return FP8BW_OK;
  if (V == 0) return fail(FP8BW_ERR_SHAPE, "an empty vocabulary has no cross entropy");
  int st;
  if ((st = check_xent_operand(h, T, K, ld_h, "h")) != FP8BW_OK) return st;
  if ((st = check_xent_operand(w, V, K, ld_w, "w")) != FP8BW_OK) return st;
  if (!target) return fail(FP8BW_ERR_NULL, "target must be non-null");
  if (!aligned(target, 8)) return fail(FP8BW_ERR_ALIGN, "target must be 8-byte aligned");
  return FP8BW_OK;
}

int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return fail(FP8BW_ERR_WORKSPACE, "workspace needs %zu bytes", need);
  if (!aligned(ws, 256)) return fail(FP8BW_ERR_ALIGN, "ws must be 256-byte aligned");
  return FP8BW_OK;
}

}  // namespace

FP8BW_API size_t fp8bw_linear_xent_ws_bytes(int64_t T, int64_t V, int64_t K, int backward) {
  if (T <= 0 || V <= 0 || !xent_dims_ok(T, V, K)) return 0;
  return fp8bw::xent_ws_bytes(T, V, K, backward != 0);
}

FP8BW_API int fp8bw_linear_xent_fwd(const void* h, int64_t ld_h, const void* w, int64_t ld_w,
                                    const int64_t* target, int64_t ignore_index, int64_t T, int64_t V,
                                    int64_t K, float* loss, float* lse, void* ws, size_t ws_bytes,
                                    void* stream) {
  int st = check_xent(h, ld_h, w, ld_w, target, T, V, K);
  if (st != FP8BW_OK) return st;
  if (T == 0) return ok();
  if ((st = check_f32(loss, "loss")) != FP8BW_OK) return st;
  if ((st = check_f32(lse, "lse")) != FP8BW_OK) return st;
  if ((st = check_ws(ws, ws_bytes, fp8bw_linear_xent_ws_bytes(T, V, K, 0))) != FP8BW_OK) return st;
  fp8bw::XentArgs p = {};
  p.T = T; p.V = V; p.K = K;
  p.h = h; p.ld_h = T > 1 ? ld_h : K;
  p.w = w; p.ld_w = V > 1 ? ld_w : K;
  p.target = target; p.ignore_index = ignore_index;
  p.loss = loss; p.lse = lse;
  return hip_status(fp8bw::launch_xent_fwd(p, ws, (hipStream_t)stream), "fp8bw_linear_xent_fwd");
}

FP8BW_API int fp8bw_linear_xent_bwd(const float* dloss, const void* h, int64_t ld_h, const void* w,
                                    int64_t ld_w, const int64_t* target, int64_t ignore_index,
                                    const float* lse, int64_t T, int64_t V, int64_t K, void* dh,
                                    int64_t ld_dh, void* dw, int64_t ld_dw, void* ws, size_t ws_bytes,
                                    void* stream) {
  return fp8bw_linear_xent_bwd_loss(dloss, h, ld_h, w, ld_w, target, ignore_index, lse, nullptr, T, V, K, dh,
                                    ld_dh, dw, ld_dw, ws, ws_bytes, stream);
}

FP8BW_API int fp8bw_linear_xent_bwd_loss(const float* dloss, const void* h, int64_t ld_h, const void* w,
                                         int64_t ld_w, const int64_t* target, int64_t ignore_index,
                                         const float* lse, const float* loss, int64_t T, int64_t V,
                                         int64_t K, void* dh, int64_t ld_dh, void* dw, int64_t ld_dw,
                                         void* ws, size_t ws_bytes, void* stream) {
  int st = check_xent(h, ld_h, w, ld_w, target, T, V, K);
  if (st != FP8BW_OK) return st;
  if (dw && V > 0 && (st = check_bf16(dw, V, K, ld_dw, "dw")) != FP8BW_OK) return st;
  if (T == 0) {
    if (!dw || V == 0) return ok();
    return hip_status(fp8bw::launch_zero_rows_bf16(dw, V, K, V > 1 ? ld_dw : K, (hipStream_t)stream),
                      "fp8bw_linear_xent_bwd");
  }
  if (dh && (st = check_bf16(dh, T, K, ld_dh, "dh")) != FP8BW_OK) return st;
  if ((st = check_f32(dloss, "dloss")) != FP8BW_OK) return st;
  if ((st = check_f32(lse, "lse")) != FP8BW_OK) return st;
  if (loss && (st = check_f32(loss, "loss")) != FP8BW_OK) return st;
  if (!dh && !dw) return ok();
  if ((st = check_ws(ws, ws_bytes, fp8bw_linear_xent_ws_bytes(T, V, K, 1))) != FP8BW_OK) return st;
  fp8bw::XentArgs p = {};
  p.T = T; p.V = V; p.K = K;
  p.h = h; p.ld_h = T > 1 ? ld_h : K;
  p.w = w; p.ld_w = V > 1 ? ld_w : K;
  p.target = target; p.ignore_index = ignore_index;
  p.lse = const_cast<float*>(lse);
  p.dloss = dloss;
  p.nll = loss;
  p.dh = dh; p.ld_dh = T > 1 ? ld_dh : K;
  p.dw = dw; p.ld_dw = V > 1 ? ld_dw : K;
  return hip_status(fp8bw::launch_xent_bwd(p, ws, (hipStream_t)stream), "fp8bw_linear_xent_bwd");
}

// ---------------------------------------------------------------------------
// AdamW.

namespace {

int check_adamw_tensor(const fp8bw_adamw_tensor& t, int i, bool eight) {
  auto type_ok = [](int d) { return d == FP8BW_OUT_BF16 || d == FP8BW_OUT_F32; };
  // At most 2^24 workgroups of 2048 elements a launch (2^32 threads).
  if (t.numel < 0 || t.numel >= ((int64_t)1 << 35)) return fail(FP8BW_ERR_SHAPE, "tensor %d: numel %lld", i, (long long)t.numel);
  if (!type_ok(t.param_dtype) || !type_ok(t.grad_dtype)) return fail(FP8BW_ERR_UNSUPPORTED, "tensor %d: unknown type", i);
  if (t.master && t.param_dtype != FP8BW_OUT_BF16)
    return fail(FP8BW_ERR_UNSUPPORTED, "tensor %d: a master belongs to a bf16 parameter", i);
  if (t.numel == 0) return FP8BW_OK;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return fail(FP8BW_ERR_NULL, "tensor %d: null pointer", i);
  if (eight && (!t.exp_avg_scale || !t.root_scale)) return fail(FP8BW_ERR_NULL, "tensor %d: 8-bit states need scales", i);
  if (!eight && (t.exp_avg_scale || t.root_scale))
    return fail(FP8BW_ERR_UNSUPPORTED, "tensor %d: fp32 states take no scales", i);
  const size_t ps = t.param_dtype == FP8BW_OUT_F32 ? 4 : 2, gs = t.grad_dtype == FP8BW_OUT_F32 ? 4 : 2;
  const size_t ss = eight ? 1 : 4;
  if (!aligned(t.param, ps) || !aligned(t.grad, gs) || !aligned(t.exp_avg, ss) || !aligned(t.exp_avg_sq, ss) ||
      !aligned(t.exp_avg_scale, 4) || !aligned(t.root_scale, 4) || !aligned(t.master, 4))
    return fail(FP8BW_ERR_ALIGN, "tensor %d: a pointer is not aligned to its elements", i);
  return FP8BW_OK;
}

}  // namespace

FP8BW_API int fp8bw_adamw_step(const fp8bw_adamw_tensor* tensors, int count, int state, int64_t step,
                               double lr, double beta1, double beta2, double eps, double weight_decay,
                               const float* grad_scale, int stochastic, uint64_t seed, void* stream) {
  if (count < 0) return fail(FP8BW_ERR_SHAPE, "negative count");
  if (state != FP8BW_STATE_F32 && state != FP8BW_STATE_E4M3) return fail(FP8BW_ERR_UNSUPPORTED, "unknown state %d", state);
  if (step < 1) return fail(FP8BW_ERR_SHAPE, "step=%lld counts from 1", (long long)step);
  if (!(lr >= 0) || !(eps >= 0) || !(weight_decay >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) ||
      !std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay))
    return fail(FP8BW_ERR_UNSUPPORTED, "lr, eps and weight_decay must be >= 0, beta1 and beta2 in [0, 1)");
  if (count == 0) return ok();
  if (!tensors) return fail(FP8BW_ERR_NULL, "tensors must be non-null");
  if (!aligned(grad_scale, 4)) return fail(FP8BW_ERR_ALIGN, "grad_scale must be 4-byte aligned");
  const bool eight = state == FP8BW_STATE_E4M3;
  constexpr int64_t kManyElements = (int64_t)1 << 23;
  int64_t total = 0;   // up to kManyElements
  for (int i = 0; i < count; ++i) {
    const int st = check_adamw_tensor(tensors[i], i, eight);
    if (st != FP8BW_OK) return st;
    if (total < kManyElements) total += tensors[i].numel;
  }
  fp8bw::AdamwLaunch L = {};
  L.grad_scale = grad_scale;
  L.beta1 = (float)beta1;
  L.one_minus_beta1 = (float)(1 - beta1);
  L.beta2 = (float)beta2;
  L.one_minus_beta2 = (float)(1 - beta2);
  L.decay = (float)(1 - lr * weight_decay);
  L.step_size = (float)(lr / (1 - std::pow(beta1, (double)step)));
  L.root_factor = (float)(1 / std::sqrt(1 - std::pow(beta2, (double)step)));
  L.eps = (float)eps;
  // Runs of 2048 elements per workgroup: four once that still leaves the chip
  // several workgroups per compute unit, so that the search for the tensor and
  // the first loads' latency are paid once for them.
  L.iters = total >= kManyElements ? 4 : 1;
  const int64_t chunk = (int64_t)2048 * L.iters;
  int64_t groups = 0;
  auto flush = [&]() -> hipError_t {
    const hipError_t e = L.count > 0 ? fp8bw::launch_adamw(L, (int)groups, eight, stochastic != 0, (hipStream_t)stream)
                                     : hipSuccess;
    L.count = 0;
    groups = 0;
    return e;
  };
  for (int i = 0; i < count; ++i) {
    const fp8bw_adamw_tensor& t = tensors[i];
    if (t.numel == 0) continue;
    const int64_t n = cdiv(t.numel, chunk);
    if (L.count == fp8bw::kAdamwTensors || groups + n >= ((int64_t)1 << 24)) {
      const hipError_t e = flush();
      if (e != hipSuccess) return hip_status(e, "fp8bw_adamw_step");
    }
    fp8bw::AdamwTensor& d = L.t[L.count];
    d.param = t.param; d.grad = t.grad; d.m = t.exp_avg; d.v = t.exp_avg_sq;
    d.m_scale = t.exp_avg_scale; d.root_scale = t.root_scale; d.master = t.master;
    d.numel = t.numel;
    d.key = fp8bw::adamw_key(seed, i);
    d.flags = (t.param_dtype == FP8BW_OUT_F32 ? fp8bw::kAdamwParamF32 : 0) |
              (t.grad_dtype == FP8BW_OUT_F32 ? fp8bw::kAdamwGradF32 : 0);
    L.first[L.count++] = (int)groups;
    groups += n;
  }
  return hip_status(flush(), "fp8bw_adamw_step");
}
