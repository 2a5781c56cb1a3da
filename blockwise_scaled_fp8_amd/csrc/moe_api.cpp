// C ABI of the mixture-of-experts operators: sort, gather and combine, the
// gated activation, the grouped weight gradient and the grouped quantizer.
// Validation and dispatch only; the contracts are in include/fp8bw.h.

#include <initializer_list>

#include "check.h"
#include "launch.h"

using namespace fp8bw::api;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 24, kMaxRows = (int64_t)1 << 27;
// A launch has fewer than 2^32 threads: 64 a piece of 512 columns, 512 a tile.
constexpr int64_t kMaxPieces = (int64_t)1 << 26, kMaxTiles = (int64_t)1 << 23;

bool sort_dims_ok(int64_t tokens, int64_t topk, int64_t experts, int64_t align) {
  return tokens >= 0 && tokens < kMaxTokens && topk >= 1 && topk <= fp8bw::kMoeMaxTopk && experts >= 1 &&
         experts <= fp8bw::kMoeMaxExperts && align >= 1 && align <= 65536;
}

int check_i32(const void* p, const char* name) {
  if (!p) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  if (!aligned(p, 4)) return fail(FP8BW_ERR_ALIGN, "%s must be 4-byte aligned", name);
  return FP8BW_OK;
}

// The layouts of a [rows, cols] result whose 1x128 row blocks number `blocks`.
int check_layouts(const fp8bw_layouts* o, int64_t rows, int64_t cols, int64_t blocks) {
  if (!o) return fail(FP8BW_ERR_NULL, "the output layouts must be non-null");
  int st = FP8BW_OK;
  if (o->y && (st = check_bf16(o->y, rows, cols, o->ld_y, "y")) != FP8BW_OK) return st;
  if (o->q && (st = check_codes(o->q, rows, cols, o->ld_q, o->recip, o->rs_row, o->rs_kb, "q", blocks)) != FP8BW_OK)
    return st;
  if (o->qt) {
    if (rows % 16) return fail(FP8BW_ERR_SHAPE, "transposed codes need rows %% 16 == 0 (rows=%lld)", (long long)rows);
    st = check_codes(o->qt, cols, rows, o->ld_qt, o->recip_t, o->rst_row, o->rst_kb, "qt");
  }
  return st;
}

fp8bw::LayoutsOut layouts(const fp8bw_layouts& o, int64_t rows, int64_t cols, int64_t blocks) {
  fp8bw::LayoutsOut r = {};
  r.y = (uint16_t*)o.y; r.ld_y = used_stride(rows, o.ld_y);
  r.q = (uint8_t*)o.q; r.ld_q = used_stride(rows, o.ld_q);
  r.recip = o.recip; r.rs_row = used_stride(rows, o.rs_row); r.rs_kb = used_stride(blocks, o.rs_kb);
  r.qt = (uint8_t*)o.qt; r.ld_qt = used_stride(cols, o.ld_qt);
  r.recip_t = o.recip_t; r.rst_row = used_stride(cols, o.rst_row);
  r.rst_kb = used_stride(cdiv(rows, 128), o.rst_kb);
  return r;
}

// A tile's 128 rows are addressed with 32-bit byte offsets from its corner.
int check_tile_strides(std::initializer_list<int64_t> bf16_or_f32, std::initializer_list<int64_t> codes) {
  for (int64_t s : bf16_or_f32)
    if (s >= ((int64_t)1 << 22)) return fail(FP8BW_ERR_LAYOUT, "transposed codes need strides below 2^22 (%lld)", (long long)s);
  for (int64_t s : codes)
    if (s >= ((int64_t)1 << 24)) return fail(FP8BW_ERR_LAYOUT, "transposed codes need strides of codes below 2^24 (%lld)", (long long)s);
  return FP8BW_OK;
}

// Launch sizes of a [rows, cols] result and, with them, `tokens` rows read or written.
int check_size(int64_t tokens, int64_t rows, int64_t cols) {
  const int64_t pieces = cdiv(cols, 512);
  if (tokens * pieces >= kMaxPieces || rows * pieces >= kMaxPieces * 16 ||
      cdiv(rows, 128) * cdiv(cols, 128) >= kMaxTiles)
    return fail(FP8BW_ERR_SHAPE, "%lld rows of %lld columns are more than one launch takes",
                (long long)(tokens > rows ? tokens : rows), (long long)cols);
  return FP8BW_OK;
}

int check_table(int64_t tokens, int64_t topk, int64_t rows, int64_t cols) {
  if (tokens < 0 || rows < 0 || cols < 0) return fail(FP8BW_ERR_SHAPE, "negative dimension");
  if (topk < 1 || topk > fp8bw::kMoeMaxTopk)
    return fail(FP8BW_ERR_SHAPE, "topk=%lld must be in [1, %d]", (long long)topk, fp8bw::kMoeMaxTopk);
  if (tokens >= kMaxTokens || rows >= kMaxRows)
    return fail(FP8BW_ERR_SHAPE, "tokens=%lld must be below 2^24 and rows=%lld below 2^27", (long long)tokens,
                (long long)rows);
  if (cols % 16 || cols > 65536)
    return fail(FP8BW_ERR_SHAPE, "cols=%lld must be a multiple of 16 and at most 65536", (long long)cols);
  if ((tokens == 0) != (rows == 0))
    return fail(FP8BW_ERR_SHAPE, "tokens=%lld with rows=%lld", (long long)tokens, (long long)rows);
  return check_size(tokens, rows, cols);
}

int check_weight(const void* w, int dtype) {
  if (dtype != FP8BW_OUT_BF16 && dtype != FP8BW_OUT_F32)
    return fail(FP8BW_ERR_UNSUPPORTED, "unknown weight type %d", dtype);
  if (!aligned(w, dtype == FP8BW_OUT_F32 ? 4 : 2))
    return fail(FP8BW_ERR_ALIGN, "weight must be aligned to its elements");
  return FP8BW_OK;
}

int check_swiglu(int64_t rows, int64_t ffn) {
  if (rows < 0 || ffn < 0) return fail(FP8BW_ERR_SHAPE, "negative dimension");
  if (ffn % 16 || ffn > ((int64_t)1 << 20))
    return fail(FP8BW_ERR_SHAPE, "ffn=%lld must be a multiple of 16 and at most 2^20", (long long)ffn);
  if (rows >= kMaxRows) return fail(FP8BW_ERR_SHAPE, "rows=%lld must be below 2^27", (long long)rows);
  return check_size(rows, rows, ffn);
}

}  // namespace

FP8BW_API int64_t fp8bw_moe_rows(int64_t tokens, int64_t topk, int64_t experts, int64_t align) {
  if (!sort_dims_ok(tokens, topk, experts, align)) return 0;
  const int64_t n = tokens * topk, filled = experts < n ? experts : n;
  const int64_t rows = align * (filled + (n - filled) / align);
  return rows < kMaxRows ? rows : 0;
}

FP8BW_API size_t fp8bw_moe_sort_ws_bytes(int64_t tokens, int64_t topk, int64_t experts) {
  if (!sort_dims_ok(tokens, topk, experts, 1)) return 0;
  return align_up(fp8bw::moe_sort_ws_bytes(tokens * topk, (int)experts));
}

FP8BW_API int fp8bw_moe_sort(const void* expert, int index_bits, int64_t tokens, int64_t topk,
                             int64_t experts, int64_t align, int64_t rows, int32_t* row,
                             int32_t* source, int32_t* group_end, void* ws, size_t ws_bytes,
                             void* stream) {
  if (index_bits != 32 && index_bits != 64)
    return fail(FP8BW_ERR_UNSUPPORTED, "index_bits=%d must be 32 or 64", index_bits);
  if (!sort_dims_ok(tokens, topk, experts, align))
    return fail(FP8BW_ERR_SHAPE,
                "tokens=%lld topk=%lld experts=%lld align=%lld: tokens must be in [0, 2^24), topk in [1, %d], experts "
                "in [1, %d], align in [1, 65536]",
                (long long)tokens, (long long)topk, (long long)experts, (long long)align, fp8bw::kMoeMaxTopk,
                fp8bw::kMoeMaxExperts);
  const int64_t need = fp8bw_moe_rows(tokens, topk, experts, align);
  if (rows >= kMaxRows || (need == 0 && tokens > 0))
    return fail(FP8BW_ERR_SHAPE, "2^27 rows or more");
  if (rows < need) return fail(FP8BW_ERR_SHAPE, "rows=%lld: the slots may need %lld", (long long)rows, (long long)need);
  int st;
  if ((st = check_i32(group_end, "group_end")) != FP8BW_OK) return st;
  if (tokens > 0) {
    if (!expert) return fail(FP8BW_ERR_NULL, "expert must be non-null");
    if (!aligned(expert, index_bits / 8)) return fail(FP8BW_ERR_ALIGN, "expert must be aligned to its elements");
    if ((st = check_i32(row, "row")) != FP8BW_OK) return st;
  }
  if (rows > 0 && (st = check_i32(source, "source")) != FP8BW_OK) return st;
  const size_t nws = fp8bw_moe_sort_ws_bytes(tokens, topk, experts);
  if (nws > 0 && (st = check_ws(ws, ws_bytes, nws)) != FP8BW_OK) return st;
  fp8bw::MoeSortArgs p = {};
  p.expert = expert; p.wide = index_bits == 64;
  p.n = tokens * topk;
  p.experts = (int)experts; p.align = (int)align;
  p.rows = rows;
  p.row = row; p.source = source; p.group_end = group_end;
  p.counts = (int*)ws;
  return hip_status(fp8bw::launch_moe_sort(p, (hipStream_t)stream), "fp8bw_moe_sort");
}

namespace {

int moe_gather(const void* x, int64_t ld_x, const void* y, int64_t ld_y, const void* weight, int weight_dtype,
               int64_t tokens, int64_t topk, const int32_t* row, const int32_t* source, int64_t rows,
               int64_t cols, const fp8bw_layouts* out, void* dweight, void* stream, const char* x_name,
               const char* what) {
  int st = check_table(tokens, topk, rows, cols);
  if (st != FP8BW_OK) return st;
  if (tokens == 0 || cols == 0) return ok();
  if ((st = check_bf16(x, tokens, cols, ld_x, x_name)) != FP8BW_OK) return st;
  if ((st = check_i32(row, "row")) != FP8BW_OK) return st;
  if ((st = check_i32(source, "source")) != FP8BW_OK) return st;
  if ((st = check_weight(weight, weight_dtype)) != FP8BW_OK) return st;
  const int64_t blocks = cdiv(cols, 128);
  if ((st = check_layouts(out, rows, cols, blocks)) != FP8BW_OK) return st;
  if (dweight) {
    if ((st = check_bf16(y, rows, cols, ld_y, "y")) != FP8BW_OK) return st;
    if ((st = check_weight(dweight, weight_dtype)) != FP8BW_OK) return st;
  }
  fp8bw::MoeGatherArgs p = {};
  p.table.tokens = tokens; p.table.rows = rows; p.table.topk = (int)topk;
  p.table.row = row; p.table.source = source;
  p.cols = cols;
  p.x = (const uint16_t*)x; p.ld_x = used_stride(tokens, ld_x);
  p.weight.p = weight; p.weight.f32 = weight_dtype == FP8BW_OUT_F32;
  p.out = layouts(*out, rows, cols, blocks);
  p.y = (const uint16_t*)y; p.ld_y = used_stride(rows, ld_y);
  p.dweight = dweight;
  if (p.out.qt && (st = check_tile_strides({p.out.y ? p.out.ld_y : 0}, {p.out.q ? p.out.ld_q : 0, p.out.ld_qt})) != FP8BW_OK)
    return st;
  return hip_status(fp8bw::launch_moe_gather(p, (hipStream_t)stream), what);
}

}  // namespace

FP8BW_API int fp8bw_moe_gather(const void* x, int64_t ld_x, int64_t tokens, int64_t topk,
                               const int32_t* row, const int32_t* source, int64_t rows, int64_t cols,
                               const fp8bw_layouts* out, void* stream) {
  return moe_gather(x, ld_x, nullptr, 0, nullptr, FP8BW_OUT_F32, tokens, topk, row, source, rows, cols, out, nullptr,
                    stream, "x", "fp8bw_moe_gather");
}

FP8BW_API int fp8bw_moe_combine(const void* y, int64_t ld_y, const void* weight, int weight_dtype,
                                int64_t tokens, int64_t topk, const int32_t* row, int64_t rows,
                                int64_t cols, void* out, int64_t ld_out, void* stream) {
  int st = check_table(tokens, topk, rows, cols);
  if (st != FP8BW_OK) return st;
  if (tokens == 0 || cols == 0) return ok();
  if ((st = check_bf16(y, rows, cols, ld_y, "y")) != FP8BW_OK) return st;
  if ((st = check_weight(weight, weight_dtype)) != FP8BW_OK) return st;
  if ((st = check_i32(row, "row")) != FP8BW_OK) return st;
  if ((st = check_bf16(out, tokens, cols, ld_out, "out")) != FP8BW_OK) return st;
  fp8bw::MoeCombineArgs p = {};
  p.table.tokens = tokens; p.table.rows = rows; p.table.topk = (int)topk;
  p.table.row = row;
  p.cols = cols;
  p.y = (const uint16_t*)y; p.ld_y = used_stride(rows, ld_y);
  p.weight.p = weight; p.weight.f32 = weight_dtype == FP8BW_OUT_F32;
  p.out = (uint16_t*)out; p.ld_out = used_stride(tokens, ld_out);
  return hip_status(fp8bw::launch_moe_combine(p, (hipStream_t)stream), "fp8bw_moe_combine");
}

FP8BW_API int fp8bw_moe_combine_bwd(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y,
                                    const void* weight, int weight_dtype, int64_t tokens, int64_t topk,
                                    const int32_t* row, const int32_t* source, int64_t rows,
                                    int64_t cols, const fp8bw_layouts* dy, void* dweight, void* stream) {
  // An empty sum: every weight's gradient is zero, and there may be no columns to read.
  if (dweight && cols == 0 && tokens > 0)
    return fail(FP8BW_ERR_SHAPE, "the weights' gradient needs columns");
  return moe_gather(dout, ld_dout, y, ld_y, weight, weight_dtype, tokens, topk, row, source, rows, cols, dy, dweight,
                    stream, "dout", "fp8bw_moe_combine_bwd");
}

FP8BW_API int fp8bw_swiglu_fwd(const void* h, int64_t ld_h, int64_t rows, int64_t ffn,
                               const fp8bw_layouts* out, void* hq, int64_t ld_hq, float* h_recip,
                               int64_t hr_row, int64_t hr_kb, void* stream) {
  int st = check_swiglu(rows, ffn);
  if (st != FP8BW_OK) return st;
  if (rows == 0 || ffn == 0) return ok();
  const int64_t blocks = cdiv(ffn, 128);
  if ((st = check_bf16(h, rows, 2 * ffn, ld_h, "h")) != FP8BW_OK) return st;
  if ((st = check_layouts(out, rows, ffn, blocks)) != FP8BW_OK) return st;
  if (hq && (st = check_codes(hq, rows, 2 * ffn, ld_hq, h_recip, hr_row, hr_kb, "hq", 2 * blocks)) != FP8BW_OK)
    return st;
  if (!out->y && !out->q && !out->qt && !hq) return ok();
  fp8bw::SwigluFwdArgs p = {};
  p.rows = rows; p.ffn = ffn;
  p.h = h; p.ld_h = used_stride(rows, ld_h);
  p.out = layouts(*out, rows, ffn, blocks);
  p.hq = (uint8_t*)hq; p.ld_hq = used_stride(rows, ld_hq);
  p.h_recip = h_recip; p.hr_row = used_stride(rows, hr_row); p.hr_kb = hr_kb;
  if (p.out.qt && (st = check_tile_strides({p.ld_h}, {p.out.ld_qt})) != FP8BW_OK) return st;
  return hip_status(fp8bw::launch_swiglu_fwd(p, (hipStream_t)stream), "fp8bw_swiglu_fwd");
}

FP8BW_API int fp8bw_swiglu_bwd(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h,
                               const float* h_recip, int64_t hr_row, int64_t hr_kb, int64_t rows,
                               int64_t ffn, const fp8bw_layouts* dh, void* act_qt, int64_t ld_act_qt,
                               float* act_recip_t, int64_t art_row, int64_t art_kb, void* stream) {
  int st = check_swiglu(rows, ffn);
  if (st != FP8BW_OK) return st;
  if (rows == 0 || ffn == 0) return ok();
  const int64_t blocks = cdiv(ffn, 128);
  // (without an output of dh nothing reads dy)
  const bool grads = dh && (dh->y || dh->q || dh->qt);
  if ((dy || grads) && (st = check_bf16(dy, rows, ffn, ld_dy, "dy")) != FP8BW_OK) return st;
  if (h_recip) {
    if (!h) return fail(FP8BW_ERR_NULL, "h must be non-null");
    st = check_codes(h, rows, 2 * ffn, ld_h, h_recip, hr_row, hr_kb, "h", 2 * blocks);
  } else {
    st = check_bf16(h, rows, 2 * ffn, ld_h, "h");
  }
  if (st != FP8BW_OK) return st;
  if ((st = check_layouts(dh, rows, 2 * ffn, 2 * blocks)) != FP8BW_OK) return st;
  if (act_qt) {
    if (rows % 16) return fail(FP8BW_ERR_SHAPE, "transposed codes need rows %% 16 == 0 (rows=%lld)", (long long)rows);
    if ((st = check_codes(act_qt, ffn, rows, ld_act_qt, act_recip_t, art_row, art_kb, "act_qt")) != FP8BW_OK) return st;
  }
  if (!grads && !act_qt) return ok();
  fp8bw::SwigluBwdArgs p = {};
  p.rows = rows; p.ffn = ffn;
  p.dy = (const uint16_t*)dy; p.ld_dy = used_stride(rows, ld_dy);
  p.h = h; p.ld_h = used_stride(rows, ld_h);
  p.h_recip = h_recip; p.hr_row = used_stride(rows, hr_row); p.hr_kb = hr_kb;
  p.dh = layouts(*dh, rows, 2 * ffn, 2 * blocks);
  p.act_qt = (uint8_t*)act_qt; p.ld_act_qt = ld_act_qt;
  p.act_recip_t = act_recip_t; p.art_row = art_row; p.art_kb = used_stride(cdiv(rows, 128), art_kb);
  if ((p.dh.qt || act_qt) &&
      (st = check_tile_strides({grads ? p.ld_dy : 0, h_recip ? 0 : p.ld_h, h_recip ? p.hr_row : 0, p.dh.y ? p.dh.ld_y : 0},
                               {h_recip ? p.ld_h : 0, p.dh.q ? p.dh.ld_q : 0, p.dh.qt ? p.dh.ld_qt : 0,
                                act_qt ? ld_act_qt : 0})) != FP8BW_OK)
    return st;
  return hip_status(fp8bw::launch_swiglu_bwd(p, (hipStream_t)stream), "fp8bw_swiglu_bwd");
}

namespace {

int check_wgrad_operand(const void* q, int64_t rows, int64_t K, int64_t ld, const float* recip, int64_t s_row,
                        int64_t s_kb, const char* name) {
  if (!q) return fail(FP8BW_ERR_NULL, "%s must be non-null", name);
  return check_codes(q, rows, K, ld, recip, s_row, s_kb, name);
}

}  // namespace

FP8BW_API size_t fp8bw_grouped_wgrad_ws_bytes(int64_t M, int64_t N, int64_t K, int groups) {
  if (groups < 1 || groups > (1 << 20) || M <= 0 || N <= 0 || K <= 0 || K % 128 || M > kMaxDim || N > kMaxDim ||
      K > kMaxDim)
    return 0;
  fp8bw::GemmProblem p = {};
  p.M = M; p.N = N; p.K = K;
  return align_up(fp8bw::grouped_wgrad_ws_bytes(p, groups));
}

FP8BW_API int fp8bw_grouped_wgrad_plan(int64_t M, int64_t N, int64_t K, int groups, int out_dtype, int64_t* info) {
  if (!info) return fail(FP8BW_ERR_NULL, "info must be non-null");
  if (out_dtype != FP8BW_OUT_BF16 && out_dtype != FP8BW_OUT_F32)
    return fail(FP8BW_ERR_UNSUPPORTED, "unknown output type %d", out_dtype);
  if (groups < 1 || groups > (1 << 20) || M <= 0 || N <= 0 || K <= 0 || M > kMaxDim || N > kMaxDim || K > kMaxDim ||
      K % 128)
    return fail(FP8BW_ERR_SHAPE, "plan needs 0 < M, N, K <= 2^30, K %% 128 == 0 and groups in [1, 2^20]");
  fp8bw::GemmProblem p = {};
  p.M = M; p.N = N; p.K = K; p.lda = K; p.ldb = K; p.ldo = N;
  p.ra_s_row = 1; p.ra_s_kb = M;
  p.rb_s_row = 1; p.rb_s_kb = N;
  p.mode = fp8bw::kBlockB1x128;
  p.out_kind = out_dtype == FP8BW_OUT_BF16 ? fp8bw::kOutBf16 : fp8bw::kOutF32;
  if (!fp8bw::grouped_wgrad_ok(p, groups))
    return fail(FP8BW_ERR_UNSUPPORTED, "%d groups of [%lld, %lld] are more output tiles than one launch takes", groups,
                (long long)M, (long long)N);
  const fp8bw::WgradRun w = fp8bw::grouped_wgrad_run(p, groups, groups > 1 ? M * N : 0);
  info[0] = w.cfg;
  info[1] = w.splits;
  info[2] = w.tiles;
  info[3] = w.stream;
  return ok();
}

FP8BW_API int fp8_scaled_grouped_gemm_blockwise_wgrad(
    const void* a, int64_t lda, const float* ra, int64_t ra_s_row, int64_t ra_s_kb, const void* b,
    int64_t ldb, const float* rb, int64_t rb_s_row, int64_t rb_s_kb, int groups, const int* group_end,
    int64_t M, int64_t N, int64_t K, void* out, int64_t ldo, int64_t out_s_group, int out_dtype,
    void* ws, size_t ws_bytes, void* stream) {
  if (groups < 1 || groups > (1 << 20)) return fail(FP8BW_ERR_SHAPE, "groups=%d must be in [1, 2^20]", groups);
  if (M < 0 || N < 0 || K < 0) return fail(FP8BW_ERR_SHAPE, "negative dimension");
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return fail(FP8BW_ERR_SHAPE, "dimension too large");
  if (K % 128) return fail(FP8BW_ERR_SHAPE, "blockwise GEMM needs K %% 128 == 0 (K=%lld)", (long long)K);
  if (out_dtype != FP8BW_OUT_BF16 && out_dtype != FP8BW_OUT_F32)
    return fail(FP8BW_ERR_UNSUPPORTED, "unknown output type %d", out_dtype);
  if (M == 0 || N == 0) return ok();
  int st;
  if ((st = check_i32(group_end, "group_end")) != FP8BW_OK) return st;
  if (!out) return fail(FP8BW_ERR_NULL, "out must be non-null");
  if (!aligned(out, 16)) return fail(FP8BW_ERR_ALIGN, "out must be 16-byte aligned");
  if (ldo < N || !extent_ok(M, ldo, N)) return fail(FP8BW_ERR_LAYOUT, "ldo=%lld not allowed", (long long)ldo);
  const int64_t extent = (M - 1) * ldo + N;
  if (groups > 1 && (out_s_group < extent || out_s_group > (kMaxExtent - extent) / (groups - 1)))
    return fail(FP8BW_ERR_LAYOUT, "out_s_group=%lld must be >= (M-1)*ldo + N, and the groups below 2^48 elements",
                (long long)out_s_group);
  const int64_t kb = K / 128;
  if (kb > 0) {
    if ((st = check_wgrad_operand(a, M, K, lda, ra, ra_s_row, ra_s_kb, "a")) != FP8BW_OK) return st;
    if ((st = check_wgrad_operand(b, N, K, ldb, rb, rb_s_row, rb_s_kb, "b")) != FP8BW_OK) return st;
  }
  fp8bw::GemmProblem p = {};
  p.a = a; p.lda = used_stride(M, lda);
  p.b = b; p.ldb = used_stride(N, ldb);
  p.ra = ra; p.ra_s_row = used_stride(M, ra_s_row); p.ra_s_kb = used_stride(kb, ra_s_kb);
  p.rb = rb; p.rb_s_row = used_stride(N, rb_s_row); p.rb_s_kb = used_stride(kb, rb_s_kb);
  p.out = out; p.ldo = ldo; p.M = M; p.N = N; p.K = K;
  p.mode = fp8bw::kBlockB1x128;
  p.out_kind = out_dtype == FP8BW_OUT_BF16 ? fp8bw::kOutBf16 : fp8bw::kOutF32;
  if (!fp8bw::grouped_wgrad_ok(p, groups))
    return fail(FP8BW_ERR_UNSUPPORTED, "%d groups of [%lld, %lld] are more output tiles than one launch takes", groups,
                (long long)M, (long long)N);
  const size_t need = align_up(fp8bw::grouped_wgrad_ws_bytes(p, groups));
  if (need > 0 && (st = check_ws(ws, ws_bytes, need)) != FP8BW_OK) return st;
  return hip_status(fp8bw::launch_grouped_wgrad(p, groups, group_end, groups > 1 ? out_s_group : 0, ws,
                                                (hipStream_t)stream),
                    "fp8_scaled_grouped_gemm_blockwise_wgrad");
}

FP8BW_API int fp8_blockwise_quant_grouped(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                          int64_t x_s_group, int groups, int transpose, void* q,
                                          int64_t ld_q, int64_t q_s_group, float* recip, int64_t rs_row,
                                          int64_t rs_kb, int64_t recip_s_group, void* stream) {
  if (groups < 1 || groups > 65535) return fail(FP8BW_ERR_SHAPE, "groups=%d must be in [1, 65535]", groups);
  if (transpose != 0 && transpose != 1) return fail(FP8BW_ERR_UNSUPPORTED, "transpose must be 0 or 1");
  if (rows < 0 || cols < 0) return fail(FP8BW_ERR_SHAPE, "negative dimension");
  if (rows > kMaxDim || cols > kMaxDim) return fail(FP8BW_ERR_SHAPE, "dimension too large");
  if (cols % 16 || (transpose && rows % 16))
    return fail(FP8BW_ERR_SHAPE, "cols=%lld, and rows=%lld with transpose, must be multiples of 16", (long long)cols,
                (long long)rows);
  if (rows == 0 || cols == 0) return ok();
  const int64_t rb = cdiv(rows, 128), cb = cdiv(cols, 128);
  if (rb > kMaxGridY || rb * cb >= ((int64_t)1 << 24) / groups) return fail(FP8BW_ERR_SHAPE, "too many blocks");
  int st = check_bf16(x, rows, cols, ld_x, "x");
  if (st != FP8BW_OK) return st;
  if (!q) return fail(FP8BW_ERR_NULL, "q must be non-null");
  const int64_t qr = transpose ? cols : rows, qc = transpose ? rows : cols;
  const int64_t ni = transpose ? cb : rb, nj = transpose ? rb : cb;
  if ((st = check_codes(q, qr, qc, ld_q, recip, 1, ni, "q", 1)) != FP8BW_OK) return st;
  if (!strides_injective(ni, nj, rs_row, rs_kb))
    return fail(FP8BW_ERR_LAYOUT, "scale strides (%lld, %lld) alias or are negative", (long long)rs_row,
                (long long)rs_kb);
  if (groups > 1) {
    const int64_t qe = (qr - 1) * used_stride(qr, ld_q) + qc;
    const int64_t re = (ni - 1) * used_stride(ni, rs_row) + (nj - 1) * used_stride(nj, rs_kb) + 1;
    const int64_t xe = (rows - 1) * used_stride(rows, ld_x) + cols;
    if (x_s_group < 0 || x_s_group % 8 || x_s_group > (kMaxExtent - xe) / (groups - 1))
      return fail(FP8BW_ERR_LAYOUT, "x_s_group=%lld must be >= 0 and a multiple of 8", (long long)x_s_group);
    if (q_s_group < qe || q_s_group % 16 || q_s_group > (kMaxExtent - qe) / (groups - 1))
      return fail(FP8BW_ERR_LAYOUT, "q_s_group=%lld must be >= %lld and a multiple of 16", (long long)q_s_group,
                  (long long)qe);
    if (recip_s_group < re || recip_s_group > (kMaxExtent - re) / (groups - 1))
      return fail(FP8BW_ERR_LAYOUT, "recip_s_group=%lld must be >= %lld", (long long)recip_s_group, (long long)re);
  }
  return hip_status(
      fp8bw::launch_quant_128x128_grouped(x, rows, cols, used_stride(rows, ld_x), groups > 1 ? x_s_group : 0, groups,
                                          transpose, q, used_stride(qr, ld_q), groups > 1 ? q_s_group : 0, recip,
                                          used_stride(ni, rs_row), used_stride(nj, rs_kb),
                                          groups > 1 ? recip_s_group : 0, (hipStream_t)stream),
      "fp8_blockwise_quant_grouped");
}
