/*
 * fp8bw.h -- C ABI of libfp8bw.so: blockwise- and tensorwise-scaled FP8
 * (OCP E4M3) quantization and GEMM for AMD MI355X (gfx950), and the operators
 * around an FP8 linear and an FP8 mixture-of-experts layer in a training step.
 *
 * Sources, cited by page title and section:
 *   [REPRO]   pytorch/ao PR "add repro for blockwise _scaled_mm
 *             investigation" -- What Changed; Findings So Far; review
 *             comments (the 1x128 x 128x128 and 1x128 x 1x128 recipes).
 *   [INTEG]   pytorch/ao PR "integrate torch._scaled_mm into
 *             Float8BlockwiseLinear and add bench script" -- Summary
 *             (reciprocal scales, column-major scale layout); Benchmarks
 *             (linear forward + backward at M16640 N5120 K8192).
 *   [GENERIC] pytorch/ao PR "add more generic kernel for fp8 blockwise
 *             scaling" -- Performance table (1x128 and 128x128 blocks).
 *   [AITER]   ROCm/aiter issue "Does gemm_a8w8 support per-tensor quant?"
 *             -- Steps to Reproduce (per-tensor quant, out = x @ w.T,
 *             dequant reference x_q.float() * x_scale).
 *   [INDUCT]  pytorch/pytorch inductor FP8 tensorwise issue -- Describe the
 *             bug (16x32x32 fp32-out tensorwise case).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Pointers marked "device" are HIP device pointers; the library never
 *    allocates, frees or copies device memory and never synchronizes the
 *    host.  Scratch comes from a caller-owned workspace sized by the
 *    matching *_ws_bytes query.  The caller owns every buffer.
 *  - `stream` is a hipStream_t (NULL = the legacy default stream).  All work
 *    is enqueued on it in order; the call returns after enqueueing.
 *  - bf16 tensors are raw 16-bit bf16 bit patterns; FP8 tensors are OCP
 *    E4M3 ("e4m3fn") codes, one byte each; scales are fp32.
 *  - Matrices are row-major with a leading dimension `ld*` in elements.
 *    Every matrix pointer must be 16-byte aligned, bf16 input leading
 *    dimensions a multiple of 8 and FP8 leading dimensions a multiple of 16
 *    (GEMM output leading dimensions only need ldo >= N).  The stride of a
 *    dimension of size 1 is ignored.  Every element offset a call can form
 *    ((rows - 1) * ld + cols of each matrix, the last scale of a strided
 *    scale grid, the last group of a grouped operand) must be below 2^48;
 *    larger ones give FP8BW_ERR_LAYOUT.
 *  - Dimensions are at most 2^30 (quantizer rows 2^32).  The GEMM and
 *    linear size queries return 0 for larger ones (the calls reject them),
 *    and fp8bw_gemm_ws_bytes_for_split returns SIZE_MAX when the size does
 *    not fit a size_t.
 *  - A *reciprocal scale* ("recip") is the dequantization multiplier: the
 *    quantizer computes s = 448 / max(amax, 1e-12) per block, stores
 *    codes = satRNE_e4m3(x * s) and recip = 1 / s (both fp32 IEEE ops),
 *    so x ~= e4m3_value(code) * recip ([INTEG] Summary; [AITER]).
 *  - Validation runs on the host before any HIP call.  A rejected call
 *    enqueues nothing and returns a status != FP8BW_OK;
 *    fp8bw_last_error() gives a message for the calling thread.  A launch
 *    failure returns FP8BW_ERR_HIP.  No exception crosses the ABI and the
 *    library prints nothing.
 *  - Zero-sized problems (rows == 0, cols == 0, M == 0 or N == 0) succeed
 *    and enqueue nothing (the tensorwise quantizer still writes its recip).
 *  - Inputs must be finite; outputs must not alias inputs.  Results for
 *    non-finite inputs are unspecified.
 */
#ifndef FP8BW_H
#define FP8BW_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8BW_OK = 0,
  FP8BW_ERR_NULL = 1,        /* a required pointer is NULL */
  FP8BW_ERR_SHAPE = 2,       /* negative or unsupported dimension */
  FP8BW_ERR_LAYOUT = 3,      /* leading dimension / scale stride not allowed */
  FP8BW_ERR_ALIGN = 4,       /* pointer or leading dimension misaligned */
  FP8BW_ERR_UNSUPPORTED = 5, /* unknown enum value or config */
  FP8BW_ERR_WORKSPACE = 6,   /* workspace NULL or too small */
  FP8BW_ERR_HIP = 7          /* a HIP launch failed */
} fp8bw_status;

typedef enum { FP8BW_BLOCK_1x128 = 0, FP8BW_BLOCK_128x128 = 1 } fp8bw_block;
typedef enum { FP8BW_OUT_BF16 = 0, FP8BW_OUT_F32 = 1 } fp8bw_out;

/* Version of this ABI (incremented on incompatible change). */
int fp8bw_abi_version(void);
/* Static string for a status code. */
const char* fp8bw_status_str(int status);
/* Message for the last rejected call on this thread ("" if none). */
const char* fp8bw_last_error(void);

/*
 * fp8_blockwise_quant -- dynamic E4M3 quantization with per-block amax
 * scales ([GENERIC] Performance table: block_shape (1,128) and (128,128);
 * [INTEG] Summary: reciprocal scales written by the quantizer itself).
 *
 *   x      device bf16 [rows, cols], leading dim ld_x.
 *   block  FP8BW_BLOCK_1x128: one scale per row per 128 columns
 *          (transpose=0), or per column per 128 rows (transpose=1: the
 *          wgrad operands dY^T, X^T).
 *          FP8BW_BLOCK_128x128: one scale per 128x128 tile (weights);
 *          transpose=1 writes W^T codes for the dgrad GEMM.  A tile's amax
 *          is orientation-independent, so these codes are exactly the
 *          transpose of the transpose=0 codes.
 *   q      device E4M3 output.  transpose=0: q[rows, cols] (ld_q >= cols).
 *          transpose=1: q = x^T [cols, rows] (ld_q >= rows).
 *   recip  device fp32 reciprocal scales, indexed by (output row or output
 *          row block i, output column block j) at recip[i*rs_row + j*rs_kb]:
 *            1x128,   transpose=0: i = row r, j = r's 128-column block
 *            1x128,   transpose=1: i = column c (output row), j = 128-row block
 *            128x128, transpose=0: i = 128-row block, j = 128-column block
 *            128x128, transpose=1: i = 128-column block, j = 128-row block
 *          Column-major ([INTEG] Summary) is rs_row = 1, rs_kb = number of
 *          i indices; any non-negative strides are accepted.
 *   Blocks at a ragged edge take their amax over the valid elements only.
 *   Requires cols % 16 == 0, and rows % 16 == 0 when transpose=1.
 */
int fp8_blockwise_quant(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int block,
                        int transpose, void* q, int64_t ld_q, float* recip, int64_t rs_row,
                        int64_t rs_kb, void* stream);

/*
 * fp8_blockwise_quant_dual -- both layouts from one read of x: the same
 * codes and scales as fp8_blockwise_quant with transpose=0 into (q, recip)
 * and with transpose=1 into (qt, recip_t), for a training step that needs
 * X and X^T (or dY and dY^T, or W and W^T) and would otherwise read the
 * bf16 tensor twice; the quantizers are the part of the fp8 linear step
 * the pages single out as slow ([INTEG] Benchmarks).
 *
 *   block    FP8BW_BLOCK_1x128: q = 1x128 blocks along the columns with
 *            recip[r*rs_row + kb*rs_kb]; qt = x^T with 1x128 blocks along
 *            the rows, recip_t[c*rst_row + mb*rst_kb].
 *            FP8BW_BLOCK_128x128: q = tile-scaled codes, recip[rb*rs_row +
 *            cb*rs_kb]; qt = their transpose, recip_t[cb*rst_row +
 *            rb*rst_kb] (the same values in the other index order).
 *   q, qt    device E4M3 [rows, cols] (ld_q >= cols) and [cols, rows]
 *            (ld_qt >= rows); the two must not overlap (checked).
 *   stream_t nonzero: qt is written with nontemporal stores, which keep the
 *            transposed codes from evicting the caches' contents (for codes
 *            read only much later, such as the X^T a training forward keeps
 *            for its backward, while q feeds the GEMM that runs next).  The
 *            same bits either way.
 *   Requires cols % 16 == 0 and rows % 16 == 0; each output is validated as
 *   in fp8_blockwise_quant, and results are bit-identical to two calls of it.
 */
int fp8_blockwise_quant_dual(const void* x, int64_t rows, int64_t cols, int64_t ld_x, int block,
                             void* q, int64_t ld_q, float* recip, int64_t rs_row, int64_t rs_kb,
                             void* qt, int64_t ld_qt, float* recip_t, int64_t rst_row,
                             int64_t rst_kb, int stream_t, void* stream);

/*
 * fp8_tensorwise_quant -- one scale for the whole tensor ([AITER]
 * per_tensor_quant: the scale returned is the dequant multiplier).
 *   x [rows, cols] bf16 (ld_x), q [rows, cols] E4M3 (ld_q), recip: one
 *   device fp32.  ws: device scratch of fp8bw_tensorwise_quant_ws_bytes().
 *   Two launches (partial amax, then quantize); deterministic.
 *   Requires cols % 16 == 0.
 */
size_t fp8bw_tensorwise_quant_ws_bytes(int64_t rows, int64_t cols);
int fp8_tensorwise_quant(const void* x, int64_t rows, int64_t cols, int64_t ld_x, void* q,
                         int64_t ld_q, float* recip, void* ws, size_t ws_bytes, void* stream);

/*
 * fp8_tensorwise_quant_noalloc -- fp8_tensorwise_quant without a workspace
 * argument, for callers that cannot allocate device memory (code under HIP
 * graph capture, tight serving loops, harnesses that forbid allocation).
 * The partial amaxes go to a 4 KiB array the library holds on every GPU it
 * runs on until the process ends (at most 1024 partials, enough for any
 * input, so no size is refused for scratch; FP8BW_ERR_WORKSPACE guards the
 * invariant).  The call allocates nothing; its first call on a device looks
 * up that device's copy of the array (the device current at the call).
 * Results are bit-identical to fp8_tensorwise_quant.  All calls on one GPU
 * share the array: calls that overlap in time on one GPU (different
 * streams) race and give undefined results; calls ordered on one stream are
 * safe.  Arguments, layout and errors otherwise as fp8_tensorwise_quant.
 */
int fp8_tensorwise_quant_noalloc(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                 void* q, int64_t ld_q, float* recip, void* stream);

/*
 * fp8_scaled_gemm_blockwise -- out[M, N] = sum_kb ra[m, kb] * rb[beta(n), kb]
 *                              * sum_{k in block kb} a[m, k] * b[n, k]
 * ([REPRO] What Changed: the blockwise GEMM on the same codes and
 * reciprocal scales as the dequantized matmul; out = A . B^T as F.linear).
 *
 *   a   device E4M3 [M, K], lda; ra: 1x128 scales of A,
 *       ra[m*ra_s_row + kb*ra_s_kb].
 *   b   device E4M3 [N, K], ldb.  b_block selects rb's meaning:
 *         FP8BW_BLOCK_128x128: rb[(n/128)*rb_s_row + kb*rb_s_kb]  (fwd, dgrad)
 *         FP8BW_BLOCK_1x128:   rb[n*rb_s_row + kb*rb_s_kb]        (wgrad)
 *       Scale strides: the column-major layout the quantizers write
 *       (s_row = 1, s_kb >= rows: [INTEG] Summary) is the fast one; any
 *       other non-overlapping nested strides (row-major, transposed or
 *       padded views) are accepted as they are, without a copy.  Strides
 *       that alias (one stride does not span the other dimension's whole
 *       extent) or are negative give FP8BW_ERR_LAYOUT.
 *   out device [M, N] bf16 (RNE from the fp32 accumulator) or fp32, ldo.
 *   K % 128 == 0 (K blocks may number anything, e.g. 1001 or 1002).
 *   Each K block is accumulated in fp32 by the matrix cores and rescaled in
 *   fp32 before it is added to the running sum.
 *   ws: device scratch for split-K partials; size from
 *   fp8bw_gemm_blockwise_ws_bytes(M, N, K) (may be 0 -> ws may be NULL).
 */
size_t fp8bw_gemm_blockwise_ws_bytes(int64_t M, int64_t N, int64_t K);
int fp8_scaled_gemm_blockwise(const void* a, int64_t lda, const float* ra, int64_t ra_s_row,
                              int64_t ra_s_kb, const void* b, int64_t ldb, const float* rb,
                              int64_t rb_s_row, int64_t rb_s_kb, int b_block, int64_t M,
                              int64_t N, int64_t K, void* out, int64_t ldo, int out_dtype,
                              void* ws, size_t ws_bytes, void* stream);

/*
 * fp8_scaled_gemm_blockwise_kn -- the same GEMM with B given in [K, N]
 * layout: out[M, N] = sum_kb ra[m, kb] * rb[beta(n), kb]
 *                     * sum_{k in block kb} a[m, k] * b_kn[k, n].
 * The second operand arrives as the transposed (column-major) view of an
 * [N, K] matrix, the way torch._scaled_mm takes the weight ([AITER] Steps to
 * Reproduce: the weight passed as its .t() view); e.g. dX = dY . W from W's
 * own codes, whose 128x128 blocks and scales serve W^T unchanged (block amax
 * does not depend on orientation), with no transposed copy of the codes.
 *   b_kn device E4M3 [K, N], row stride ldb >= N (N contiguous).
 *   rb   indexed by (output column n, K block) exactly as in
 *        fp8_scaled_gemm_blockwise (for W's scales sw[nb_w][kb_w]: the view
 *        with strides swapped).
 * The kernel reads B's [K block, 256 columns] tiles into LDS row by row and
 * forms the matrix-core operands with transposing LDS reads; outputs are
 * bit-identical to fp8_scaled_gemm_blockwise on b = b_kn^T.
 * Needs M >= 256, N >= 256, N % 16 == 0 (and N % 64 == 0 for 128x128 B
 * scales), 256 * ldb + K < 2^31 and K % 128 == 0; other problems give
 * FP8BW_ERR_UNSUPPORTED (use fp8_scaled_gemm_blockwise on a [N, K] copy).
 * Workspace: fp8bw_gemm_blockwise_ws_bytes(M, N, K).  Other arguments and
 * errors as fp8_scaled_gemm_blockwise.
 */
int fp8_scaled_gemm_blockwise_kn(const void* a, int64_t lda, const float* ra, int64_t ra_s_row,
                                 int64_t ra_s_kb, const void* b_kn, int64_t ldb, const float* rb,
                                 int64_t rb_s_row, int64_t rb_s_kb, int b_block, int64_t M,
                                 int64_t N, int64_t K, void* out, int64_t ldo, int out_dtype,
                                 void* ws, size_t ws_bytes, void* stream);

/*
 * Same as fp8_scaled_gemm_blockwise with an explicit tile configuration
 * (0 .. fp8bw_gemm_num_configs()-1, or -1 for the built-in choice) and
 * split-K count (>= 1, or 0 for the built-in choice).  Every configuration
 * computes the same result up to fp32 rounding order; this entry point
 * lets tests force each one (a kernel variant can be wrong where the
 * others are right: [INDUCT] Describe the bug).  Workspace for an explicit
 * split s is fp8bw_gemm_ws_bytes_for_split(M, N, s).
 */
int fp8bw_gemm_num_configs(void);

/*
 * fp8bw_gemm_blockwise_plan -- how fp8_scaled_gemm_blockwise runs an
 * M x N x K problem with contiguous operands and column-major scales on
 * the current device (host query, launches nothing; for profiling and
 * reporting).  Fills info[6] (caller-owned host array): tile
 * configuration, whole-problem split-K count, split count of the leftover
 * tiles of a partial last round, total tiles, tiles run unsplit, workspace
 * bytes.  Requires 0 < M, N, K and K % 128 == 0.
 */
int fp8bw_gemm_blockwise_plan(int64_t M, int64_t N, int64_t K, int b_block, int64_t* info);
size_t fp8bw_gemm_ws_bytes_for_split(int64_t M, int64_t N, int splits);
int fp8_scaled_gemm_blockwise_cfg(const void* a, int64_t lda, const float* ra, int64_t ra_s_row,
                                  int64_t ra_s_kb, const void* b, int64_t ldb, const float* rb,
                                  int64_t rb_s_row, int64_t rb_s_kb, int b_block, int64_t M,
                                  int64_t N, int64_t K, void* out, int64_t ldo, int out_dtype,
                                  int config, int splits, void* ws, size_t ws_bytes,
                                  void* stream);

/*
 * fp8_scaled_gemm_tensorwise -- out[M, N] = (sum_k a[m, k] * b[n, k]) * ra * rb
 * ([AITER]: per-tensor scales, out = x @ w.T; [INDUCT]: fp32 output).
 *   ra, rb: one device fp32 each (dequant multipliers).
 *   K % 16 == 0 (K need not be a multiple of 128).  No workspace.
 */
int fp8_scaled_gemm_tensorwise(const void* a, int64_t lda, const float* ra, const void* b,
                               int64_t ldb, const float* rb, int64_t M, int64_t N, int64_t K,
                               void* out, int64_t ldo, int out_dtype, void* stream);

/*
 * fp8_scaled_gemm_blockwise_bias / fp8_scaled_gemm_tensorwise_bias -- the
 * same GEMMs with a bias epilogue.  Both GEMM interfaces on the pages take
 * an optional bias (aiter gemm_a8w8 and torch._scaled_mm, [AITER] Steps to
 * Reproduce; the inductor tests parametrize has_bias, [INDUCT] Describe the
 * bug); the pages pass None and do not define its arithmetic.  Here:
 *
 *   out[m, n] = cast(acc[m, n] + bias[n])
 *
 * where acc is the fp32 result the call without bias would cast (after the
 * per-tensor scaling for the tensorwise GEMM), the bias value is widened
 * from bf16 exactly, the add is one fp32 add, and cast is RNE to bf16 or
 * none for fp32 out.  With split-K the add happens once, in the reduce.
 *
 *   bias   device bf16 [N], contiguous, 2-byte aligned; NULL = no bias
 *          (then identical to the call without _bias).
 *   Every other argument, status and workspace rule is that of the call
 *   without _bias.
 */
int fp8_scaled_gemm_blockwise_bias(const void* a, int64_t lda, const float* ra, int64_t ra_s_row,
                                   int64_t ra_s_kb, const void* b, int64_t ldb, const float* rb,
                                   int64_t rb_s_row, int64_t rb_s_kb, int b_block, int64_t M,
                                   int64_t N, int64_t K, const void* bias, void* out, int64_t ldo,
                                   int out_dtype, void* ws, size_t ws_bytes, void* stream);
int fp8_scaled_gemm_tensorwise_bias(const void* a, int64_t lda, const float* ra, const void* b,
                                    int64_t ldb, const float* rb, int64_t M, int64_t N, int64_t K,
                                    const void* bias, void* out, int64_t ldo, int out_dtype,
                                    void* stream);

/*
 * fp8_scaled_grouped_gemm_blockwise -- one call for G GEMMs that share N
 * and K and split the rows of A and out into consecutive groups, each with
 * its own B (the mixture-of-experts layout: tokens sorted by expert, one
 * weight per expert; the pages mention the grouped scaled matmul of MoE
 * training in [INTEG]'s review discussion).  For every group g and row m of
 * it, out[m, :] is what fp8_scaled_gemm_blockwise gives for that row with B_g
 * (1x128 A scales, 128x128 B scales):
 *
 *   rows of group g: [group_end[g-1], group_end[g])   (group_end[-1] = 0)
 *   B_g  = b  + g * b_s_group   [N, K] codes, leading dim ldb
 *   rb_g = rb + g * rb_s_group  scales of B_g, rb_g[(n/128)*rb_s_row + kb*rb_s_kb]
 *
 *   a, ra       device [M, K] codes and their column-major 1x128 scales
 *               ra[m + kb*ra_s_kb] (ra_s_kb >= M) for all groups' rows.
 *   group_end   DEVICE int32 [groups], cumulative row ends, read by the
 *               kernel (no host synchronization).  Values are clamped to
 *               [previous end, M]: a malformed table cannot make the kernel
 *               read or write outside A, ra and out.  Rows past the last end
 *               are not written.
 *   b_s_group   >= (N-1)*ldb + K, a multiple of 16 (distinct weights).
 *   rb_s_group  large enough that groups' scale grids do not overlap.
 *   Requires K % 128 == 0; no split-K, no workspace.  Problems with
 *   M >= 256 and N >= 128 (and 256*lda + K, 256*ldb + K < 2^31) run on the
 *   large-tile kernels, others on the small-tile kernel.  With up to 64
 *   groups on the large tiles the call enqueues two launches: the second
 *   takes the groups' last partial row tiles of at most 128 rows as 64-row
 *   tiles when the table (read on the device) shows that this saves a round
 *   of the GPU's compute units; otherwise it returns at once.  Every row is
 *   written by exactly one launch.  The grids must fit in 2^31 - 1
 *   workgroups (else FP8BW_ERR_UNSUPPORTED).
 */
int fp8_scaled_grouped_gemm_blockwise(const void* a, int64_t lda, const float* ra,
                                      int64_t ra_s_kb, const void* b, int64_t ldb,
                                      int64_t b_s_group, const float* rb, int64_t rb_s_row,
                                      int64_t rb_s_kb, int64_t rb_s_group, int groups,
                                      const int* group_end, int64_t M, int64_t N, int64_t K,
                                      void* out, int64_t ldo, int out_dtype, void* stream);

/*
 * FP8 blockwise linear layer, fwd / dgrad / wgrad ([INTEG] Summary:
 * Float8BlockwiseLinear; [REPRO] review comments: 1x128 x 128x128 on the
 * grad path, 1x128 x 1x128 for the weight gradient).  All tensors are
 * contiguous row-major bf16: X[M, K], W[N, K], dY[M, N].
 *   fwd:   Y[M, N]  = X . W^T   (X 1x128, W 128x128)        K % 128 == 0
 *   dgrad: dX[M, K] = dY . W    (dY 1x128, W^T 128x128)     N % 128 == 0
 *   wgrad: dW[N, K] = dY^T . X  (dY^T, X^T 1x128 along M)   M % 128 == 0
 * Each quantizes its inputs into the caller's workspace (codes and
 * reciprocal scales) and runs the blockwise GEMM; bf16 output.
 * which = 0 fwd, 1 dgrad, 2 wgrad for the workspace query (3 and 4: the
 * fused entry points below).  All dims must also be multiples of 16.
 */
size_t fp8bw_linear_ws_bytes(int64_t M, int64_t N, int64_t K, int which);
int fp8_linear_fwd(const void* x, const void* w, void* y, int64_t M, int64_t N, int64_t K,
                   void* ws, size_t ws_bytes, void* stream);
int fp8_linear_dgrad(const void* dy, const void* w, void* dx, int64_t M, int64_t N, int64_t K,
                     void* ws, size_t ws_bytes, void* stream);
int fp8_linear_wgrad(const void* dy, const void* x, void* dw, int64_t M, int64_t N, int64_t K,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * FP8 blockwise linear with each large bf16 tensor read once per step: the
 * same three GEMMs and the same codes and scales as fp8_linear_fwd / _dgrad
 * / _wgrad (bit-identical outputs), with fused quantization
 * (fp8_blockwise_quant_dual): the forward quantizes X once into X (1x128
 * along K) and X^T (1x128 along M), keeping X^T's codes and scales for the
 * backward (written with nontemporal stores, so that X's codes stay cached
 * for the forward GEMM), and W into W (128x128); the backward quantizes dY
 * once into dY
 * and dY^T, and W into W^T right before the dgrad GEMM.  The quantizers are
 * the part of the fp8 linear step the pages single out as slow ([INTEG]
 * Benchmarks); fp8 X^T codes are also half the size of the bf16 X a
 * backward would otherwise keep.  W^T is written by the backward rather
 * than kept from the forward because the dgrad GEMM then reads it from the
 * memory-side cache it was just written to (one more read of W, 2 bytes per
 * weight, against a faster dgrad GEMM).
 *
 *   fp8_linear_fwd_save: Y[M, N] = X . W^T; writes `saved`.
 *     Requires K % 128 == 0 (and M, N, K multiples of 16).
 *   fp8_linear_bwd: dX[M, K] = dY . W and dW[N, K] = dY^T . X from dY, the
 *     same bf16 W [N, K] and the `saved` of the forward with the same X, W,
 *     M, N, K.  dx or dw may be null to skip that gradient.  Requires
 *     M % 128 == 0 and N % 128 == 0.
 *   saved   caller device memory of fp8bw_linear_saved_bytes(M, N, K)
 *           bytes, 256-byte aligned, owned by the caller between the two
 *           calls; its layout is internal to the library.
 *   ws      workspace of fp8bw_linear_ws_bytes(M, N, K, which) bytes with
 *           which = 3 (fwd_save) or 4 (bwd), 256-byte aligned.
 * Errors as for fp8_linear_fwd; nothing is launched on an error.
 */
size_t fp8bw_linear_saved_bytes(int64_t M, int64_t N, int64_t K);
int fp8_linear_fwd_save(const void* x, const void* w, void* y, int64_t M, int64_t N, int64_t K,
                        void* saved, size_t saved_bytes, void* ws, size_t ws_bytes, void* stream);
int fp8_linear_bwd(const void* dy, const void* w, const void* saved, size_t saved_bytes, void* dx,
                   void* dw, int64_t M, int64_t N, int64_t K, void* ws, size_t ws_bytes,
                   void* stream);

/*
 * fp8bw_rms_norm_fwd -- root-mean-square norm in front of an FP8 linear, with
 * the residual's addition and the linear's operand codes from the same pass:
 *
 *   s[r, c]  = bf16(x[r, c] + residual[r, c])     (s = x without a residual)
 *   rstd[r]  = 1 / sqrt(mean_c s[r, c]^2 + eps)
 *   v[r, c]  = s[r, c] * rstd[r] * weight[c]      (fp32)
 *   y = bf16(v); (q, recip) = codes of v in 1x128 blocks along the columns;
 *   (qt, recip_t) = codes of v^T in 1x128 blocks along the rows
 *
 *   x, residual  device bf16 [rows, cols] (ld_x, ld_res); residual may be NULL.
 *   sum          device bf16 [rows, cols] (ld_sum): s.  Required with a
 *                residual, not used without; it may be x or residual itself
 *                (same pointer and leading dimension), no other overlap.
 *   weight       device [cols], bf16 (weight_dtype FP8BW_OUT_BF16) or fp32
 *                (FP8BW_OUT_F32), 16-byte aligned.
 *   rstd         device fp32 [rows], for the backward.
 *   y, q, qt     outputs, each may be NULL: y bf16 (ld_y); q E4M3 [rows, cols]
 *                (ld_q) with recip[r*rs_row + kb*rs_kb]; qt E4M3 [cols, rows]
 *                (ld_qt) with recip_t[c*rst_row + mb*rst_kb].  The codes
 *                follow the quantizers' recipe on the fp32 v (not on y).
 *   Requires cols % 16 == 0, cols <= 16384, rows < 2^22, and rows % 16 == 0
 *   with qt (one more launch, which reads s again).  eps >= 0.
 */
int fp8bw_rms_norm_fwd(const void* x, int64_t ld_x, const void* residual, int64_t ld_res,
                       const void* weight, int weight_dtype, float eps, int64_t rows, int64_t cols,
                       void* sum, int64_t ld_sum, float* rstd, void* y, int64_t ld_y, void* q,
                       int64_t ld_q, float* recip, int64_t rs_row, int64_t rs_kb, void* qt,
                       int64_t ld_qt, float* recip_t, int64_t rst_row, int64_t rst_kb,
                       void* stream);

/*
 * fp8bw_rms_norm_bwd -- its gradients (codes pass gradients straight through):
 *   h = s * rstd, d = dy * weight
 *   dx[r, c]   = bf16(rstd * (d - h * mean_c(d * h)) + dres)
 *   dweight[c] = sum_r dy * h                (in the weight's type)
 * dx is the gradient of x and of the residual alike.
 *
 *   dy, s, dres  device bf16 [rows, cols]; dres, the gradient that reaches s
 *                past the norm, may be NULL.  rstd as the forward wrote it.
 *   dx           device bf16 [rows, cols]; dweight device [cols].
 *   ws           fp8bw_rms_norm_bwd_ws_bytes(rows, cols) bytes, 16-byte
 *                aligned (fp32 partial sums of dweight, joined in a fixed
 *                order: results repeat bit for bit).
 * With rows == 0 dweight is not written.
 */
size_t fp8bw_rms_norm_bwd_ws_bytes(int64_t rows, int64_t cols);
int fp8bw_rms_norm_bwd(const void* dy, int64_t ld_dy, const void* s, int64_t ld_s,
                       const float* rstd, const void* weight, int weight_dtype, const void* dres,
                       int64_t ld_dres, int64_t rows, int64_t cols, void* dx, int64_t ld_dx,
                       void* dweight, void* ws, size_t ws_bytes, void* stream);

/*
 * fp8bw_linear_xent_fwd / _bwd / _bwd_loss -- softmax cross entropy of a linear head over
 * a large vocabulary, logits z = h . w^T, without keeping the logits:
 *
 *   lse[t]  = log sum_v exp(z[t, v]);  loss[t] = lse[t] - z[t, target[t]]
 *   G[t, v] = (exp(z[t, v] - lse[t]) - [v == target[t]]) * dloss[t]
 *   dh = G . w,  dw = G^T . h
 *
 *   h, w     device bf16 [T, K] (ld_h) and [V, K] (ld_w).
 *   target   device int64 [T].  A target equal to ignore_index gives loss 0
 *            and no gradient.  Any other target outside [0, V) gives a NaN
 *            loss and no gradient.  What the rows of h of tokens without a
 *            gradient (those, and dloss 0) hold reaches neither dh nor dw.
 *   loss, lse, dloss  device fp32 [T]; one loss per token, so that a caller's
 *            mean, sum or weights are dloss.  The loss is formed as log(1 + sum_{v !=
 *            target} exp(z[t, v] - z[t, target])): its relative error is a few units
 *            of fp32 beside the logits', also where it is far below a rounding of lse.
 *            fp8bw_linear_xent_bwd_loss takes the forward's losses (or NULL) and forms
 *            the target's entry of G, p - 1, as expm1(-loss).  From lse alone
 *            (fp8bw_linear_xent_bwd, or loss NULL) that entry is off by lse's rounding,
 *            about 2^-24 |lse|, which is all of it for a token that confident.
 *   dh, dw   device bf16 [T, K] (ld_dh) and [V, K] (ld_dw); either may be NULL.
 *   The backward takes the vocabulary in pieces: each piece's logits are made
 *   again and become its part of G (bf16) in the workspace, whose size does
 *   not grow with V beyond one piece.  G's rows are rounded to bf16 and their
 *   sums, which are zero in exact numbers, taken out of dh with the target's
 *   row of w: dh[t] = sum_v G[t, v] (w[v] - w[target[t]]), so that what the
 *   rows of w share does not carry G's rounding into dh.
 *   ws       fp8bw_linear_xent_ws_bytes(T, V, K, backward) bytes, 256-byte
 *            aligned (backward: 0 or 1).
 *   Requires K % 64 == 0, 64 <= K <= 2^20, V <= 2^28, T <= 2^24, leading
 *   dimensions a multiple of 8 and at most 2^22 - K / 128, and
 *   ceil(a / 256) * ceil(b / 256) < 2^23 for any two of T, V, K.  With V == 0 every
 *   call with T > 0 is rejected (an empty sum has no logarithm); with T == 0 dw is set
 *   to zero.
 */
size_t fp8bw_linear_xent_ws_bytes(int64_t T, int64_t V, int64_t K, int backward);
int fp8bw_linear_xent_fwd(const void* h, int64_t ld_h, const void* w, int64_t ld_w,
                          const int64_t* target, int64_t ignore_index, int64_t T, int64_t V,
                          int64_t K, float* loss, float* lse, void* ws, size_t ws_bytes,
                          void* stream);
int fp8bw_linear_xent_bwd(const float* dloss, const void* h, int64_t ld_h, const void* w,
                          int64_t ld_w, const int64_t* target, int64_t ignore_index,
                          const float* lse, int64_t T, int64_t V, int64_t K, void* dh,
                          int64_t ld_dh, void* dw, int64_t ld_dw, void* ws, size_t ws_bytes,
                          void* stream);
int fp8bw_linear_xent_bwd_loss(const float* dloss, const void* h, int64_t ld_h, const void* w,
                               int64_t ld_w, const int64_t* target, int64_t ignore_index,
                               const float* lse, const float* loss, int64_t T, int64_t V, int64_t K,
                               void* dh, int64_t ld_dh, void* dw, int64_t ld_dw, void* ws,
                               size_t ws_bytes, void* stream);

/*
 * fp8bw_adamw_step -- one AdamW step over many tensors, in place:
 *
 *   g = grad * grad_scale[0]                       (1 if grad_scale is NULL)
 *   m = beta1 m + (1 - beta1) g;  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay)
 *       - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 *   tensors  host array of `count`; each is contiguous, at the alignment of
 *            its elements.  p is the fp32 master where there is one (param,
 *            bf16, then receives its rounding), else param.
 *   state    FP8BW_STATE_F32: exp_avg and exp_avg_sq are fp32 [numel].
 *            FP8BW_STATE_E4M3: they hold E4M3 codes [numel] of m and of
 *            sqrt(v), with fp32 scales [ceil(numel / 128)] per 128 elements,
 *            m = code * exp_avg_scale, sqrt(v) = code * root_scale; the step
 *            writes power-of-two scales, the least that hold the block's
 *            largest value within 448 (1 for a block of zeros).  A positive
 *            sqrt(v) is never rounded to code 0.  A moment that is infinite or
 *            NaN becomes the NaN code and has no part in its block's scale.
 *            Codes 0 with any finite scale are the start.
 *   stochastic  nonzero: codes, and bf16 parameters without a master, are
 *            rounded up or down at random, in proportion to the remainder, by
 *            16 bits per value of a hash of (seed, index of the tensor in
 *            `tensors`, element).  Equal arguments give equal results; use
 *            another seed each step, and in calls that share a seed another
 *            index for every tensor (an entry of numel 0 takes up an index and
 *            may be all zeros).  The hash is of 32 bits, the tensor's key added
 *            to the element: of 2^32 elements and more some share their numbers.
 *            Zero: to nearest.
 *   step     counts from 1.  lr, weight_decay and eps >= 0; 0 <= beta1, beta2 < 1.
 * One launch per 40 tensors.  numel < 2^35.
 */
typedef enum { FP8BW_STATE_F32 = 0, FP8BW_STATE_E4M3 = 1 } fp8bw_state;
typedef struct {
  void* param;
  const void* grad;
  void* exp_avg;
  void* exp_avg_sq;
  float* exp_avg_scale; /* NULL with fp32 states */
  float* root_scale;    /* NULL with fp32 states */
  float* master;        /* NULL: none */
  int64_t numel;
  int param_dtype;      /* fp8bw_out */
  int grad_dtype;       /* fp8bw_out */
} fp8bw_adamw_tensor;
int fp8bw_adamw_step(const fp8bw_adamw_tensor* tensors, int count, int state, int64_t step,
                     double lr, double beta1, double beta2, double eps, double weight_decay,
                     const float* grad_scale, int stochastic, uint64_t seed, void* stream);

/*
 * Experts: the operators around the grouped GEMM in a mixture-of-experts layer.
 *
 * A slot i = t * topk + j is token t's j-th choice of an expert.  fp8bw_moe_sort
 * gives every slot a row, in the order of its expert and then of the slots, each
 * expert's rows padded to a multiple of `align` (1, or 128 for the grouped weight
 * gradient):
 *
 *   group_end[e] = sum_{f <= e} ceil(n_f / align) * align,  n_f slots of expert f
 *   row[i]       = (group_end[e] - padded n_e) + number of slots i' < i of expert e
 *   source[r]    = the slot with row r; -1 for padding and behind the last end
 *
 *   expert     device [tokens, topk], int32 (index_bits 32) or int64 (64).  A slot
 *              whose number is outside [0, experts) has no expert: row -1.
 *   rows       at least fp8bw_moe_rows(tokens, topk, experts, align), which holds
 *              the slots however they fall; known without reading the device.
 *   row, source, group_end   device int32 [tokens, topk], [rows], [experts].
 *              group_end is the table that the grouped GEMM takes.
 *   ws         fp8bw_moe_sort_ws_bytes(tokens, topk, experts) bytes, 256-byte aligned
 *              (0 for few slots: ws may be NULL).
 *   Requires 1 <= topk <= 64, 1 <= experts <= 1024, 1 <= align <= 65536,
 *   tokens < 2^24, rows < 2^27 (fp8bw_moe_rows is 0 for larger ones).
 */
int64_t fp8bw_moe_rows(int64_t tokens, int64_t topk, int64_t experts, int64_t align);
size_t fp8bw_moe_sort_ws_bytes(int64_t tokens, int64_t topk, int64_t experts);
int fp8bw_moe_sort(const void* expert, int index_bits, int64_t tokens, int64_t topk, int64_t experts,
                   int64_t align, int64_t rows, int32_t* row, int32_t* source, int32_t* group_end,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * The outputs of a [rows, cols] result v (fp32); each pointer may be NULL.  A host struct.
 *   y   device bf16 [rows, cols]
 *   q   device E4M3 [rows, cols] in 1x128 blocks along the columns, with
 *       recip[r*rs_row + kb*rs_kb]
 *   qt  device E4M3 [cols, rows]: codes of v^T in 1x128 blocks along the rows, with
 *       recip_t[c*rst_row + mb*rst_kb]; needs rows % 16 == 0
 * The codes follow the quantizers' recipe on v (not on y), which is one of finite values.
 * Here a NaN becomes the NaN code and has no part in its block's scale; an infinity makes
 * its block's reciprocal scale infinite, its own code NaN and the block's finite codes 0.
 */
typedef struct {
  void* y;
  int64_t ld_y;
  void* q;
  int64_t ld_q;
  float* recip;
  int64_t rs_row, rs_kb;
  void* qt;
  int64_t ld_qt;
  float* recip_t;
  int64_t rst_row, rst_kb;
} fp8bw_layouts;

/*
 * fp8bw_moe_gather -- token rows in the sorted order: v[r] = x[source[r] / topk],
 * zeros (code 0) where a row has no slot.  Its gradient is fp8bw_moe_combine without
 * weights.
 *   x   device bf16 [tokens, cols].  row and source: as fp8bw_moe_sort wrote them (a
 *       row outside [0, rows) and a source outside [0, tokens * topk) count as -1; a
 *       table whose row and source are not each other's inverse gives unspecified
 *       values).
 *
 * fp8bw_moe_combine -- the experts' rows joined: out[t] = sum_j weight[t, j] *
 * y[row[t, j]] over the slots that have a row, in fp32 in the slots' order; zeros for
 * a token without any.  What y holds in other rows is not read.
 *   y   device bf16 [rows, cols]; weight device [tokens, topk], fp32 or bf16
 *       (weight_dtype), NULL: ones; out device bf16 [tokens, cols].
 *
 * fp8bw_moe_combine_bwd -- its gradients: v[r] = weight[source[r]] * dout[source[r] /
 * topk] (zeros without a slot) in dy's layouts, and dweight[t, j] = sum_c dout[t, c] *
 * y[row[t, j], c] (0 without a row) in the weight's type, or NULL.  y is read only for
 * dweight.  With qt asked for and dweight, two launches.
 *
 * All three: cols % 16 == 0, cols <= 65536, tokens < 2^24, rows < 2^27, and fewer than
 * 2^26 pieces of 512 columns of tokens and 2^23 tiles of 128 rows x 128 columns.
 * rows >= 1 if tokens >= 1, and no rows without tokens.  Transposed codes need rows
 * % 16 == 0, y's leading dimension below 2^22 and those of codes below 2^24.
 */
int fp8bw_moe_gather(const void* x, int64_t ld_x, int64_t tokens, int64_t topk, const int32_t* row,
                     const int32_t* source, int64_t rows, int64_t cols, const fp8bw_layouts* out,
                     void* stream);
int fp8bw_moe_combine(const void* y, int64_t ld_y, const void* weight, int weight_dtype, int64_t tokens,
                      int64_t topk, const int32_t* row, int64_t rows, int64_t cols, void* out,
                      int64_t ld_out, void* stream);
int fp8bw_moe_combine_bwd(const void* dout, int64_t ld_dout, const void* y, int64_t ld_y,
                          const void* weight, int weight_dtype, int64_t tokens, int64_t topk,
                          const int32_t* row, const int32_t* source, int64_t rows, int64_t cols,
                          const fp8bw_layouts* dy, void* dweight, void* stream);

/*
 * fp8bw_swiglu_fwd -- the gated activation between an MLP's two products:
 *
 *   h = [g | u],  v = g * sigmoid(g) * u
 *
 *   h    device bf16 [rows, 2 ffn]; out: the layouts of v [rows, ffn].
 *   hq   device E4M3 [rows, 2 ffn], a checkpoint of h for the backward in half its
 *        bytes, in 1x128 blocks of each half: h_recip[r*hr_row + kb*hr_kb], kb in
 *        [0, 2 ceil(ffn / 128)), the gate's blocks first.  NULL: not written.
 *
 * fp8bw_swiglu_bwd -- its gradient, with s = sigmoid(g):
 *   dg = dy * u * s * (1 + g * (1 - s)),  du = dy * g * s
 *
 *   dy   device bf16 [rows, ffn]; not read, and may be NULL, if dh asks for nothing.
 *   h    bf16 with h_recip NULL, else a checkpoint's codes and its scales; g and u are
 *        then the values that the codes stand for.
 *   dh   the layouts of [dg | du] [rows, 2 ffn]; q in 1x128 blocks of each half.
 *   act_qt   device E4M3 [ffn, rows] or NULL: codes of v^T, made again, in 1x128 blocks
 *        along the rows, act_recip_t[c*art_row + mb*art_kb]: the second product's
 *        operand of its weight gradient.
 *
 * Both: ffn % 16 == 0, ffn <= 2^20, rows < 2^27, fewer than 2^26 pieces of 512 columns
 * and 2^23 tiles of 128 x 128 of v.  Transposed codes need rows % 16 == 0, leading
 * dimensions of bf16 and row strides of h_recip below 2^22, and of codes below 2^24.
 */
int fp8bw_swiglu_fwd(const void* h, int64_t ld_h, int64_t rows, int64_t ffn, const fp8bw_layouts* out,
                     void* hq, int64_t ld_hq, float* h_recip, int64_t hr_row, int64_t hr_kb,
                     void* stream);
int fp8bw_swiglu_bwd(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, const float* h_recip,
                     int64_t hr_row, int64_t hr_kb, int64_t rows, int64_t ffn, const fp8bw_layouts* dh,
                     void* act_qt, int64_t ld_act_qt, float* act_recip_t, int64_t art_row,
                     int64_t art_kb, void* stream);

/*
 * fp8_scaled_grouped_gemm_blockwise_wgrad -- the weight gradients of a grouped GEMM,
 * one [M, N] product per group over that group's rows, which are the contraction:
 *
 *   out_g[m, n] = sum_{kb in group g} ra[m, kb] * rb[n, kb] * sum_{k in kb} a[m, k] * b[n, k]
 *
 *   a, b       device E4M3 [M, K] and [N, K]: the transposed codes of the two [K, ..]
 *              matrices (dY^T and X^T), in 1x128 blocks along K with scales
 *              ra[m*ra_s_row + kb*ra_s_kb], rb[n*rb_s_row + kb*rb_s_kb] (strides as in
 *              fp8_scaled_gemm_blockwise).
 *   group_end  DEVICE int32 [groups], cumulative ends along K, multiples of 128 (a sort
 *              with align 128): group g contracts the blocks [group_end[g-1] / 128,
 *              group_end[g] / 128), clamped to K.  Codes outside are not used.  A group
 *              without blocks gives zeros.
 *   out        device [M, N] per group, bf16 or fp32, ldo, out_s_group elements apart
 *              (>= (M - 1) * ldo + N).
 *   ws         fp8bw_grouped_wgrad_ws_bytes(M, N, K, groups) bytes, 256-byte aligned:
 *              fp32 partials of few tiles over long contractions, joined in a fixed
 *              order (0 where there are none: ws may be NULL).
 *   Requires K % 128 == 0, 1 <= groups <= 2^20 and fewer than 2^23 output tiles (times the
 *   pieces of their contractions); errors as fp8_scaled_gemm_blockwise.
 *
 * fp8bw_grouped_wgrad_plan -- how such a call runs with contiguous operands and outputs and
 * column-major scales on the current device (host query, launches nothing; for profiling and
 * tests).  Fills info[4] (caller-owned host array): tile configuration (0: 128x128, 1: 64x64,
 * 3: 256x256), pieces of every group's contraction, output tiles of all groups, and 1 where
 * one workgroup per compute unit runs the tiles as one stream, else 0.  Requires 0 < M, N, K
 * and K % 128 == 0.
 */
size_t fp8bw_grouped_wgrad_ws_bytes(int64_t M, int64_t N, int64_t K, int groups);
int fp8bw_grouped_wgrad_plan(int64_t M, int64_t N, int64_t K, int groups, int out_dtype, int64_t* info);
int fp8_scaled_grouped_gemm_blockwise_wgrad(const void* a, int64_t lda, const float* ra,
                                            int64_t ra_s_row, int64_t ra_s_kb, const void* b,
                                            int64_t ldb, const float* rb, int64_t rb_s_row,
                                            int64_t rb_s_kb, int groups, const int* group_end,
                                            int64_t M, int64_t N, int64_t K, void* out, int64_t ldo,
                                            int64_t out_s_group, int out_dtype, void* ws,
                                            size_t ws_bytes, void* stream);

/*
 * fp8_blockwise_quant_grouped -- fp8_blockwise_quant with 128x128 blocks of `groups`
 * matrices of one shape in one launch (the experts' weights, as they are or transposed):
 * group g is x + g*x_s_group, with codes at q + g*q_s_group and scales at recip +
 * g*recip_s_group.  Strides between groups must keep the outputs apart (x's may be any
 * multiple of 8).  Arguments and errors otherwise as fp8_blockwise_quant; 1 <= groups
 * <= 65535 and fewer than 2^24 blocks.
 */
int fp8_blockwise_quant_grouped(const void* x, int64_t rows, int64_t cols, int64_t ld_x,
                                int64_t x_s_group, int groups, int transpose, void* q, int64_t ld_q,
                                int64_t q_s_group, float* recip, int64_t rs_row, int64_t rs_kb,
                                int64_t recip_s_group, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8BW_H */
