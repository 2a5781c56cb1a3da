// Root-mean-square norm of a residual stream for gfx950, forward (bf16 and
// blockwise E4M3 outputs) and backward.
//
//   s    = bf16(x + residual)                 (s = x without a residual)
//   rstd = 1 / sqrt(mean_c s[r, c]^2 + eps)
//   v    = s * rstd * weight                   (fp32)
//   y    = bf16(v);  q = E4M3 codes of v in 1x128 blocks along the columns;
//   qt   = E4M3 codes of v^T in 1x128 blocks along the rows (the operand a
//          linear's weight gradient contracts over its tokens)
//
// The codes are made from v itself, not from its bf16 rounding, with the
// quantizers' recipe (s_blk = 448 / max(amax, 1e-12), recip = 1 / s_blk).
//
// Backward, with h = s * rstd and d = dy * weight:
//   dx = rstd * (d - h * mean_c(d * h)) + dres,   dweight = sum_r dy * h
//
// Every kernel streams: rows are read once into registers with 16-byte
// loads, sums are fp32 in a fixed order (DPP within a wave, then LDS, no
// atomics), so results repeat bit for bit.

#include "launch.h"
#include "vec8.h"

namespace fp8bw {

// Sum over the TPR threads of a row; `red` holds one float per wave and is
// not written again before the caller's next barrier or its other half.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < TPR / 64; ++w) v += red[w];
  }
  return v;
}

__device__ __forceinline__ void load_weight8(const NormWeight& w, int col, float (&f)[8]) {
  if (w.f32) {
    const float4 a = *(const float4*)((const float*)w.p + col);
    const float4 b = *(const float4*)((const float*)w.p + col + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
    unpack8(*(const uint4*)((const uint16_t*)w.p + col), f);
  }
}

// 8 weights as they are stored, kept packed between uses.
template <bool F32>
struct Weight8 {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int col) {
    if constexpr (F32) {
      a = *(const uint4*)((const float*)p + col);
      b = *(const uint4*)((const float*)p + col + 4);
    } else {
      a = *(const uint4*)((const uint16_t*)p + col);
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    if constexpr (F32) {
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
      f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
      f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
      unpack8(a, f);
    }
  }
};

// The compiler may not look through this: without it, it keeps a packed value's
// 8 floats instead of its 4 registers across a reduction or a loop.
__device__ __forceinline__ void keep_packed(uint4& u) {
  asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
}

// v of 8 columns: the product order (s * rstd) * weight is the same in the
// row kernel and the transposing kernel, so both quantize the same values.
__device__ __forceinline__ void normed8(const uint4& s, float rstd, const float (&w)[8], float (&v)[8]) {
  unpack8(s, v);
#pragma unroll
  for (int c = 0; c < 8; ++c) v[c] = v[c] * rstd * w[c];
}

// ---------------------------------------------------------------------------
// Which of a workgroup's rows this wave works on, known to be the same for all
// its lanes: row addresses then stay in scalar registers.
template <int TPR>
__device__ __forceinline__ int row_slot() {
  return TPR == 64 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
}

// Forward, one row per TPR threads: thread t holds chunks t, t + TPR, .. of 8
// columns, so a 16-lane DPP row holds one 1x128 block.  The row stays in
// registers between the sum of squares and the outputs.  Bound by HBM: 16640 x
// 8192 with residual and codes 151 to 155 us (6.2 TB/s); one row of 8192 3 us.
template <int TPR, int CH>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_fwd_kernel(const NormFwdArgs p) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  __shared__ float red[BLOCK / 64];
  const int64_t r = (int64_t)blockIdx.x * (BLOCK / TPR) + row_slot<TPR>();
  const int t = threadIdx.x % TPR;
  if (r >= p.rows) return;   // whole waves (TPR 64: no barrier; else one row a workgroup)
  const uint16_t* const x = p.x + r * p.ld_x;
  uint4 s[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int col = (k * TPR + t) * 8;
    s[k] = make_uint4(0, 0, 0, 0);
    if (col < p.cols) s[k] = load_stream(x + col);
  }
  if (p.residual) {
    const uint16_t* const res = p.residual + r * p.ld_res;
    uint4 u[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      u[k] = make_uint4(0, 0, 0, 0);
      if (col < p.cols) u[k] = load_stream(res + col);
    }
    uint16_t* const sum = p.sum + r * p.ld_sum;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      float a[8], b[8];
      unpack8(s[k], a);
      unpack8(u[k], b);
#pragma unroll
      for (int c = 0; c < 8; ++c) a[c] += b[c];
      s[k] = pack8(a);
      if (col < p.cols) *(uint4*)(sum + col) = s[k];
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float a[8];
    unpack8(s[k], a);
#pragma unroll
    for (int c = 0; c < 8; ++c) ss = __builtin_fmaf(a[c], a[c], ss);
  }
  ss = row_sum<TPR>(ss, red);
  const float rstd = 1.0f / __builtin_sqrtf(ss / (float)p.cols + p.eps);
  if (t == 0) p.rstd[r] = rstd;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int col = (k * TPR + t) * 8;
    const bool in = col < p.cols;
    float w[8], v[8];
    load_weight8(p.weight, in ? col : 0, w);
    normed8(s[k], rstd, w, v);
    if (p.y && in) *(uint4*)(p.y + r * p.ld_y + col) = pack8(v);
    if (p.q) {
      float m = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(v[c]));   // 0 past the last column
      const float sc = scale_from_amax(row16_max(m));
      uint2 code;
      code.x = cvt4_e4m3(v[0] * sc, v[1] * sc, v[2] * sc, v[3] * sc);
      code.y = cvt4_e4m3(v[4] * sc, v[5] * sc, v[6] * sc, v[7] * sc);
      if (in) {
        *(uint2*)(p.q + r * p.ld_q + col) = code;
        if ((t & 15) == 0) p.recip[r * p.rs_row + (col >> 7) * p.rs_kb] = recip_of_scale(sc);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Transposed codes qt from s and rstd: one workgroup per 128 x 128 tile of v,
// one scale per column of the tile.  Thread t owns columns 8 (t % 16) .. + 7
// of rows 4 j .. 4 j + 3 and 64 + 4 j .. (j = t / 16); codes go through an LDS
// tile stored [column][row] whose dword d of column c sits at
// d ^ 4 ((c / 8) % 8), and out as 16-byte pieces of output rows.  s passes the
// caches by, and so does qt, which nobody reads before the backward (both
// kernels at 16640 x 8192: 237 us; with ordinary loads and stores 256 us).
__global__ __launch_bounds__(256) void rms_norm_quant_t_kernel(const NormFwdArgs p) {
  __shared__ float red[4][128];
  __shared__ float ssc[128];
  __shared__ __attribute__((aligned(16))) uint32_t tile[128 * 32];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int g = tid & 15, j = tid >> 4;
  const int64_t cb = blockIdx.x, rb = blockIdx.y;
  const int64_t col = cb * 128 + g * 8;
  const bool col_in = col < p.cols;
  const uint16_t* const s = p.residual ? p.sum : p.x;
  const int64_t ld = p.residual ? p.ld_sum : p.ld_x;
  uint4 u[8];
  float rs[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int64_t r = rb * 128 + 64 * (k >> 2) + 4 * j + (k & 3);
    const bool in = col_in && r < p.rows;
    u[k] = load_stream(s + (in ? r * ld + col : 0));
    rs[k] = in ? p.rstd[r] : 0.f;
    if (!in) u[k] = make_uint4(0, 0, 0, 0);
  }
  float w[8];
  load_weight8(p.weight, col_in ? (int)col : 0, w);
  float v[8][8];
  float m[8] = {};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    normed8(u[k], rs[k], w, v[k]);
#pragma unroll
    for (int c = 0; c < 8; ++c) m[c] = fmaxf(m[c], fabsf(v[k][c]));
  }
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    m[c] = fmaxf(m[c], __shfl_xor(m[c], 16));
    m[c] = fmaxf(m[c], __shfl_xor(m[c], 32));
    if (lane < 16) red[wave][8 * g + c] = m[c];
  }
  __syncthreads();
  if (tid < 128) {
    const float a = fmaxf(fmaxf(red[0][tid], red[1][tid]), fmaxf(red[2][tid], red[3][tid]));
    const float sc = scale_from_amax(a);
    ssc[tid] = sc;
    if (cb * 128 + tid < p.cols)
      p.recip_t[(cb * 128 + tid) * p.rst_row + rb * p.rst_kb] = recip_of_scale(sc);
  }
  __syncthreads();
  const int sw = 4 * (g & 7);
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float sc = ssc[8 * g + c];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      tile[(8 * g + c) * 32 + ((16 * h + j) ^ sw)] =
          cvt4_e4m3(v[4 * h][c] * sc, v[4 * h + 1][c] * sc, v[4 * h + 2][c] * sc, v[4 * h + 3][c] * sc);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int id = tid + 256 * i;
    const int oc = id >> 3, seg = id & 7;
    const uint4 val = *(const uint4*)&tile[oc * 32 + ((4 * seg) ^ (4 * ((oc >> 3) & 7)))];
    const int64_t orow = cb * 128 + oc, ocol = rb * 128 + 16 * seg;
    if (orow < p.cols && ocol < p.rows) {
      const u32x4 t = {val.x, val.y, val.z, val.w};
      __builtin_nontemporal_store(t, (u32x4*)(p.qt + orow * p.ld_qt + ocol));
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: workgroup b takes rows b RPW + sub, + gridDim.x RPW, ..; a thread
// keeps the weight gradient of its columns in registers over all its rows, and
// the workgroup writes one partial row at the end, which a second kernel sums
// in order (30000 x 2048: 124 us with a partial row per four rows' threads).
// While a row is reduced and written, the next row's s and dy are on their
// way; rows stay packed in registers, and bf16 weights over all rows, while
// fp32 weights, twice as many registers, are loaded again.  Bound by HBM: 16640 x
// 8192 with dres 188 us (6.0 TB/s; 243 us without the next row's loads in
// flight), with an fp32 weight 210 us.
template <int TPR, int CH, bool WF32>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void rms_norm_bwd_kernel(const NormBwdArgs p) {
  constexpr int BLOCK = TPR < 256 ? 256 : TPR;
  constexpr int RPW = BLOCK / TPR;
  __shared__ float red[2][BLOCK / 64];
  const int sub = row_slot<TPR>(), t = threadIdx.x % TPR;
  const int cols = (int)p.cols;
  float acc[CH][8] = {};
  Weight8<WF32> wk[CH];
  if constexpr (!WF32) {
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      wk[k].load(p.weight.p, col < cols ? col : 0);
    }
  }
  uint4 u[CH], g[CH];
  auto load_row = [&](int64_t r) {
    const uint16_t* const s = p.s + r * p.ld_s;
    const uint16_t* const dy = p.dy + r * p.ld_dy;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      u[k] = g[k] = make_uint4(0, 0, 0, 0);
      if (col < cols) {
        u[k] = load_stream(s + col);
        g[k] = load_stream(dy + col);
      }
    }
  };
  int flip = 0;
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t r = (int64_t)blockIdx.x * RPW + sub;
  if (r < p.rows) load_row(r);
  for (; r < p.rows; r += step) {
    uint4 e[CH], cu[CH], cg[CH];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      e[k] = make_uint4(0, 0, 0, 0);
      if (p.dres && col < cols) e[k] = load_stream(p.dres + r * p.ld_dres + col);
      cu[k] = u[k];
      cg[k] = g[k];
    }
    if (r + step < p.rows) load_row(r + step);
    const float rstd = p.rstd[r];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      float h[8], d[8], w[8];
      if constexpr (WF32) wk[k].load(p.weight.p, col < cols ? col : 0);
      else keep_packed(wk[k].a);
      wk[k].get(w);
      unpack8(cu[k], h);
      unpack8(cg[k], d);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        h[c] *= rstd;
        acc[k][c] = __builtin_fmaf(d[c], h[c], acc[k][c]);
        dot = __builtin_fmaf(d[c] * w[c], h[c], dot);
      }
    }
    // the two halves of `red` alternate, so one barrier a row suffices
    const float mean = row_sum<TPR>(dot, red[flip]) / (float)cols;
    flip ^= 1;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int col = (k * TPR + t) * 8;
      keep_packed(cu[k]);
      keep_packed(cg[k]);
      float h[8], d[8], w[8], z[8];
      if constexpr (WF32) wk[k].load(p.weight.p, col < cols ? col : 0);
      else keep_packed(wk[k].a);
      wk[k].get(w);
      unpack8(cu[k], h);
      unpack8(cg[k], d);
      unpack8(e[k], z);
#pragma unroll
      for (int c = 0; c < 8; ++c) z[c] += rstd * (d[c] * w[c] - (h[c] * rstd) * mean);
      if (col < cols) *(uint4*)(p.dx + r * p.ld_dx + col) = pack8(z);
    }
  }
  // The workgroup's rows, in order, in one partial row.
  if constexpr (RPW > 1) {
    __shared__ __attribute__((aligned(16))) float rest[RPW - 1][CH][TPR][8];
    if (sub) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int c = 0; c < 8; ++c) rest[sub - 1][k][t][c] = acc[k][c];
    }
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < RPW - 1; ++i)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[k][c] += rest[i][k][t][c];
  }
  float* const part = p.partial + (int64_t)blockIdx.x * p.cols;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int col = (k * TPR + t) * 8;
    if (col < p.cols) {
      *(float4*)(part + col) = make_float4(acc[k][0], acc[k][1], acc[k][2], acc[k][3]);
      *(float4*)(part + col + 4) = make_float4(acc[k][4], acc[k][5], acc[k][6], acc[k][7]);
    }
  }
}

// dweight[c] = sum over the partial rows, in order: 32 columns (one 128-byte
// line a row) x 32 row groups a workgroup, the groups joined through LDS.
__global__ __launch_bounds__(1024) void rms_norm_dweight_kernel(const float* __restrict__ partial,
                                                                int parts, int64_t cols,
                                                                void* __restrict__ dw, int f32) {
  __shared__ float red[32][33];
  const int c = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  float v = 0.f;
  if (col < cols) {
#pragma unroll 8
    for (int i = grp; i < parts; i += 32) v += partial[(int64_t)i * cols + col];
  }
  red[grp][c] = v;
  __syncthreads();
  if (grp == 0 && col < cols) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += red[i][c];
    if (f32) ((float*)dw)[col] = v;
    else ((uint16_t*)dw)[col] = (uint16_t)f32_to_bf16_rne(v);
  }
}

// ---------------------------------------------------------------------------
// Threads per row and chunks per thread.  With many rows the row stays with
// as few threads as hold it in at most 4 chunks (cheapest reduction); with
// fewer rows than fill the chip a row gets as many threads as it has chunks.
static void norm_shape(int64_t rows, int64_t cols, int* tpr, int* ch) {
  const int64_t chunks = cols / 8;
  int t = 64;
  if (rows >= 512) {
    while (t < 1024 && chunks > 4 * t) t *= 4;
  } else {
    while (t < 1024 && chunks > t) t *= 4;
  }
  int c = 1;
  while (c * t < chunks) c *= 2;
  *tpr = t;
  *ch = c;
}

#define FP8BW_NORM_DISPATCH(KERNEL, ...)                                     \
  do {                                                                       \
    if (tpr == 64 && ch == 1) KERNEL(64, 1);                                 \
    else if (tpr == 64 && ch == 2) KERNEL(64, 2);                            \
    else if (tpr == 64) KERNEL(64, 4);                                       \
    else if (tpr == 256 && ch == 1) KERNEL(256, 1);                          \
    else if (tpr == 256 && ch == 2) KERNEL(256, 2);                          \
    else if (tpr == 256) KERNEL(256, 4);                                     \
    else if (ch == 1) KERNEL(1024, 1);                                       \
    else KERNEL(1024, 2);                                                    \
  } while (0)

static hipError_t launch_norm_rows(const NormFwdArgs& p, int tpr, int ch, hipStream_t stream) {
  const int block = tpr < 256 ? 256 : tpr;
  const unsigned grid = (unsigned)((p.rows + block / tpr - 1) / (block / tpr));
#define FP8BW_K(T, C) hipLaunchKernelGGL((rms_norm_fwd_kernel<T, C>), dim3(grid), dim3(block), 0, stream, p)
  FP8BW_NORM_DISPATCH(FP8BW_K);
#undef FP8BW_K
  return hipGetLastError();
}

hipError_t launch_rms_norm_fwd(const NormFwdArgs& p, hipStream_t stream) {
  int tpr, ch;
  norm_shape(p.rows, p.cols, &tpr, &ch);
  const hipError_t e = launch_norm_rows(p, tpr, ch, stream);
  if (e != hipSuccess || !p.qt) return e;
  hipLaunchKernelGGL(rms_norm_quant_t_kernel,
                     dim3((unsigned)((p.cols + 127) / 128), (unsigned)((p.rows + 127) / 128)),
                     dim3(256), 0, stream, p);
  return hipGetLastError();
}

// Workgroups of the backward (at most); each writes a partial row.
constexpr int kNormBwdGroups = 1024;
static int norm_bwd_grid(int64_t rows, int rpw) {
  const int64_t n = (rows + rpw - 1) / rpw;
  return (int)(n < kNormBwdGroups ? n : kNormBwdGroups);
}

size_t rms_norm_bwd_ws_bytes(int64_t rows, int64_t cols) {
  int tpr, ch;
  norm_shape(rows, cols, &tpr, &ch);
  const int rpw = tpr < 256 ? 256 / tpr : 1;
  return (size_t)norm_bwd_grid(rows, rpw) * (size_t)cols * sizeof(float);
}

hipError_t launch_rms_norm_bwd(const NormBwdArgs& p, hipStream_t stream) {
  int tpr, ch;
  norm_shape(p.rows, p.cols, &tpr, &ch);
  const int block = tpr < 256 ? 256 : tpr;
  const int rpw = block / tpr;
  const int grid = norm_bwd_grid(p.rows, rpw);
#define FP8BW_K(T, C)                                                                                    \
  do {                                                                                                   \
    if (p.weight.f32) hipLaunchKernelGGL((rms_norm_bwd_kernel<T, C, true>), dim3(grid), dim3(block), 0, stream, p); \
    else hipLaunchKernelGGL((rms_norm_bwd_kernel<T, C, false>), dim3(grid), dim3(block), 0, stream, p);  \
  } while (0)
  FP8BW_NORM_DISPATCH(FP8BW_K);
#undef FP8BW_K
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(rms_norm_dweight_kernel, dim3((unsigned)((p.cols + 31) / 32)), dim3(1024), 0, stream,
                     p.partial, grid, p.cols, p.dweight, p.weight.f32);
  return hipGetLastError();
}

}  // namespace fp8bw
