// The gated activation between an FP8 MLP's two products for gfx950, with E4M3
// outputs, 8-bit checkpoints and the backward pass from either.
//
//   h = [g | u], v = silu(g) u = g s u,  s = sigmoid(g) = 1 / (1 + exp(-g))
//   dg = dv u s (1 + g (1 - s)),  du = dv g s
//
// A checkpoint is h in E4M3 codes with a scale per 1x128 block of each half;
// the backward from it computes with the values the codes stand for.  All
// arithmetic is fp32; exp is the hardware's exp2 of g log2(e) and 1 / (1 + e)
// its reciprocal (1 ulp each; the product's rounding adds |g| 2^-24 to exp's
// relative error), far below the outputs' bf16 or E4M3 step.
//
// Everything here streams: each input is read once with 16-byte (codes: 8-byte)
// loads, and every layout is written from registers.

#include "launch.h"
#include "vec8.h"

namespace fp8bw {

// Below 2^-126 (g under -87.3) s may be flushed, and is 0 where exp(-g) is
// infinite; g s is then -0, as g / (1 + exp(-g)) is.
__device__ __forceinline__ float sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g * -1.44269504088896341f));
}

// KEPT: codes that nothing reads before the backward, which pass the caches by and
// leave them to the next product's operand (33280 rows of 2 x 5120: this kernel
// after itself 233 -> 197 us, with an 8192 x 5120 product behind it 1415 -> 1350;
// the operand's own codes written that way too: 212 and 1380).
template <bool KEPT = false>
__device__ __forceinline__ void put_codes8(const float (&f)[8], float scale, uint8_t* q, bool in) {
  const uint2 code = codes8(f, scale);
  if (!in) return;
  if constexpr (KEPT) {
    const u32x2 c = {code.x, code.y};
    __builtin_nontemporal_store(c, (u32x2*)q);
  } else {
    *(uint2*)q = code;
  }
}

// Eight values of row r, columns col .. + 7 of one half of h: `half` 0 the gate,
// 1 the other.
struct HalfIn {
  uint4 raw;      // 8 bf16, or 8 codes in x and y
  float recip;
};
template <bool CODES>
__device__ __forceinline__ HalfIn load_half(const void* h, int64_t ld_h, const float* recip, int64_t hr_row,
                                            int64_t hr_kb, int64_t ffn, int64_t r, int64_t col, int half, bool in) {
  HalfIn x;
  x.recip = 0.f;
  if constexpr (CODES) {
    const uint8_t* const q = (const uint8_t*)h + (in ? r * ld_h + half * ffn + col : 0);
    const u32x2 t = __builtin_nontemporal_load((const u32x2*)q);
    x.raw = make_uint4(t.x, t.y, 0, 0);
    const int64_t blocks = (ffn + 127) >> 7;
    x.recip = recip[in ? r * hr_row + (half * blocks + (col >> 7)) * hr_kb : 0];
  } else {
    x.raw = load_stream((const uint16_t*)h + (in ? r * ld_h + half * ffn + col : 0));
  }
  if (!in) x.raw = make_uint4(0, 0, 0, 0);
  return x;
}
template <bool CODES>
__device__ __forceinline__ void half_values(const HalfIn& x, float (&f)[8]) {
  if constexpr (CODES) values8(make_uint2(x.raw.x, x.raw.y), x.recip, f);
  else unpack8(x.raw, f);
}

// ---------------------------------------------------------------------------
// Rows: a wave takes a piece of 512 columns of P rows of v, all loads in flight
// first; a 16-lane DPP row holds one 1x128 block of each half, and the three scales
// of v, g and u are divided by three of its lanes at once.  A workgroup's 4 P rows
// follow one another, so that their scales, which lie row by row, leave in whole
// 32-byte sectors (with the pieces of a row side by side instead 98 MB more are
// written of 527, and 211 us against 204).  HBM: codes and checkpoint of 33280 rows
// of 2 x 5120, 204 us for 1.21 GB (5.9 TB/s); 8 rows of 2 x 8192 2.7 us, the launch.
template <int P>
struct RowPieces {
  int row[P];
  int col;   // first column
  __device__ __forceinline__ RowPieces(uint32_t workgroup, uint32_t pieces) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t r = workgroup / pieces;
    col = (int)(workgroup - r * pieces) * 512;
#pragma unroll
    for (int k = 0; k < P; ++k) row[k] = (int)((4 * r + wave) * P) + k;
  }
};

template <int P>
__global__ __launch_bounds__(256) void swiglu_fwd_rows_kernel(const SwigluFwdArgs p, uint32_t pieces) {
  const int lane = threadIdx.x & 63;
  const RowPieces<P> at(blockIdx.x, pieces);
  HalfIn gate[P], up[P];
  int64_t row[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    row[k] = at.row[k];
    col[k] = at.col + lane * 8;
    in[k] = row[k] < p.rows && col[k] < p.ffn;
    gate[k] = load_half<false>(p.h, p.ld_h, nullptr, 0, 0, p.ffn, row[k], col[k], 0, in[k]);
    up[k] = load_half<false>(p.h, p.ld_h, nullptr, 0, 0, p.ffn, row[k], col[k], 1, in[k]);
  }
  const int64_t blocks = (p.ffn + 127) >> 7;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (row[k] >= p.rows) return;
    const int64_t r = row[k], c0 = col[k], kb = c0 >> 7;
    float g[8], u[8], v[8];
    half_values<false>(gate[k], g);
    half_values<false>(up[k], u);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[c] = g[c] * sigmoid(g[c]) * u[c];
    if (p.out.y && in[k]) *(uint4*)(p.out.y + r * p.out.ld_y + c0) = pack8(v);
    if (!p.out.q && !p.hq) continue;
    // three blocks: v, g, u
    const float amax[3] = {row16_amax(v), row16_amax(g), row16_amax(u)};
    float scale[3];
    const float recip = row16_scales(amax, scale);
    const int i = lane & 15;   // writes the scale of block i
    if (p.out.q) {
      put_codes8(v, scale[0], p.out.q + r * p.out.ld_q + c0, in[k]);
      if (in[k] && i == 0) p.out.recip[r * p.out.rs_row + kb * p.out.rs_kb] = recip;
    }
    if (p.hq) {
      uint8_t* const hq = p.hq + r * p.ld_hq + c0;
      put_codes8<true>(g, scale[1], hq, in[k]);
      put_codes8<true>(u, scale[2], hq + p.ffn, in[k]);
      const int64_t first = c0 - 8 * i;   // the block's first column: in range where the block has any
      if (first < p.ffn && (i == 1 || i == 2))
        p.h_recip[r * p.hr_row + ((i - 1) * blocks + (first >> 7)) * p.hr_kb] = recip;
    }
  }
}

// The gradients of eight values, in the place of the inputs: g <- dg, u <- du,
// d <- v.
__device__ __forceinline__ void swiglu_grad(float& g, float& u, float& d) {
  const float s = sigmoid(g), a = g * s;
  const float v = a * u, dg = d * u * __builtin_fmaf(a, 1.f - s, s), du = d * a;
  g = dg;
  u = du;
  d = v;
}

template <int P, bool CODES>
__global__ __launch_bounds__(256) void swiglu_bwd_rows_kernel(const SwigluBwdArgs p, uint32_t pieces) {
  const int lane = threadIdx.x & 63;
  const RowPieces<P> at(blockIdx.x, pieces);
  HalfIn gate[P], up[P];
  uint4 dy[P];
  int64_t row[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    row[k] = at.row[k];
    col[k] = at.col + lane * 8;
    in[k] = row[k] < p.rows && col[k] < p.ffn;
    dy[k] = load_stream(p.dy + (in[k] ? row[k] * p.ld_dy + col[k] : 0));
    gate[k] = load_half<CODES>(p.h, p.ld_h, p.h_recip, p.hr_row, p.hr_kb, p.ffn, row[k], col[k], 0, in[k]);
    up[k] = load_half<CODES>(p.h, p.ld_h, p.h_recip, p.hr_row, p.hr_kb, p.ffn, row[k], col[k], 1, in[k]);
    if (!in[k]) dy[k] = make_uint4(0, 0, 0, 0);
  }
  const int64_t blocks = (p.ffn + 127) >> 7;
#pragma unroll
  for (int k = 0; k < P; ++k) {
    if (row[k] >= p.rows) return;
    const int64_t r = row[k], c0 = col[k];
    float g[8], u[8], d[8];
    half_values<CODES>(gate[k], g);
    half_values<CODES>(up[k], u);
    unpack8(dy[k], d);
#pragma unroll
    for (int c = 0; c < 8; ++c) swiglu_grad(g[c], u[c], d[c]);
    if (p.dh.y && in[k]) {
      uint16_t* const y = p.dh.y + r * p.dh.ld_y + c0;
      *(uint4*)y = pack8(g);
      *(uint4*)(y + p.ffn) = pack8(u);
    }
    if (p.dh.q) {
      uint8_t* const q = p.dh.q + r * p.dh.ld_q + c0;
      const float amax[2] = {row16_amax(g), row16_amax(u)};
      float scale[2];
      const float recip = row16_scales(amax, scale);
      put_codes8(g, scale[0], q, in[k]);
      put_codes8(u, scale[1], q + p.ffn, in[k]);
      const int i = lane & 15;
      const int64_t first = c0 - 8 * i;
      if (first < p.ffn && i < 2) p.dh.recip[r * p.dh.rs_row + (i * blocks + (first >> 7)) * p.dh.rs_kb] = recip;
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: 128 rows x 128 columns of v (and of both halves), from which the
// transposed codes and every other layout are written.  A tile's corner is in
// scalar registers and a thread's offsets from it in 32 bits (the host keeps
// 128 leading dimensions below 2^31 bytes): with 64-bit addresses a lane the
// backward spilled.  The backward's column maxima come before its row codes: the
// magnitudes that both use then cost no instruction of their own (455 to 328 us in
// all).  HBM, with the vector pipe close behind: 33280 rows of 2 x 5120 from a
// checkpoint, dh in both code layouts and the activation's transposed codes, 326 us
// for 1.57 GB, 4.8 TB/s.
struct Tile {
  int64_t rb, cb;     // row and column block
  int row, col;       // this thread's first row and column, of 4 and of 8
  int rows, cols;     // of the tile that exist
};
__device__ __forceinline__ Tile tile_of(int64_t rows, int64_t ffn, int col_tiles) {
  Tile t;
  t.rb = blockIdx.x / col_tiles;
  t.cb = blockIdx.x - t.rb * col_tiles;
  t.row = (threadIdx.x >> 4) * 4;
  t.col = (threadIdx.x & 15) * 8;
  t.rows = (int)min(rows - t.rb * 128, (int64_t)128);
  t.cols = (int)min(ffn - t.cb * 128, (int64_t)128);
  return t;
}

// Both halves of h's rows, as the row kernels hold them.
template <bool CODES>
__device__ __forceinline__ void load_tile_halves(const Tile& t, const void* h, int64_t ld_h, const float* recip,
                                                 int64_t hr_row, int64_t hr_kb, int64_t ffn, HalfIn (&gate)[4],
                                                 HalfIn (&up)[4]) {
  const int64_t corner = t.rb * 128 * ld_h + t.cb * 128, blocks = (ffn + 127) >> 7;
  const float* const gr = CODES ? recip + t.rb * 128 * hr_row + t.cb * hr_kb : nullptr;
  const float* const ur = CODES ? gr + blocks * hr_kb : nullptr;
  const uint32_t row_at = t.row * (uint32_t)ld_h + t.col, recip_at = t.row * (uint32_t)hr_row;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool in = t.row + k < t.rows && t.col < t.cols;
    const uint32_t at = in ? row_at + (uint32_t)k * (uint32_t)ld_h : 0;
    if constexpr (CODES) {
      const uint8_t* const g = (const uint8_t*)h + corner;
      const u32x2 a = __builtin_nontemporal_load((const u32x2*)(g + at));
      const u32x2 b = __builtin_nontemporal_load((const u32x2*)(g + ffn + at));
      gate[k].raw = in ? make_uint4(a.x, a.y, 0, 0) : make_uint4(0, 0, 0, 0);
      up[k].raw = in ? make_uint4(b.x, b.y, 0, 0) : make_uint4(0, 0, 0, 0);
      const uint32_t ar = in ? recip_at + (uint32_t)k * (uint32_t)hr_row : 0;
      gate[k].recip = gr[ar];
      up[k].recip = ur[ar];
    } else {
      const uint16_t* const g = (const uint16_t*)h + corner;
      gate[k].raw = load_stream(g + at);
      up[k].raw = load_stream(g + ffn + at);
      if (!in) gate[k].raw = up[k].raw = make_uint4(0, 0, 0, 0);
    }
  }
}

template <bool CODES>
__global__ __launch_bounds__(512, 4) void swiglu_fwd_tile_kernel(const SwigluFwdArgs p, int col_tiles) {
  __shared__ TileLds<1, 4> L;
  const Tile t = tile_of(p.rows, p.ffn, col_tiles);
  const int tid = threadIdx.x, lane16 = tid & 15;
  const int64_t blocks = (p.ffn + 127) >> 7;
  const LayoutsOut& o = p.out;
  HalfIn gate[4], up[4];
  load_tile_halves<CODES>(t, p.h, p.ld_h, p.in_recip, p.ir_row, p.ir_kb, p.ffn, gate, up);
  float v[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = t.rb * 128 + t.row + k;
    const bool row_in = t.row + k < t.rows, in = row_in && t.col < t.cols;
    float g[8], u[8];
    half_values<CODES>(gate[k], g);
    half_values<CODES>(up[k], u);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[k][c] = g[c] * sigmoid(g[c]) * u[c];
    if constexpr (CODES) continue;
    const int64_t col = t.cb * 128 + t.col;
    if (o.y && in) *(uint4*)(o.y + r * o.ld_y + col) = pack8(v[k]);
    if (!o.q && !p.hq) continue;
    const float amax[3] = {row16_amax(v[k]), row16_amax(g), row16_amax(u)};
    float scale[3];
    const float recip = row16_scales(amax, scale);
    if (o.q) {
      put_codes8(v[k], scale[0], o.q + r * o.ld_q + col, in);
      if (lane16 == 0 && row_in) o.recip[r * o.rs_row + t.cb * o.rs_kb] = recip;
    }
    if (p.hq) {
      uint8_t* const hq = p.hq + r * p.ld_hq + col;
      put_codes8<true>(g, scale[1], hq, in);
      put_codes8<true>(u, scale[2], hq + p.ffn, in);
      if ((lane16 == 1 || lane16 == 2) && row_in)
        p.h_recip[r * p.hr_row + ((lane16 - 1) * blocks + t.cb) * p.hr_kb] = recip;
    }
  }
  tile_column_max(L, 0, v);
  __syncthreads();
  if (tid < 128) {
    const float s = tile_column_scale(L, 0, tid);
    if (tid < t.cols) o.recip_t[(t.cb * 128 + tid) * o.rst_row + t.rb * o.rst_kb] = recip_of_scale(s);
  }
  __syncthreads();
  tile_codes(L, 0, v);
  __syncthreads();
  store_transposed(L, 0, o.qt + t.cb * 128 * o.ld_qt + t.rb * 128, o.ld_qt, t.rows, t.cols);
}

// Arrays of a tile: 0 dg, 1 du, 2 v.
template <bool CODES>
__global__ __launch_bounds__(512, 4) void swiglu_bwd_tile_kernel(const SwigluBwdArgs p, int col_tiles) {
  __shared__ TileLds<3, 4> L;
  const Tile t = tile_of(p.rows, p.ffn, col_tiles);
  const int tid = threadIdx.x, lane16 = tid & 15;
  const int64_t blocks = (p.ffn + 127) >> 7;
  const LayoutsOut& o = p.dh;
  HalfIn gate[4], up[4];
  uint4 dy[4];
  load_tile_halves<CODES>(t, p.h, p.ld_h, p.h_recip, p.hr_row, p.hr_kb, p.ffn, gate, up);
  const uint16_t* const dy_corner = p.dy + t.rb * 128 * p.ld_dy + t.cb * 128;
  const uint32_t dy_at = t.row * (uint32_t)p.ld_dy + t.col;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool in = t.row + k < t.rows && t.col < t.cols;
    dy[k] = load_stream(dy_corner + (in ? dy_at + (uint32_t)k * (uint32_t)p.ld_dy : 0));
    if (!in) dy[k] = make_uint4(0, 0, 0, 0);
  }
  float g[4][8], u[4][8], d[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    half_values<CODES>(gate[k], g[k]);
    half_values<CODES>(up[k], u[k]);
    unpack8(dy[k], d[k]);
#pragma unroll
    for (int c = 0; c < 8; ++c) swiglu_grad(g[k][c], u[k][c], d[k][c]);
    __builtin_amdgcn_sched_barrier(0);
  }
  tile_column_max(L, 0, g);
  tile_column_max(L, 1, u);
  tile_column_max(L, 2, d);
  if (o.y) {
    uint16_t* const corner = o.y + t.rb * 128 * o.ld_y + t.cb * 128;
    uint32_t at = t.row * (uint32_t)o.ld_y + t.col;
#pragma unroll
    for (int k = 0; k < 4; ++k, at += (uint32_t)o.ld_y) {
      if (t.row + k < t.rows && t.col < t.cols) {
        *(uint4*)(corner + at) = pack8(g[k]);
        *(uint4*)(corner + p.ffn + at) = pack8(u[k]);
      }
    }
  }
  if (o.q) {
    // the blocks of 4 rows of both halves: block i = 4 half + row
    float amax[8], scale[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      amax[k] = row16_amax(g[k]);
      amax[4 + k] = row16_amax(u[k]);
    }
    const float recip = row16_scales(amax, scale);
    uint8_t* const corner = o.q + t.rb * 128 * o.ld_q + t.cb * 128;
    uint32_t at = t.row * (uint32_t)o.ld_q + t.col;
#pragma unroll
    for (int k = 0; k < 4; ++k, at += (uint32_t)o.ld_q) {
      const bool in = t.row + k < t.rows && t.col < t.cols;
      put_codes8(g[k], scale[k], corner + at, in);
      put_codes8(u[k], scale[4 + k], corner + p.ffn + at, in);
    }
    if (lane16 < 8 && t.row + (lane16 & 3) < t.rows)
      o.recip[(t.rb * 128 + t.row + (lane16 & 3)) * o.rs_row + ((lane16 >> 2) * blocks + t.cb) * o.rs_kb] = recip;
  }
  __syncthreads();
  if (tid < 384) {
    const int a = tid >> 7, c = tid & 127;
    const float recip = recip_of_scale(tile_column_scale(L, a, c));
    if (c < t.cols) {
      if (a < 2 && o.qt) o.recip_t[(a * p.ffn + t.cb * 128 + c) * o.rst_row + t.rb * o.rst_kb] = recip;
      if (a == 2 && p.act_qt) p.act_recip_t[(t.cb * 128 + c) * p.art_row + t.rb * p.art_kb] = recip;
    }
  }
  __syncthreads();
  tile_codes(L, 0, g);
  __builtin_amdgcn_sched_barrier(0);
  tile_codes(L, 1, u);
  __builtin_amdgcn_sched_barrier(0);
  tile_codes(L, 2, d);
  __syncthreads();
  if (o.qt) {
    uint8_t* const corner = o.qt + t.cb * 128 * o.ld_qt + t.rb * 128;
    store_transposed(L, 0, corner, o.ld_qt, t.rows, t.cols);
    store_transposed(L, 1, corner + p.ffn * o.ld_qt, o.ld_qt, t.rows, t.cols);
  }
  if (p.act_qt)
    store_transposed(L, 2, p.act_qt + t.cb * 128 * p.ld_act_qt + t.rb * 128, p.ld_act_qt, t.rows, t.cols);
}

// Two rows a wave once that still leaves several workgroups per compute unit
// (forward, 33280 rows of 2 x 5120 with a checkpoint: 204 us with two, 207 with
// four, 224 with one and as many rows a workgroup as with four).
constexpr int64_t kManyPieces = 8192;
constexpr int kRows = 2;

static dim3 rows_grid(int64_t rows, int64_t pieces, int each) {
  return dim3((unsigned)((rows + 4 * each - 1) / (4 * each) * pieces));
}

hipError_t launch_swiglu_fwd(const SwigluFwdArgs& p, hipStream_t stream) {
  if (p.out.qt) {
    const int64_t ct = (p.ffn + 127) / 128, tiles = ct * ((p.rows + 127) / 128);
    if (p.in_recip)
      hipLaunchKernelGGL(swiglu_fwd_tile_kernel<true>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    else
      hipLaunchKernelGGL(swiglu_fwd_tile_kernel<false>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.ffn + 511) / 512;
  if (p.rows * pieces >= kManyPieces)
    hipLaunchKernelGGL(swiglu_fwd_rows_kernel<kRows>, rows_grid(p.rows, pieces, kRows), dim3(256), 0, stream, p, (uint32_t)pieces);
  else
    hipLaunchKernelGGL(swiglu_fwd_rows_kernel<1>, rows_grid(p.rows, pieces, 1), dim3(256), 0, stream, p, (uint32_t)pieces);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdArgs& p, hipStream_t stream) {
  // v^T alone: no gradient is computed and dy is not read (33280 rows of 2 x 5120: from a
  // checkpoint 108 us, from bf16 160).
  if (!p.dh.y && !p.dh.q && !p.dh.qt) {
    SwigluFwdArgs f = {};
    f.rows = p.rows; f.ffn = p.ffn;
    f.h = p.h; f.ld_h = p.ld_h;
    f.in_recip = p.h_recip; f.ir_row = p.hr_row; f.ir_kb = p.hr_kb;
    f.out.qt = p.act_qt; f.out.ld_qt = p.ld_act_qt;
    f.out.recip_t = p.act_recip_t; f.out.rst_row = p.art_row; f.out.rst_kb = p.art_kb;
    return launch_swiglu_fwd(f, stream);
  }
  if (p.dh.qt || p.act_qt) {
    const int64_t ct = (p.ffn + 127) / 128, tiles = ct * ((p.rows + 127) / 128);
    if (p.h_recip)
      hipLaunchKernelGGL(swiglu_bwd_tile_kernel<true>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    else
      hipLaunchKernelGGL(swiglu_bwd_tile_kernel<false>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.ffn + 511) / 512;
  const bool many = p.rows * pieces >= kManyPieces;
#define FP8BW_K(P, C) \
  hipLaunchKernelGGL((swiglu_bwd_rows_kernel<P, C>), rows_grid(p.rows, pieces, P), dim3(256), 0, stream, p, (uint32_t)pieces)
  if (p.h_recip) {
    if (many) FP8BW_K(kRows, true);
    else FP8BW_K(1, true);
  } else {
    if (many) FP8BW_K(kRows, false);
    else FP8BW_K(1, false);
  }
#undef FP8BW_K
  return hipGetLastError();
}

}  // namespace fp8bw
