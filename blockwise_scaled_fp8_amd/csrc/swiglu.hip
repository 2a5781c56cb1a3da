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

// Writes one 16-lane row's 1x128 block of codes of f and its reciprocal scale.
__device__ __forceinline__ void put_codes8(const float (&f)[8], uint8_t* q, float* recip, bool in) {
  const float s = scale_from_amax(row16_max(absmax8(f)));
  const uint2 code = codes8(f, s);
  if (in) {
    *(uint2*)q = code;
    if ((threadIdx.x & 15) == 0) *recip = recip_of_scale(s);
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
// Rows: a wave takes P pieces of 512 columns of a row of v, all loads in flight
// first; a 16-lane DPP row holds one 1x128 block of each half.
template <int P>
__global__ __launch_bounds__(256) void swiglu_fwd_rows_kernel(const SwigluFwdArgs p, int64_t pieces) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  HalfIn gate[P], up[P];
  int64_t row[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t item = (int64_t)blockIdx.x * 4 * P + 4 * k + wave;
    row[k] = item / pieces;
    col[k] = (item - row[k] * pieces) * 512 + lane * 8;
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
    if (p.out.q) put_codes8(v, p.out.q + r * p.out.ld_q + c0, p.out.recip + r * p.out.rs_row + kb * p.out.rs_kb, in[k]);
    if (p.hq) {
      uint8_t* const hq = p.hq + r * p.ld_hq + c0;
      float* const hr = p.h_recip + r * p.hr_row + kb * p.hr_kb;
      put_codes8(g, hq, hr, in[k]);
      put_codes8(u, hq + p.ffn, hr + blocks * p.hr_kb, in[k]);
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
__global__ __launch_bounds__(256) void swiglu_bwd_rows_kernel(const SwigluBwdArgs p, int64_t pieces) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  HalfIn gate[P], up[P];
  uint4 dy[P];
  int64_t row[P], col[P];
  bool in[P];
#pragma unroll
  for (int k = 0; k < P; ++k) {
    const int64_t item = (int64_t)blockIdx.x * 4 * P + 4 * k + wave;
    row[k] = item / pieces;
    col[k] = (item - row[k] * pieces) * 512 + lane * 8;
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
    const int64_t r = row[k], c0 = col[k], kb = c0 >> 7;
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
      float* const recip = p.dh.recip + r * p.dh.rs_row + kb * p.dh.rs_kb;
      put_codes8(g, q, recip, in[k]);
      put_codes8(u, q + p.ffn, recip + blocks * p.dh.rs_kb, in[k]);
    }
  }
}

// ---------------------------------------------------------------------------
// Tiles: 128 rows x 128 columns of v (and of both halves), from which the
// transposed codes and every other layout are written.
__device__ __forceinline__ void store_transposed(uint8_t* qt, int64_t ld_qt, int64_t cols, int64_t rows, int64_t cb,
                                                 int64_t rb, int oc, int seg, const uint4& w) {
  const int64_t orow = cb * 128 + oc, ocol = rb * 128 + 16 * seg;
  if (orow < cols && ocol < rows) {
    const u32x4 t = {w.x, w.y, w.z, w.w};
    __builtin_nontemporal_store(t, (u32x4*)(qt + orow * ld_qt + ocol));
  }
}

__global__ __launch_bounds__(512, 4) void swiglu_fwd_tile_kernel(const SwigluFwdArgs p, int col_tiles) {
  __shared__ TileLds<1> L;
  const int tid = threadIdx.x, g16 = tid & 15, j = tid >> 4;
  const int64_t rb = blockIdx.x / col_tiles, cb = blockIdx.x - rb * col_tiles;
  const int64_t col = cb * 128 + g16 * 8, blocks = (p.ffn + 127) >> 7;
  const LayoutsOut& o = p.out;
  HalfIn gate[4], up[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = rb * 128 + 4 * j + k;
    const bool in = col < p.ffn && r < p.rows;
    gate[k] = load_half<false>(p.h, p.ld_h, nullptr, 0, 0, p.ffn, r, col, 0, in);
    up[k] = load_half<false>(p.h, p.ld_h, nullptr, 0, 0, p.ffn, r, col, 1, in);
  }
  float v[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = rb * 128 + 4 * j + k;
    const bool in = col < p.ffn && r < p.rows;
    float g[8], u[8];
    half_values<false>(gate[k], g);
    half_values<false>(up[k], u);
#pragma unroll
    for (int c = 0; c < 8; ++c) v[k][c] = g[c] * sigmoid(g[c]) * u[c];
    if (o.y && in) *(uint4*)(o.y + r * o.ld_y + col) = pack8(v[k]);
    if (o.q) put_codes8(v[k], o.q + r * o.ld_q + col, o.recip + r * o.rs_row + cb * o.rs_kb, in);
    if (p.hq) {
      uint8_t* const hq = p.hq + r * p.ld_hq + col;
      float* const hr = p.h_recip + r * p.hr_row + cb * p.hr_kb;
      put_codes8(g, hq, hr, in);
      put_codes8(u, hq + p.ffn, hr + blocks * p.hr_kb, in);
    }
  }
  tile_column_max(L, 0, v);
  __syncthreads();
  if (tid < 128) {
    const float s = tile_column_scale(L, 0, tid);
    if (cb * 128 + tid < p.ffn) o.recip_t[(cb * 128 + tid) * o.rst_row + rb * o.rst_kb] = recip_of_scale(s);
  }
  __syncthreads();
  tile_codes(L, 0, v);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int id = tid + 512 * i, oc = id >> 3, seg = id & 7;
    store_transposed(o.qt, o.ld_qt, p.ffn, p.rows, cb, rb, oc, seg, tile_piece(L, 0, oc, seg));
  }
}

// Arrays of a tile: 0 dg, 1 du, 2 v.
template <bool CODES>
__global__ __launch_bounds__(512, 4) void swiglu_bwd_tile_kernel(const SwigluBwdArgs p, int col_tiles) {
  __shared__ TileLds<3> L;
  const int tid = threadIdx.x, g16 = tid & 15, j = tid >> 4;
  const int64_t rb = blockIdx.x / col_tiles, cb = blockIdx.x - rb * col_tiles;
  const int64_t col = cb * 128 + g16 * 8, blocks = (p.ffn + 127) >> 7;
  HalfIn gate[4], up[4];
  uint4 dy[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = rb * 128 + 4 * j + k;
    const bool in = col < p.ffn && r < p.rows;
    gate[k] = load_half<CODES>(p.h, p.ld_h, p.h_recip, p.hr_row, p.hr_kb, p.ffn, r, col, 0, in);
    up[k] = load_half<CODES>(p.h, p.ld_h, p.h_recip, p.hr_row, p.hr_kb, p.ffn, r, col, 1, in);
    dy[k] = load_stream(p.dy + (in ? r * p.ld_dy + col : 0));
    if (!in) dy[k] = make_uint4(0, 0, 0, 0);
  }
  float g[4][8], u[4][8], d[4][8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int64_t r = rb * 128 + 4 * j + k;
    const bool in = col < p.ffn && r < p.rows;
    half_values<CODES>(gate[k], g[k]);
    half_values<CODES>(up[k], u[k]);
    unpack8(dy[k], d[k]);
#pragma unroll
    for (int c = 0; c < 8; ++c) swiglu_grad(g[k][c], u[k][c], d[k][c]);
    if (p.dh.y && in) {
      uint16_t* const y = p.dh.y + r * p.dh.ld_y + col;
      *(uint4*)y = pack8(g[k]);
      *(uint4*)(y + p.ffn) = pack8(u[k]);
    }
    if (p.dh.q) {
      uint8_t* const q = p.dh.q + r * p.dh.ld_q + col;
      float* const recip = p.dh.recip + r * p.dh.rs_row + cb * p.dh.rs_kb;
      put_codes8(g[k], q, recip, in);
      put_codes8(u[k], q + p.ffn, recip + blocks * p.dh.rs_kb, in);
    }
  }
  tile_column_max(L, 0, g);
  tile_column_max(L, 1, u);
  tile_column_max(L, 2, d);
  __syncthreads();
  if (tid < 384) {
    const int a = tid >> 7, c = tid & 127;
    const float recip = recip_of_scale(tile_column_scale(L, a, c));
    if (cb * 128 + c < p.ffn) {
      if (a < 2 && p.dh.qt) p.dh.recip_t[(a * p.ffn + cb * 128 + c) * p.dh.rst_row + rb * p.dh.rst_kb] = recip;
      if (a == 2 && p.act_qt) p.act_recip_t[(cb * 128 + c) * p.art_row + rb * p.art_kb] = recip;
    }
  }
  __syncthreads();
  tile_codes(L, 0, g);
  tile_codes(L, 1, u);
  tile_codes(L, 2, d);
  __syncthreads();
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    if (a < 2 ? !p.dh.qt : !p.act_qt) continue;
    uint8_t* const qt = a < 2 ? p.dh.qt + a * p.ffn * p.dh.ld_qt : p.act_qt;
    const int64_t ld = a < 2 ? p.dh.ld_qt : p.ld_act_qt;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int id = tid + 512 * i, oc = id >> 3, seg = id & 7;
      store_transposed(qt, ld, p.ffn, p.rows, cb, rb, oc, seg, tile_piece(L, a, oc, seg));
    }
  }
}

// Four pieces a wave once that still leaves several workgroups per compute unit.
constexpr int64_t kManyPieces = 8192;

hipError_t launch_swiglu_fwd(const SwigluFwdArgs& p, hipStream_t stream) {
  if (p.out.qt) {
    const int64_t ct = (p.ffn + 127) / 128, tiles = ct * ((p.rows + 127) / 128);
    hipLaunchKernelGGL(swiglu_fwd_tile_kernel, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.ffn + 511) / 512, items = p.rows * pieces;
  if (items >= kManyPieces)
    hipLaunchKernelGGL(swiglu_fwd_rows_kernel<4>, dim3((unsigned)((items + 15) / 16)), dim3(256), 0, stream, p, pieces);
  else
    hipLaunchKernelGGL(swiglu_fwd_rows_kernel<1>, dim3((unsigned)((items + 3) / 4)), dim3(256), 0, stream, p, pieces);
  return hipGetLastError();
}

hipError_t launch_swiglu_bwd(const SwigluBwdArgs& p, hipStream_t stream) {
  if (p.dh.qt || p.act_qt) {
    const int64_t ct = (p.ffn + 127) / 128, tiles = ct * ((p.rows + 127) / 128);
    if (p.h_recip)
      hipLaunchKernelGGL(swiglu_bwd_tile_kernel<true>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    else
      hipLaunchKernelGGL(swiglu_bwd_tile_kernel<false>, dim3((unsigned)tiles), dim3(512), 0, stream, p, (int)ct);
    return hipGetLastError();
  }
  const int64_t pieces = (p.ffn + 511) / 512, items = p.rows * pieces;
  const bool many = items >= kManyPieces;
  const dim3 grid((unsigned)(many ? (items + 15) / 16 : (items + 3) / 4));
#define FP8BW_K(P, C) hipLaunchKernelGGL((swiglu_bwd_rows_kernel<P, C>), grid, dim3(256), 0, stream, p, pieces)
  if (p.h_recip) {
    if (many) FP8BW_K(4, true);
    else FP8BW_K(1, true);
  } else {
    if (many) FP8BW_K(4, false);
    else FP8BW_K(1, false);
  }
#undef FP8BW_K
  return hipGetLastError();
}

}  // namespace fp8bw
