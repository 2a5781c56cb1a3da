// What the streaming kernels share: eight bf16 values in a 16-byte vector,
// sums over a wavefront, and codes of 128 x 128 tiles of fp32 values in both
// layouts.
#pragma once

#include <type_traits>

#include "device_common.h"

namespace fp8bw {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16 bytes that nothing reads again soon: a load that leaves the caches alone.
__device__ __forceinline__ uint4 load_stream(const uint16_t* p) {
  const u32x4 t = __builtin_nontemporal_load((const u32x4*)p);
  return make_uint4(t.x, t.y, t.z, t.w);
}

// Sum over the 16 lanes of a DPP row, then over the wavefront; every lane
// receives the same value.
__device__ __forceinline__ float row16_sum(float v) {
  v += dpp_move<0xB1>(v);
  v += dpp_move<0x4E>(v);
  v += dpp_move<0x141>(v);
  v += dpp_move<0x140>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row16_sum(v);
  const int i = __float_as_int(v);
  const float a = __int_as_float(__builtin_amdgcn_readlane(i, 0));
  const float b = __int_as_float(__builtin_amdgcn_readlane(i, 16));
  const float c = __int_as_float(__builtin_amdgcn_readlane(i, 32));
  const float d = __int_as_float(__builtin_amdgcn_readlane(i, 48));
  return (a + b) + (c + d);
}

__device__ __forceinline__ void unpack8(const uint4& u, float (&f)[8]) {
  f[0] = bf16lo(u.x); f[1] = bf16hi(u.x);
  f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
  f[4] = bf16lo(u.z); f[5] = bf16hi(u.z);
  f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2_rne(f[0], f[1]), pack_bf16x2_rne(f[2], f[3]),
                    pack_bf16x2_rne(f[4], f[5]), pack_bf16x2_rne(f[6], f[7]));
}

__device__ __forceinline__ float absmax8(const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) m = fmaxf(m, fabsf(f[c]));
  return m;
}

// Largest of the 16 lanes of a DPP row, each holding the magnitude of its own 8
// values (never a NaN: a maximum from 0 ignores them).  As integers, in the same
// order: a float maximum of a value that came through a lane exchange takes three
// instructions, this takes one.
__device__ __forceinline__ float row16_amax(const float (&f)[8]) {
  uint32_t m = __float_as_uint(absmax8(f));
  auto step = [&](auto ctrl) {
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, decltype(ctrl)::value, 0xF, 0xF, true));
  };
  step(std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
  step(std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
  step(std::integral_constant<int, 0x141>{});   // row_half_mirror
  step(std::integral_constant<int, 0x140>{});   // row_mirror
  return __uint_as_float(m);
}

// Four E4M3 codes of values scaled by their own block's scale.  These need no
// clamp: |f| <= amax and s = 448 / max(amax, 1e-12) rounded give |f s| <= 448
// (1 + 2^-23), and what lies between 448 and 464 rounds to 448.  A NaN, which has no
// part in amax, and an infinity times its block's scale 0 become the NaN code (the
// quantizers' clamp would make them finite).
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r;
  asm("" : "=v"(r));   // any register: the two conversions write all of it
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}
// Eight E4M3 codes of f * s.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
  return make_uint2(codes4(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                    codes4(f[4] * s, f[5] * s, f[6] * s, f[7] * s));
}

// Lane I of each DPP row, to all its lanes (row_newbcast).
template <int I>
__device__ __forceinline__ float row16_lane(float v) {
  return dpp_move<0x150 + I>(v);
}

// Scales of N <= 16 blocks whose amaxes every lane of a DPP row holds.  Lane i
// divides for block i alone, 448 / amax and its reciprocal being the most
// expensive part of a block's codes (two IEEE divisions, 8 values a lane), and
// its scale is broadcast.  Returns, in lane i < N, block i's reciprocal.
template <int N, int I = 0>
__device__ __forceinline__ void row16_spread(float s, float (&scale)[N]) {
  if constexpr (I < N) {
    scale[I] = row16_lane<I>(s);
    row16_spread<N, I + 1>(s, scale);
  }
}
// amax[l] for a lane's own l < N, by selects (a loop over i would be turned into
// an array in memory indexed by l).
template <int N, int I = 1>
__device__ __forceinline__ float row16_pick(const float (&amax)[N], int l, float m) {
  if constexpr (I < N) return row16_pick<N, I + 1>(amax, l, l == I ? +amax[I] : m);
  else return m;
}
template <int N>
__device__ __forceinline__ float row16_scales(const float (&amax)[N], float (&scale)[N]) {
  static_assert(N <= 16, "one lane a block");
  const float s = scale_from_amax(row16_pick(amax, threadIdx.x & 15, amax[0]));
  row16_spread(s, scale);
  return recip_of_scale(s);
}

// Eight E4M3 codes' values times r.
__device__ __forceinline__ void values8(const uint2& q, float r, float (&f)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int w = h ? (int)q.y : (int)q.x;
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
    f[4 * h + 0] = lo.x * r; f[4 * h + 1] = lo.y * r;
    f[4 * h + 2] = hi.x * r; f[4 * h + 3] = hi.y * r;
  }
}

// P consecutive pieces of 512 columns of a wave, rows one after the other; `pieces`
// to a row, fewer than 2^30 in all.  One division, the rest by counting: P 64-bit
// divisions were most of a row kernel's scalar instructions.
template <int P>
struct Pieces {
  int row[P];
  int col[P];   // first column
  __device__ __forceinline__ Pieces(uint32_t workgroup, uint32_t pieces) {
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t first = (workgroup * 4 + wave) * P;
    uint32_t r = first / pieces, c = first - r * pieces;
#pragma unroll
    for (int k = 0; k < P; ++k) {
      row[k] = (int)r;
      col[k] = (int)c * 512;
      const bool next = ++c == pieces;
      r += next ? 1u : 0u;
      c = next ? 0u : c;
    }
  }
};

// ---------------------------------------------------------------------------
// Transposed codes of NA 128 x 128 tiles of fp32 values held by a workgroup of
// 2048 / R threads: thread (g = tid % 16, j = tid / 16) holds columns 8 g .. 8 g + 7
// of rows R j .. R j + R - 1, so a wave's loads cover 256-byte pieces of 4 rows
// and a 16-lane DPP row holds one 1x128 block of a row.  R = 8 spends the fewest
// instructions beside those an element needs (these kernels are as near the VALU's
// bound as HBM's); three arrays leave registers for R = 4 only.
//
// One scale per column: each column's R rows in registers, the 4 row groups of
// a wave by lane exchange, the waves through LDS.  A thread then quantizes its
// rows of a column into dwords of an LDS tile stored [column][row] (32 dwords a
// column); dword d of column c lies at d ^ 4 ((c / 8) % 8), which spreads a
// store's 16 column groups over the banks and keeps 16-byte groups whole, and the
// tile leaves as 16-byte pieces of output rows, 8 lanes a row.
template <int NA, int R>
struct TileLds {
  static_assert(R == 4 || R == 8, "whole dwords of rows");
  static constexpr int kWaves = 32 / R;
  float red[kWaves][NA][128];
  __attribute__((aligned(16))) float scale[NA][128];
  __attribute__((aligned(16))) uint32_t tile[NA][128 * 32];
};

// The column maxima of array a, into LDS.  Before the first barrier.  The wave's
// four row groups are joined two columns at a time: exchanging halves (then 16-lane
// rows) of two registers leaves in each lane pair one column's two values, so one
// exchange and one maximum serve both columns, and every lane writes.
__device__ __forceinline__ uint32_t max_halves(uint32_t x, uint32_t y) {
  const auto r = __builtin_amdgcn_permlane32_swap(x, y, false, false);
  return max(r[0], r[1]);   // x's maximum in lanes 0 .. 31, y's in 32 .. 63
}
__device__ __forceinline__ uint32_t max_rows(uint32_t x, uint32_t y) {
  const auto r = __builtin_amdgcn_permlane16_swap(x, y, false, false);
  return max(r[0], r[1]);   // rows 0, 2: x's, rows 1, 3: y's
}
template <int NA, int R>
__device__ __forceinline__ void tile_column_max(TileLds<NA, R>& L, int a, const float (&v)[R][8]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t m[8];   // as integers: magnitudes in the same order
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    // from 0, which ignores NaN: one left here would pass every magnitude below
    float f = 0.f;
#pragma unroll
    for (int k = 0; k < R; ++k) f = fmaxf(f, fabsf(v[k][c]));
    m[c] = __float_as_uint(f);
  }
  // 16-lane rows 0 .. 3 end with columns 0, 2, 1, 3 (and 4 further)
  const uint32_t lo = max_rows(max_halves(m[0], m[1]), max_halves(m[2], m[3]));
  const uint32_t hi = max_rows(max_halves(m[4], m[5]), max_halves(m[6], m[7]));
  float* const red = &L.red[wave][a][8 * (lane & 15) + ((lane >> 3) & 2) + (lane >> 5)];
  red[0] = __uint_as_float(lo);
  red[4] = __uint_as_float(hi);
}

// After a barrier: the scale of column c of array a, for one thread of each.
template <int NA, int R>
__device__ __forceinline__ float tile_column_scale(TileLds<NA, R>& L, int a, int c) {
  float m = 0.f;
#pragma unroll
  for (int w = 0; w < TileLds<NA, R>::kWaves; ++w) m = fmaxf(m, L.red[w][a][c]);
  const float s = scale_from_amax(m);
  L.scale[a][c] = s;
  return s;
}

// After another: array a's codes, into LDS.
template <int NA, int R>
__device__ __forceinline__ void tile_codes(TileLds<NA, R>& L, int a, const float (&v)[R][8]) {
  const int g = threadIdx.x & 15, j = threadIdx.x >> 4;
  uint32_t* const column = &L.tile[a][8 * g * 32 + ((R / 4 * j) ^ (4 * (g & 7)))];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float s = L.scale[a][8 * g + c];
    u32x2 w;
    w.x = codes4(v[0][c] * s, v[1][c] * s, v[2][c] * s, v[3][c] * s);
    if constexpr (R == 8) {
      w.y = codes4(v[4][c] * s, v[5][c] * s, v[6][c] * s, v[7][c] * s);
      *(u32x2*)(column + 32 * c) = w;
    } else {
      column[32 * c] = w.x;
    }
  }
}

// After the last: array a's tile of `rows` x `cols` existing values, to the
// transposed matrix whose rows 0 .. cols - 1 start at `corner` (rows % 16 == 0).
// Nothing reads these codes before the backward or its weight gradient: they pass
// the caches by.
template <int NA, int R>
__device__ __forceinline__ void store_transposed(const TileLds<NA, R>& L, int a, uint8_t* corner, int64_t ld, int rows,
                                                 int cols) {
  constexpr int kColumns = 256 / R;   // a pass
  const int oc = threadIdx.x >> 3, seg = threadIdx.x & 7;
  uint32_t at = oc * (uint32_t)ld + 16 * seg;
#pragma unroll
  for (int i = 0; i < 128 / kColumns; ++i, at += kColumns * (uint32_t)ld) {
    const int c = oc + kColumns * i;
    const u32x4 w = *(const u32x4*)&L.tile[a][c * 32 + ((4 * seg) ^ (4 * ((c >> 3) & 7)))];
    if (c < cols && 16 * seg < rows) __builtin_nontemporal_store(w, (u32x4*)(corner + at));
  }
}

}  // namespace fp8bw
