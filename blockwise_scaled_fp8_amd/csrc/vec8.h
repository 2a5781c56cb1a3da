// What the streaming kernels share: eight bf16 values in a 16-byte vector,
// sums over a wavefront, and codes of 128 x 128 tiles of fp32 values in both
// layouts.
#pragma once

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
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));
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

// Eight E4M3 codes of f * s.
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float s) {
  return make_uint2(cvt4_e4m3(f[0] * s, f[1] * s, f[2] * s, f[3] * s),
                    cvt4_e4m3(f[4] * s, f[5] * s, f[6] * s, f[7] * s));
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

// ---------------------------------------------------------------------------
// Transposed codes of NA 128 x 128 tiles of fp32 values held by a workgroup of
// 512 threads: thread (g = tid % 16, j = tid / 16) holds columns 8 g .. 8 g + 7
// of rows 4 j .. 4 j + 3, so a wave's loads cover 256-byte pieces of 16 rows
// and a 16-lane DPP row holds one 1x128 block of a row.
//
// One scale per column: each column's 4 rows in registers, the 4 row quads of
// a wave by two shuffles, the 8 waves through LDS.  A thread then quantizes
// its 4 rows of a column into one dword of an LDS tile stored [column][row]
// (32 dwords a column); dword d of column c lies at d ^ 4 ((c / 8) % 8), which
// spreads a store's 16 column groups over the banks and keeps 16-byte groups
// whole, and the tile leaves as 16-byte pieces of output rows, 8 lanes a row.
template <int NA>
struct TileLds {
  float red[8][NA][128];
  float scale[NA][128];
  __attribute__((aligned(16))) uint32_t tile[NA][128 * 32];
};

// The column maxima of array a, into LDS.  Before the first barrier.
template <int NA>
__device__ __forceinline__ void tile_column_max(TileLds<NA>& L, int a, const float (&v)[4][8]) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, g = tid & 15;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    float m = fmaxf(fmaxf(fabsf(v[0][c]), fabsf(v[1][c])), fmaxf(fabsf(v[2][c]), fabsf(v[3][c])));
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    if (lane < 16) L.red[wave][a][8 * g + c] = m;
  }
}

// After a barrier: the scale of column c of array a, for one thread of each.
template <int NA>
__device__ __forceinline__ float tile_column_scale(TileLds<NA>& L, int a, int c) {
  float m = 0.f;
#pragma unroll
  for (int w = 0; w < 8; ++w) m = fmaxf(m, L.red[w][a][c]);
  const float s = scale_from_amax(m);
  L.scale[a][c] = s;
  return s;
}

// After another: array a's codes, into LDS.
template <int NA>
__device__ __forceinline__ void tile_codes(TileLds<NA>& L, int a, const float (&v)[4][8]) {
  const int g = threadIdx.x & 15, j = threadIdx.x >> 4;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const float s = L.scale[a][8 * g + c];
    L.tile[a][(8 * g + c) * 32 + (j ^ (4 * (g & 7)))] =
        cvt4_e4m3(v[0][c] * s, v[1][c] * s, v[2][c] * s, v[3][c] * s);
  }
}

// After the last: 16 codes of output row (tile column) oc, rows 16 seg .. + 15.
template <int NA>
__device__ __forceinline__ uint4 tile_piece(const TileLds<NA>& L, int a, int oc, int seg) {
  return *(const uint4*)&L.tile[a][oc * 32 + ((4 * seg) ^ (4 * ((oc >> 3) & 7)))];
}

}  // namespace fp8bw
