// AdamW over many tensors in one call, with fp32 or 8-bit block-scaled
// states, for gfx950.
//
//   g = grad * grad_scale
//   m = b1 m + (1 - b1) g          v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// 8-bit states: blocks of 128 elements of the flattened tensor share a
// power-of-two scale, m is held as E4M3 codes of m / scale and v as E4M3
// codes of its root, sqrt(v) / scale: the root halves the exponent range, so
// one byte covers v over ten decades with the precision that sqrt(v) needs.
// A power-of-two scale makes dividing by it exact and leaves codes alone
// while the scale stays.  A positive root never becomes code 0: an element
// whose v vanished next to a large neighbour would be stepped by m / eps.
//
// A moment that is infinite or NaN becomes the NaN code, and the block's scale
// goes by the others: one bad gradient costs its own element, as with fp32
// states.
//
// With a seed, what is held in fewer bits (codes, and bf16 parameters that
// have no fp32 master) is rounded up or down by 16 random bits per value, in
// proportion to the remainder.  Round-to-nearest would freeze slow averages:
// v moves by a share (1 - b2) a step, far below half a code.
//
// Products and sums round separately (no fused multiply-add): the states are
// then the formula's fp32 operations one by one, and which power of two a
// block's scale takes does not hang on how an expression was compiled.
//
// Every element is read and written once; the kernel is bound by HBM: 336M bf16
// parameters with 8-bit states 680 to 690 us (5.0 TB/s; 885 us with IEEE square
// root and division and the rounding in integer arithmetic), with fp32 states and
// masters 1810 us (5.2 TB/s).

#include "device_common.h"
#include "launch.h"

namespace fp8bw {

// A mixing function of 32 bits: xor-shifts between odd multipliers taken from
// the fractional parts of sqrt(2) and sqrt(3).
__host__ __device__ __forceinline__ uint32_t mix32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xBB67AE85u;
  return x ^ (x >> 16);
}

uint32_t adamw_key(uint64_t seed, int ordinal) {
  return mix32((uint32_t)seed + 0x9E3779B9u * (uint32_t)(ordinal + 1)) + (uint32_t)(seed >> 32);
}

// Vectors at the alignment of their elements: tensors of a packed buffer may
// start anywhere, and gfx950's global loads and stores take any alignment.
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

// Elements i .. i + 7 of a tensor as fp32; `n` of them exist.
__device__ __forceinline__ void load8_f32(const float* p, int n, float (&f)[8]) {
  if (n >= 8) {
    const f32x4_any a = *(const f32x4_any*)p, b = *(const f32x4_any*)(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? p[j] : 0.f;
  }
}
__device__ __forceinline__ void store8_f32(float* p, int n, const float (&f)[8]) {
  if (n >= 8) {
    *(f32x4_any*)p = f32x4_any{f[0], f[1], f[2], f[3]};
    *(f32x4_any*)(p + 4) = f32x4_any{f[4], f[5], f[6], f[7]};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = f[j];
  }
}
__device__ __forceinline__ void load8_bf16(const uint16_t* p, int n, float (&f)[8]) {
  if (n >= 8) {
    const u32x4_any u = *(const u32x4_any*)p;
    f[0] = bf16lo(u.x); f[1] = bf16hi(u.x); f[2] = bf16lo(u.y); f[3] = bf16hi(u.y);
    f[4] = bf16lo(u.z); f[5] = bf16hi(u.z); f[6] = bf16lo(u.w); f[7] = bf16hi(u.w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < n ? bf16lo(p[j]) : 0.f;
  }
}
// bf16 bits in the low halves of b.
__device__ __forceinline__ void store8_u16(uint16_t* p, int n, const uint32_t (&b)[8]) {
  if (n >= 8) {
    *(u32x4_any*)p = u32x4_any{b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint16_t)b[j];
  }
}
__device__ __forceinline__ uint2 load8_codes(const uint8_t* p, int n) {
  if (n >= 8) {
    const u32x2_any u = *(const u32x2_any*)p;
    return make_uint2(u.x, u.y);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void store8_codes(uint8_t* p, int n, uint2 w) {
  if (n >= 8) {
    *(u32x2_any*)p = u32x2_any{w.x, w.y};
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = (uint8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
  }
}
__device__ __forceinline__ void decode8(uint2 w, float scale, float (&f)[8]) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8(w.x, 0) * scale;
  f[1] = __builtin_amdgcn_cvt_f32_fp8(w.x, 1) * scale;
  f[2] = __builtin_amdgcn_cvt_f32_fp8(w.x, 2) * scale;
  f[3] = __builtin_amdgcn_cvt_f32_fp8(w.x, 3) * scale;
  f[4] = __builtin_amdgcn_cvt_f32_fp8(w.y, 0) * scale;
  f[5] = __builtin_amdgcn_cvt_f32_fp8(w.y, 1) * scale;
  f[6] = __builtin_amdgcn_cvt_f32_fp8(w.y, 2) * scale;
  f[7] = __builtin_amdgcn_cvt_f32_fp8(w.y, 3) * scale;
}

// Exponent e of a block's scale 2^e: the least with amax <= 448 2^e (448 =
// 0.875 2^9), within fp32's normal range.  0 for an all-zero block.
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.f) return 0;
  const float fraction = __builtin_amdgcn_frexp_mantf(amax);
  const int e = __builtin_amdgcn_frexp_expf(amax) - 9 + (fraction > 0.875f ? 1 : 0);
  return max(-126, min(127, e));
}

// 8 values times 2^-exponent as E4M3 codes, magnitudes at most 448.  RANDOM:
// v_cvt_sr_fp8_f32 adds its random number, aligned to the bits that the code
// drops, and cuts: up with the probability of the remainder in units of
// 2^-16, subnormal codes included (a test compares a million values of 22
// octaves with that definition).  `shift` picks the 16 random bits.
// KEEP: what is positive gets at least the smallest code; no NaN among f.
// Infinite values (and NaN without KEEP) convert to the NaN code.
template <bool RANDOM, bool KEEP>
__device__ __forceinline__ uint2 encode8(const float (&f)[8], int exponent, const uint32_t (&rnd)[8], int shift) {
  const float inv = __builtin_amdgcn_ldexpf(1.f, -exponent);
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    y[j] = f[j] * inv;
    if constexpr (KEEP) y[j] = f[j] > 0.f ? fmaxf(y[j], 0x1p-9f) : 0.f;
  }
  if constexpr (!RANDOM) {
    // no clamp: the scale holds magnitudes within 448, and NaN stays NaN
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4], y[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6], y[7], hi, true);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
  } else {
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = shift ? rnd[j] & 0xFFFF0000u : rnd[j] << 16;
    int lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[0], r[0], 0, 0);
    lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[1], r[1], lo, 1);
    lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[2], r[2], lo, 2);
    lo = __builtin_amdgcn_cvt_sr_fp8_f32(y[3], r[3], lo, 3);
    int hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[4], r[4], 0, 0);
    hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[5], r[5], hi, 1);
    hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[6], r[6], hi, 2);
    hi = __builtin_amdgcn_cvt_sr_fp8_f32(y[7], r[7], hi, 3);
    return make_uint2((uint32_t)lo, (uint32_t)hi);
  }
}

// One workgroup takes `iters` runs of 2048 elements of one tensor; a thread's
// 8 consecutive elements lie in one 128-block, which a 16-lane DPP row holds.
template <bool EIGHT, bool RANDOM>
__global__ __launch_bounds__(256) void adamw_kernel(const AdamwLaunch L) {
#pragma clang fp contract(off)
  // The tensor of this workgroup: the last one whose first workgroup is not past it.
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.first[mid] <= (int)blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const AdamwTensor& T = L.t[lo];
  const float gs = L.grad_scale ? *L.grad_scale : 1.f;
  const int64_t base = (int64_t)((int)blockIdx.x - L.first[lo]) * L.iters * 2048;
  for (int it = 0; it < L.iters; ++it) {
    const int64_t i = base + it * 2048 + threadIdx.x * 8;
    // whole 128-blocks leave together, so the DPP reductions below are full
    if ((i & ~(int64_t)127) >= T.numel) return;
    const int64_t left = T.numel - i;
    const int n = left >= 8 ? 8 : left > 0 ? (int)left : 0;
    const int64_t at = n > 0 ? i : 0;
    float g[8], p[8], m[8], v[8], root[8];
    if (T.flags & kAdamwGradF32) load8_f32((const float*)T.grad + at, n, g);
    else load8_bf16((const uint16_t*)T.grad + at, n, g);
    if (T.master) load8_f32(T.master + at, n, p);
    else if (T.flags & kAdamwParamF32) load8_f32((const float*)T.param + at, n, p);
    else load8_bf16((const uint16_t*)T.param + at, n, p);
    const int64_t blk = i >> 7;
    if constexpr (EIGHT) {
      decode8(load8_codes((const uint8_t*)T.m + at, n), T.m_scale[blk], m);
      decode8(load8_codes((const uint8_t*)T.v + at, n), T.root_scale[blk], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] *= v[j];
    } else {
      load8_f32((const float*)T.m + at, n, m);
      load8_f32((const float*)T.v + at, n, v);
    }
    float am = 0.f, av = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = g[j] * gs;
      m[j] = m[j] * L.beta1 + gj * L.one_minus_beta1;
      v[j] = v[j] * L.beta2 + gj * gj * L.one_minus_beta2;
      if (EIGHT && j < n) {
        am = fmaxf(am, fabsf(m[j]));
        av = fmaxf(av, v[j]);
      }
    }
    bool rare = false;
    if constexpr (EIGHT) {
      // Hardware square root and reciprocal, each within 1 ulp (9.2e-8 and
      // 9.0e-8 measured): codes keep 4 bits and the step is far smaller than
      // p, while the IEEE forms bind this kernel by its arithmetic (336M
      // elements: 10% more time).  They do not take subnormals, which
      // get the IEEE root.  The same test finds the moments that are not finite
      // (an infinite or NaN gradient shows in v), which the scales leave out.
      rare = !(am < INFINITY);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        root[j] = __builtin_amdgcn_sqrtf(v[j]);
        rare |= __builtin_amdgcn_classf(v[j], 1 << 0 | 1 << 1 | 1 << 7 | 1 << 9);   // NaN, subnormal, infinite
      }
      rare = __builtin_amdgcn_ballot_w64(rare) != 0;
      if (rare) {
        am = av = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (v[j] < 0x1p-126f) root[j] = __builtin_sqrtf(v[j]);
          if (j < n && fabsf(m[j]) < INFINITY) am = fmaxf(am, fabsf(m[j]));
          if (j < n && v[j] < INFINITY) av = fmaxf(av, v[j]);
        }
      }
      am = row16_max(am);
      av = row16_max(av);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p[j] = p[j] * L.decay - m[j] * __builtin_amdgcn_rcpf(root[j] * L.root_factor + L.eps) * L.step_size;
      if (rare) {
#pragma unroll
        for (int j = 0; j < 8; ++j) root[j] = root[j] >= 0.f ? root[j] : INFINITY;   // encode8 takes no NaN here
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        p[j] = p[j] * L.decay - m[j] / (__builtin_sqrtf(v[j]) * L.root_factor + L.eps) * L.step_size;
    }
    // the first 2^32 elements' hash is of key + element alone
    const uint32_t far = RANDOM ? mix32((uint32_t)(i >> 32)) : 0u;
    uint32_t rnd[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rnd[j] = RANDOM ? mix32((T.key + (uint32_t)i + j) ^ far) : 0u;
    if constexpr (!EIGHT) {
      store8_f32((float*)T.m + at, n, m);
      store8_f32((float*)T.v + at, n, v);
    }
    // The parameter leaves before 8-bit states are encoded: 72 registers, 7
    // waves a SIMD, instead of 81 and 5 (336M elements: 679 us, 736 us).
    if (T.master) store8_f32(T.master + at, n, p);
    if (T.flags & kAdamwParamF32) {
      store8_f32((float*)T.param + at, n, p);
    } else {
      uint32_t b[8];
      if (RANDOM && !T.master) {
        // add 16 random bits below the cut, then cut: up with the probability of the remainder
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t up = (__float_as_uint(p[j]) + ((rnd[j] * 0x9E3779B9u) >> 16)) >> 16;
          b[j] = p[j] == p[j] ? up : 0x7FC0u;   // a NaN's mantissa may carry into its sign
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = f32_to_bf16_rne(p[j]);
      }
      store8_u16((uint16_t*)T.param + at, n, b);
    }
    if constexpr (EIGHT) {
      // The root's scale comes from the correctly rounded root of the largest v.
      const int em = scale_exponent(am), er = scale_exponent(__builtin_sqrtf(av));
      store8_codes((uint8_t*)T.m + at, n, encode8<RANDOM, false>(m, em, rnd, 0));
      store8_codes((uint8_t*)T.v + at, n, encode8<RANDOM, true>(root, er, rnd, 16));
      if ((threadIdx.x & 15) == 0) {
        T.m_scale[blk] = __builtin_amdgcn_ldexpf(1.f, em);
        T.root_scale[blk] = __builtin_amdgcn_ldexpf(1.f, er);
      }
    }
  }
}

hipError_t launch_adamw(const AdamwLaunch& L, int workgroups, bool eight, bool random, hipStream_t stream) {
  const dim3 grid((unsigned)workgroups), block(256);
  if (eight && random) hipLaunchKernelGGL((adamw_kernel<true, true>), grid, block, 0, stream, L);
  else if (eight) hipLaunchKernelGGL((adamw_kernel<true, false>), grid, block, 0, stream, L);
  else if (random) hipLaunchKernelGGL((adamw_kernel<false, true>), grid, block, 0, stream, L);
  else hipLaunchKernelGGL((adamw_kernel<false, false>), grid, block, 0, stream, L);
  return hipGetLastError();
}

}  // namespace fp8bw
