// pkv_int4.cuh -- the 4-bit row format and its quantisation, shared by the append and the fused
// append + decode.
//
// A row (one token, one kv head, K or V) of 128 elements is 80 bytes: 64 bytes of codes (element
// 2 j in the low half of byte j, 2 j + 1 in the high half), then for each 32 elements the fp16
// scale s and the fp16 minimum z. An element's value is s * code + z. 32 elements share a scale
// so that one outlier channel costs the resolution of its own group only; with s and z inside
// the row a 16-token chunk stays one contiguous run (1280 bytes), and a row stride of 20 words
// spreads 8 rows over all 32 shared-memory banks without a swizzle.
#pragma once

#include <cuda_fp16.h>

#include "pkv_device.cuh"

namespace pkv {

constexpr int kInt4Row = 80;        // bytes of a row
constexpr int kInt4Params = 64;     // offset of the (s, z) pairs

// Four lanes (l, l ^ 1, l ^ 2, l ^ 3) hold 8 consecutive elements each of one 32-element group:
// codes of this lane's 8 elements (first in the lowest 4 bits) and the group's (s, z) pair. All
// lanes of the warp take part.
//   z = min, s = (max - min) / 15 (in binary32) rounded up to fp16, so that code 15 reaches the
//   maximum, or rounded down where 15 s + z would pass the largest fp16; code = (x - z) / s
//   rounded to nearest, ties to even (0 where s is 0).
// A group with a NaN or an infinity gets s = z = NaN: all of it reads back as NaN.
// range / 15 is a product with RN(1 / 15) corrected by its exact remainder, which gives the
// correctly rounded quotient (Markstein's theorem on division by a correctly rounded
// reciprocal). The codes come from a product with an approximate 1 / s, rounded to an integer by
// adding 1.5 2^23 in the same operation (conversions run at a sixteenth of its rate and made the
// append compute-bound); products nearer than 1e-5 to a border between two codes send the lane
// through int4_exact_code. That is twice what they can be off: the reciprocal by 2 units in the last
// place (2^-22 of it), x - z by half of one, so a quotient at the last border, 14.5, by
// 14.5 (2^-22 + 2^-24) + 2^-25 = 4.4e-6.
constexpr float kInt4Magic = 12582912.f;   // 1.5 * 2^23, bits 0x4b400000

// The code of x in a group with minimum lo and scale s > 0, q its approximate (x - lo) / s: the
// exact remainder decides, the rounding error of x - lo included.
__device__ __forceinline__ uint32_t int4_exact_code(float x, float lo, float s, float q) {
  const float k = fminf(floorf(q), 15.f);
  const float d = x - lo, bb = d - x;              // x - lo = d + off exactly
  const float off = (x - (d - bb)) + (-lo - bb);
  const float rem = fmaf(-(k + 0.5f), s, d) + off;  // past the border if > 0
  const uint32_t c = static_cast<uint32_t>(k);
  return min(c + (rem > 0.f || (rem == 0.f && (c & 1u)) ? 1u : 0u), 15u);
}

// Two fp32 numbers in a register pair: one instruction for both.
__device__ __forceinline__ uint64_t f32x2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 f32x2_parts(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f32x2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// (s, z) of a group from (min, -max) of its elements; false for a NaN or an infinity in there.
__device__ __forceinline__ bool int4_scale(__half2 mm, uint32_t& params, float& lo, float& sf) {
  lo = __low2float(mm);
  const float hi = -__high2float(mm);
  const float range = hi - lo;
  if (!(range <= 131008.f)) {
    params = 0x7fff7fffu;
    return false;
  }
  constexpr float kInv15 = 1.f / 15.f;
  const float q15 = range * kInv15;
  __half s = __float2half_ru(fmaf(fmaf(-15.f, q15, range), kInv15, q15));
  sf = __half2float(s);
  if (fmaf(15.f, sf, lo) > 65504.f) {
    s = __hmin(s, __float2half_rz(__fdiv_rn(65504.f - lo, 15.f)));
    sf = __half2float(s);
  }
  const __half2 sz = __halves2half2(s, __low2half(mm));
  params = *reinterpret_cast<const uint32_t*>(&sz);
  return true;
}

// The codes of 8 elements, r the approximate 1 / s (0 where s is 0).
__device__ __forceinline__ uint32_t int4_codes(const uint4& h, float lo, float sf, float r) {
  const __half2* p = reinterpret_cast<const __half2*>(&h);
  const uint64_t nlo2 = f32x2(-lo, -lo), r2 = f32x2(r, r), magic2 = f32x2(kInt4Magic, kInt4Magic),
                 minus2 = f32x2(-1.f, -1.f);
  float off = 0.f;
  uint32_t c = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(p[i]);
    const uint64_t d = f32x2_add(f32x2(f.x, f.y), nlo2);
    const uint64_t m = f32x2_fma(d, r2, magic2);
    const float2 e = f32x2_parts(f32x2_fma(d, r2, f32x2_fma(m, minus2, magic2)));
    const float2 mf = f32x2_parts(m);
    off = fmaxf(off, fmaxf(fabsf(e.x), fabsf(e.y)));
    c += (__float_as_uint(mf.x) << (8 * i)) + (__float_as_uint(mf.y) << (8 * i + 4));
  }
  // the magic number's own bits, shifted and summed
  constexpr uint32_t kBias = 0x4b400000u + (0x4b400000u << 4) + (0x4b400000u << 8);
  c -= kBias;
  if (off > 0.5f - 1e-5f) {
    c = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(p[i]);
      c |= int4_exact_code(f.x, lo, sf, (f.x - lo) * r) << (8 * i);
      c |= int4_exact_code(f.y, lo, sf, (f.y - lo) * r) << (8 * i + 4);
    }
  }
  return c;
}

// s is a multiple of 2^-24: its reciprocal does not overflow.
__device__ __forceinline__ float int4_reciprocal(float sf) {
  return sf > 0.f ? __fdividef(1.f, sf) : 0.f;
}

// (min, -max) of 8 elements: one shuffle and one packed minimum take a step for both.
__device__ __forceinline__ __half2 int4_extremes(const uint4& h) {
  const __half2* p = reinterpret_cast<const __half2*>(&h);
  const __half2 lo2 = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
  const __half2 hi2 = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
  return __halves2half2(__hmin_nan(__low2half(lo2), __high2half(lo2)),
                        __hneg(__hmax_nan(__low2half(hi2), __high2half(hi2))));
}

__device__ __forceinline__ void int4_quantise(const uint4& h, uint32_t& codes, uint32_t& params) {
  __half2 mm = int4_extremes(h);
  mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
  mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
  float lo, sf;
  codes = 0u;
  if (int4_scale(mm, params, lo, sf)) codes = int4_codes(h, lo, sf, int4_reciprocal(sf));
}

// A whole group (32 elements) in one thread: the same bytes.
__device__ __forceinline__ void int4_quantise_group(const uint4 (&h)[4], uint4& codes,
                                                    uint32_t& params) {
  const __half2* p = reinterpret_cast<const __half2*>(h);
  __half2 lo2 = p[0], hi2 = p[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) {
    lo2 = __hmin2_nan(lo2, p[i]);
    hi2 = __hmax2_nan(hi2, p[i]);
  }
  const __half2 mm = __halves2half2(__hmin_nan(__low2half(lo2), __high2half(lo2)),
                                    __hneg(__hmax_nan(__low2half(hi2), __high2half(hi2))));
  float lo, sf;
  codes = make_uint4(0u, 0u, 0u, 0u);
  if (!int4_scale(mm, params, lo, sf)) return;
  const float r = int4_reciprocal(sf);
  codes = make_uint4(int4_codes(h[0], lo, sf, r), int4_codes(h[1], lo, sf, r),
                     int4_codes(h[2], lo, sf, r), int4_codes(h[3], lo, sf, r));
}

// Codes in the low halves of a word's two 16-bit halves, as fp16 (exact): c_lo takes bits 0-3,
// c_hi bits 4-7. 0x6400 is 1024, whose last place is 1: OR-ing a code in gives 1024 + code (or
// 1024 + 16 code), and one packed operation takes the 1024 off again.
__device__ __forceinline__ __half2 int4_lo(uint32_t x) {
  const uint32_t u = (x & 0x000f000fu) | 0x64006400u;
  return __hsub2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(0x6400)));
}
__device__ __forceinline__ __half2 int4_hi(uint32_t x) {
  const uint32_t u = (x & 0x00f000f0u) | 0x64006400u;
  return __hfma2(*reinterpret_cast<const __half2*>(&u),
                 __half2half2(__ushort_as_half(0x2c00)),     // 1 / 16
                 __half2half2(__ushort_as_half(0xd400)));    // -64
}

__device__ __forceinline__ uint32_t half2_bits(__half2 v) {
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ __half2 as_half2(uint32_t u) {
  return *reinterpret_cast<const __half2*>(&u);
}

}  // namespace pkv
