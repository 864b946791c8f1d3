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
// The code comes from a product with 1 / s (off by at most 2^-22 relative, so by 4e-6 of a
// step); one that lies nearer than 1e-5 to a border between two codes is decided by the exact
// remainder, the rounding error of x - z included. A division per element instead made the
// append compute-bound.
__device__ __forceinline__ void int4_quantise(const uint4& h, uint32_t& codes, uint32_t& params) {
  const __half2* p = reinterpret_cast<const __half2*>(&h);
  __half2 lo2 = __hmin2_nan(__hmin2_nan(p[0], p[1]), __hmin2_nan(p[2], p[3]));
  __half2 hi2 = __hmax2_nan(__hmax2_nan(p[0], p[1]), __hmax2_nan(p[2], p[3]));
  // (min, -max) in one register: one shuffle and one packed minimum per step
  __half2 mm = __halves2half2(__hmin_nan(__low2half(lo2), __high2half(lo2)),
                              __hneg(__hmax_nan(__low2half(hi2), __high2half(hi2))));
  mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, 1));
  mm = __hmin2_nan(mm, __shfl_xor_sync(0xffffffffu, mm, 2));
  const float lo = __low2float(mm), hi = -__high2float(mm);
  const float range = hi - lo;
  if (!(range <= 131008.f)) {   // a NaN or an infinity
    codes = 0u;
    params = 0x7fff7fffu;
    return;
  }
  const __half up = __float2half_ru(__fdiv_rn(range, 15.f));
  const __half top = __float2half_rz(__fdiv_rn(65504.f - lo, 15.f));
  const __half s = __hmin(up, top);
  const __half2 sz = __halves2half2(s, __low2half(mm));
  params = *reinterpret_cast<const uint32_t*>(&sz);
  const float sf = __half2float(s);
  const float r = sf > 0.f ? __fdiv_rn(1.f, sf) : 0.f;   // at most 2^24: s is a multiple of 2^-24
  codes = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(p[i]);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float d = (e ? f.y : f.x) - lo;
      const float q = d * r;
      float k = rintf(q);
      if (fabsf(q - k) > 0.5f - 1e-5f) {
        k = floorf(q);
        const float a = e ? f.y : f.x, bb = d - a;              // a - lo = d + off
        const float off = (a - (d - bb)) + (-lo - bb);
        const float rem = fmaf(-(k + 0.5f), sf, d) + off;       // over the border if > 0
        if (rem > 0.f || (rem == 0.f && (static_cast<int>(k) & 1))) k += 1.f;
      }
      codes |= static_cast<uint32_t>(min(static_cast<int>(k), 15)) << (4 * (2 * i + e));
    }
  }
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
