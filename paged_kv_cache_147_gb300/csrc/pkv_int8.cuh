// pkv_int8.cuh -- the 8-bit cache's format and its quantisation.
//
// A block of tokens of one kv head shares one scale for its keys and one for its values; a row (one
// token, one kv head, K or V) is 128 bytes of codes, an element's value is scale * (code - 128).
// Scales are powers of two, 2^-30 to 2^9:
//  * a block's scale has to grow when a larger row arrives. A code then moves to the new grid by
//    rint(c 2^-k); the errors of repeated moves are halves of ever larger steps, together less than
//    one step of the last scale, where arbitrary scales, growing a little with every token, would
//    add half a step each time. A scale has at most one bit more than the rows need.
//  * codes times scale are exact wherever they go (fp16, fp32), and so are sums of codes times whole
//    numbers: the block selection gives the same answer in any order of summation.
// Codes lie in 1 .. 255 (128 is zero): as unsigned bytes one byte permutation makes fp16 numbers of
// them. A scale that is NaN says that a NaN or an infinity was written; all of the block is NaN then.
#pragma once

#include <cuda_fp16.h>

#include "pkv_device.cuh"

namespace pkv {

constexpr int kInt8Low = -30, kInt8High = 9;   // exponents of a scale
constexpr uint32_t kInt8Zeros = 0x80808080u;   // four codes of zero
constexpr uint32_t kNanBits = 0x7fffffffu;

// The least scale s with top <= 127 s (2^9 at most); NaN for a top that is NaN or infinite.
__device__ __forceinline__ float int8_scale(float top) {
  if (!(top <= 65504.f)) return __uint_as_float(kNanBits);
  // 127 is 1.984375 * 2^6: adding 2^17 - 1 to the bits carries into the exponent past that
  const int e = static_cast<int>((__float_as_uint(top) + 0x1ffffu) >> 23) - 6;
  return __uint_as_float(static_cast<uint32_t>(min(max(e, 127 + kInt8Low), 127 + kInt8High)) << 23);
}

// 1 / s of a power of two (0 for NaN).
__device__ __forceinline__ float int8_inverse(float s) {
  return s == s ? __uint_as_float((254u << 23) - __float_as_uint(s)) : 0.f;
}

// What `top` needs, and what the block has: the larger, NaN if either is.
__device__ __forceinline__ float int8_grown(float need, float old) {
  return old != old ? old : (need != need ? need : fmaxf(need, old));
}

// Quantises elements at one scale (a power of two, or NaN: all codes are zeros). x / s is a product
// with 1 / s, and adding 1664 = 1.5 * 2^10 + 128 in the same packed operation rounds it to a whole
// number, ties to even, and leaves the code in the sum's low byte: one rounding in all, as in 32 bits.
struct Int8Quantiser {
  __half2 up, r;   // 1 / s in two factors: 1 / s alone may be past fp16
  int kind;        // 0: one factor; 1: two; 2: the greatest scale; 3: NaN

  __device__ __forceinline__ explicit Int8Quantiser(float s) {
    const int e = static_cast<int>(__float_as_uint(s) >> 23) - 127;
    kind = s != s ? 3 : e == kInt8High ? 2 : e < -15 ? 1 : 0;
    up = __float2half2_rn(32768.f);
    r = __float2half2_rn(s != s ? 0.f
                                : __uint_as_float(static_cast<uint32_t>(127 - e - (e < -15 ? 15 : 0)) << 23));
  }
  // (PLAIN: for kind 0 only)
  template <bool PLAIN = false>
  __device__ __forceinline__ uint2 codes(uint4 h) const {
    if (!PLAIN && kind == 3) return make_uint2(kInt8Zeros, kInt8Zeros);
    const __half2 magic = __half2half2(__ushort_as_half(0x6680));
    __half2* p = reinterpret_cast<__half2*>(&h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!PLAIN && kind == 1) p[i] = __hmul2(p[i], up);   // (exact: below 2^-8 before)
      p[i] = __hfma2(p[i], r, magic);
      // only at the greatest scale can an element pass 127.5 steps
      if (!PLAIN && kind == 2)
        p[i] = __hmax2(__hmin2(p[i], __half2half2(__ushort_as_half(0x66ff))),
                       __half2half2(__ushort_as_half(0x6601)));
    }
    return make_uint2(__byte_perm(h.x, h.y, 0x6420), __byte_perm(h.z, h.w, 0x6420));
  }
};

// Code i of a word as a float, without the offset.
template <int I>
__device__ __forceinline__ float int8_value(uint32_t w) {
  return __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 | I)) - (8388608.f + 128.f);
}

// Codes on a grid 1 / f times as coarse (f <= 1, a power of two or 0). 1024 + u is an fp16 number with
// u as its lowest bits, and (1024 + u) f + (1664 - 1152 f) = 1664 + (u - 128) f, rounded once, leaves
// the new code in its low byte; the constant is a whole number down to f = 2^-7, below which nothing
// is left of a code.
struct Int8Mover {
  __half2 f, c;
  bool none;

  __device__ __forceinline__ explicit Int8Mover(float factor) : none(!(factor >= 0x1p-7f)) {
    f = __float2half2_rn(none ? 0.f : factor);
    c = __float2half2_rn(1664.f - (none ? 0.f : 1152.f * factor));
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
    if (none) return kInt8Zeros;
    uint32_t lo = __byte_perm(w, 0x64646464u, 0x4140), hi = __byte_perm(w, 0x64646464u, 0x4342);
    const __half2 l2 = __hfma2(*reinterpret_cast<const __half2*>(&lo), f, c);
    const __half2 h2 = __hfma2(*reinterpret_cast<const __half2*>(&hi), f, c);
    lo = *reinterpret_cast<const uint32_t*>(&l2);
    hi = *reinterpret_cast<const uint32_t*>(&h2);
    return __byte_perm(lo, hi, 0x6420);
  }
  __device__ __forceinline__ uint4 operator()(const uint4& w) const {
    return make_uint4((*this)(w.x), (*this)(w.y), (*this)(w.z), (*this)(w.w));
  }
};

}  // namespace pkv
