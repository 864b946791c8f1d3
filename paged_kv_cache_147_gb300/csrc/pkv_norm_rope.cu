// pkv_norm_rope.cu -- RMS norm of each query and key head with its own weight, and the
// rotate-half position rotation, in one pass: what comes between the projections and the cache.
//
//   r = 1 / sqrt(mean_d x_d^2 + eps),  y_d = x_d r w_d,
//   out_d = y_d cos_d - y_{d+64} sin_d,  out_{d+64} = y_{d+64} cos_d + y_d sin_d   (d < 64)
//
// all in fp32, one rounding to fp16 at the end. Every element is read once and written once, so
// memory bounds it (256 bytes in and out per head): 16 lanes take a head, lane l the dims
// 4 l .. 4 l + 3 and 64 + 4 l .. 64 + 4 l + 3, so that both halves of a rotated pair are in one
// lane (8-byte accesses, 128 contiguous bytes per half-warp) and the only exchange is the sum of
// squares. A half-warp takes HPT heads of one token: their loads are all in flight before the
// first sum, and the token's cos / sin row is loaded once for them. Prompts take four heads and
// streaming accesses (8192 tokens x 72 heads: 52.8 us, 5.8 TB/s; with cached accesses 56.0, with
// two or eight heads 61.8 each; 16-byte accesses by 8 lanes a head 52.1 to 54.0, no difference),
// decode steps one head, for the shorter chain (64 x 14 heads: 2.2 us against 3.3).
#include <cuda_fp16.h>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kHead = 128;

struct NormRopeArgs {
  const __half* q;
  const __half* k;
  __half* q_out;
  __half* k_out;
  int64_t q_stride, k_stride;   // elements from one token's heads to the next one's
  const __half* q_weight;
  const __half* k_weight;
  const int64_t* positions;
  const float4* cos_sin;        // [n_index][32] float4: two (cos, sin) pairs
  float eps;
  int n_index, num_tokens, hq, heads, groups;   // heads = hq + hkv, groups = ceil(heads / HPT)
  unsigned int* err;
};

__device__ __forceinline__ void unpack4(uint2 u, float (&f)[4]) {
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&u.x));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&u.y));
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

template <bool STREAM>
__device__ __forceinline__ uint2 load(const __half* p) {
  const uint2* q = reinterpret_cast<const uint2*>(p);
  return STREAM ? __ldcs(q) : *q;
}
template <bool STREAM>
__device__ __forceinline__ void store(__half* p, uint2 v) {
  uint2* q = reinterpret_cast<uint2*>(p);
  if (STREAM) __stcs(q, v);
  else *q = v;
}

template <int HPT, bool STREAM>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const NormRopeArgs a) {
  griddep_wait();
  const int l = threadIdx.x & 15;
  const int64_t unit = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> 4;
  const int64_t t = unit / a.groups;
  const int h0 = static_cast<int>(unit - t * a.groups) * HPT;
  const bool in = t < a.num_tokens;
  const int64_t pos = in ? a.positions[t] : -1;
  if (pos >= a.n_index && l == 0 && h0 == 0) atomicOr(a.err, PKV_DEVERR_POSITION);
  const bool live = pos >= 0 && pos < a.n_index;
  uint2 lo[HPT], hi[HPT];
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = h0 + i;
    lo[i] = hi[i] = make_uint2(0, 0);
    if (live && h < a.heads) {
      const __half* x = h < a.hq ? a.q + t * a.q_stride + h * kHead
                                 : a.k + t * a.k_stride + (h - a.hq) * kHead;
      lo[i] = load<STREAM>(x + 4 * l);
      hi[i] = load<STREAM>(x + 64 + 4 * l);
    }
  }
  float4 cs[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  if (live) {
    cs[0] = a.cos_sin[pos * 32 + 2 * l];
    cs[1] = a.cos_sin[pos * 32 + 2 * l + 1];
  }
  const float c[4] = {cs[0].x, cs[0].z, cs[1].x, cs[1].z};
  const float s[4] = {cs[0].y, cs[0].w, cs[1].y, cs[1].w};
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = h0 + i;
    float x[4], y[4];
    unpack4(lo[i], x);
    unpack4(hi[i], y);
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) sum = fmaf(x[e], x[e], fmaf(y[e], y[e], sum));
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!live || h >= a.heads) continue;
    const float r = rsqrtf(fmaf(sum, 1.f / kHead, a.eps));
    const __half* w = h < a.hq ? a.q_weight : a.k_weight;
    float wx[4], wy[4];
    unpack4(*reinterpret_cast<const uint2*>(w + 4 * l), wx);
    unpack4(*reinterpret_cast<const uint2*>(w + 64 + 4 * l), wy);
    float ox[4], oy[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float u = x[e] * r * wx[e], v = y[e] * r * wy[e];
      ox[e] = u * c[e] - v * s[e];
      oy[e] = v * c[e] + u * s[e];
    }
    __half* out = h < a.hq
                      ? a.q_out + (t * a.hq + h) * kHead
                      : a.k_out + (t * (a.heads - a.hq) + (h - a.hq)) * kHead;
    store<STREAM>(out + 4 * l, make_uint2(pack_half2(ox[0], ox[1]), pack_half2(ox[2], ox[3])));
    store<STREAM>(out + 64 + 4 * l,
                  make_uint2(pack_half2(oy[0], oy[1]), pack_half2(oy[2], oy[3])));
  }
}

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int launch_status() { return cuda_status(cudaGetLastError()); }

template <int HPT, bool STREAM>
int launch(NormRopeArgs& a, cudaStream_t stream) {
  a.groups = (a.heads + HPT - 1) / HPT;
  const int64_t blocks = (static_cast<int64_t>(a.num_tokens) * a.groups * 16 + kThreads - 1) /
                         kThreads;
  if (blocks > 0x7fffffff) return PKV_EINVAL;
  return launch_waiting(&norm_rope_kernel<HPT, STREAM>, static_cast<unsigned>(blocks), kThreads,
                        0, stream, a);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_qk_norm_rope(void* q_out, void* k_out, const void* q, const void* k, int64_t q_stride,
                     int64_t k_stride, const void* q_weight, const void* k_weight, float eps,
                     const int64_t* positions, const float* cos_sin, int n_index, int num_tokens,
                     int num_q_heads, int num_kv_heads, int head_dim, pkv_stream_t stream) {
  if (num_tokens < 0 || num_q_heads < 1 || num_kv_heads < 1 || head_dim != kHead || n_index < 1 ||
      !(eps >= 0.f) || num_q_heads > (1 << 20) || num_kv_heads > (1 << 20) ||
      q_stride < static_cast<int64_t>(num_q_heads) * kHead ||
      k_stride < static_cast<int64_t>(num_kv_heads) * kHead || q_stride % 4 != 0 ||
      k_stride % 4 != 0)
    return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !k_out || !q || !k || !q_weight || !k_weight || !positions || !cos_sin)
    return PKV_EINVAL;
  if (!aligned8(q) || !aligned8(k) || !aligned8(q_out) || !aligned8(k_out) ||
      !aligned8(q_weight) || !aligned8(k_weight) || !aligned16(cos_sin))
    return PKV_EINVAL;
  NormRopeArgs a;
  a.err = device_error_ptr();
  if (!a.err) return launch_status();
  a.q = static_cast<const __half*>(q);
  a.k = static_cast<const __half*>(k);
  a.q_out = static_cast<__half*>(q_out);
  a.k_out = static_cast<__half*>(k_out);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.q_weight = static_cast<const __half*>(q_weight);
  a.k_weight = static_cast<const __half*>(k_weight);
  a.positions = positions;
  a.cos_sin = reinterpret_cast<const float4*>(cos_sin);
  a.eps = eps;
  a.n_index = n_index;
  a.num_tokens = num_tokens;
  a.hq = num_q_heads;
  a.heads = num_q_heads + num_kv_heads;
  // one head or four a half-warp, us: 896 heads 2.0 / 2.9, 9216 2.5 / 2.9, 16416 3.4 / 3.5, 18432
  // 3.6 / 3.5, 36864 5.4 / 4.6, 147456 16.7 / 14.1
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (static_cast<int64_t>(num_tokens) * a.heads <= 16384) return launch<1, false>(a, st);
  return launch<4, true>(a, st);
}

}  // extern "C"
