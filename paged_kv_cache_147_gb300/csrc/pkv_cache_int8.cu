// pkv_cache_int8.cu -- the 8-bit cache's own edits: the append (quantise, scatter, and bring the
// touched blocks to their new scales), the widening of whole blocks to fp16, and the block copy.
//
// All move bytes. The append reads 256 and writes 128 per row; a block that rows are added to is
// read and written again only when its scale grows (its largest element doubles, so a few times
// in a block's life).
#include <algorithm>

#include "pkv_int8.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarpRows = 16;    // rows of a block that a warp holds in registers
constexpr int kSpan = 16;        // tokens whose blocks one team looks after in a large call

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }

// A team of W warps (W rows of 16 make a block) takes, for one kv head and K or V, every block whose
// first row of the call is among its `span` tokens; the block's other rows are among the bs - 1
// tokens behind that one. All rows stay in registers between the pass that finds the scale and the
// one that writes codes.
template <int W>
__global__ void __launch_bounds__(W < 4 ? kThreads : W * 32)
kv_append_int8_kernel(const uint4* k, const uint4* v, const int64_t* slots, int num_tokens,
                      uint8_t* k_cache, uint8_t* v_cache, float* scales, uint8_t* bounds,
                      int64_t num_slots, int num_kv_heads, int span, unsigned jobs,
                      unsigned int* err) {
  griddep_wait();
  constexpr int kTeams = W < 4 ? 4 / W : 1;
  constexpr int kBs = W * kWarpRows;
  constexpr int kShift = W == 1 ? 4 : W == 2 ? 5 : W == 4 ? 6 : W == 8 ? 7 : 8;
  __shared__ float top_s[kTeams][W];
  __shared__ uint32_t rows_s[kTeams][W];          // which rows of the block the call writes
  __shared__ uint4 ends_s[kTeams][W][32];         // per channel least and greatest new element
  const int lane = threadIdx.x & 31;
  const int team = threadIdx.x / (W * 32), w = (threadIdx.x >> 5) % W;
  const unsigned job = blockIdx.x * kTeams + team;
  if (job >= jobs) return;
  const unsigned which = job & 1;
  const unsigned part = (job >> 1) / num_kv_heads;
  const int h = static_cast<int>((job >> 1) - part * num_kv_heads);
  const int64_t first = static_cast<int64_t>(part) * span;
  auto team_sync = [&]() {
    if (W == 1) __syncwarp();
    else named_barrier_sync(1 + team, W * 32);
  };
  // the block of a token, -1 for none
  auto block_of = [&](int64_t t) -> int64_t {
    if (t < 0 || t >= num_tokens) return -1;
    const int64_t s = slots[t];
    return s >= 0 && s < num_slots ? s >> kShift : -1;
  };
  if (which == 0 && h == 0 && w == 0 && lane < span && first + lane < num_tokens &&
      slots[first + lane] >= num_slots)
    atomicOr(err, PKV_DEVERR_SLOT);

  const int64_t mine = lane < span ? block_of(first + lane) : -1;
  const int64_t before = lane < span ? block_of(first + lane - 1) : -1;
  unsigned heads = __ballot_sync(0xffffffffu, mine >= 0 && mine != before);
  const uint4* src = which ? v : k;
  uint8_t* cache = which ? v_cache : k_cache;
  const int c = lane & 15, odd = lane >> 4;

  for (; heads; heads &= heads - 1) {
    const int at = __ffs(heads) - 1;
    const int64_t t0 = first + at;
    const int64_t blk = __shfl_sync(0xffffffffu, mine, at);
    // not the first of its block if one of the bs - 1 tokens before it goes there too
    bool seen = false;
#pragma unroll
    for (int i = 0; i < (kBs + 30) / 32; ++i) {
      const int back = 1 + i * 32 + lane;
      seen |= back < kBs && block_of(t0 - back) == blk;
    }
    if (__any_sync(0xffffffffu, seen)) continue;

    // ---- this warp's 16 tokens: where they go, their elements ----
    int off = -1;
    if (lane < kWarpRows) {
      const int64_t t = t0 + w * kWarpRows + lane;
      if (block_of(t) == blk) off = static_cast<int>(slots[t] & (kBs - 1));
    }
    uint4 x[8];
    __half2 big = as_h2(0u);
    __half2 lo[4], hi[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      lo[j] = as_h2(0x7c007c00u);
      hi[j] = as_h2(0xfc00fc00u);
    }
    const bool any = __any_sync(0xffffffffu, off >= 0);
    if (any) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool live = __shfl_sync(0xffffffffu, off, 2 * i + odd) >= 0;
        const int64_t t = t0 + w * kWarpRows + 2 * i + odd;
        x[i] = live ? src[(t * num_kv_heads + h) * 16 + c] : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool live = __shfl_sync(0xffffffffu, off, 2 * i + odd) >= 0;
        const __half2* p = reinterpret_cast<const __half2*>(&x[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          big = __hmax2_nan(big, __habs2(p[j]));
          if (live) {
            lo[j] = __hmin2(lo[j], p[j]);
            hi[j] = __hmax2(hi[j], p[j]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
    float top = __half2float(__hmax_nan(__low2half(big), __high2half(big)));
    // ---- the team's: largest element, rows written ----
    if (W > 1) {
      if (lane == 0) {
        top_s[team][w] = top;
        rows_s[team][w] = 0u;
      }
      team_sync();
      if (off >= 0) atomicOr(&rows_s[team][off >> 4], 1u << (off & 15));
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float o = top_s[team][i];
        top = o != o || top != top ? __uint_as_float(kNanBits) : fmaxf(top, o);
      }
      if (bounds && which == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = __hmin2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
          hi[j] = __hmax2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
        }
        ends_s[team][w][lane] =
            odd ? make_uint4(h2_bits(hi[0]), h2_bits(hi[1]), h2_bits(hi[2]), h2_bits(hi[3]))
                : make_uint4(h2_bits(lo[0]), h2_bits(lo[1]), h2_bits(lo[2]), h2_bits(lo[3]));
      }
      team_sync();
    }
    uint32_t written;   // of this warp's 16 rows of the block
    bool fresh;
    if (W == 1) {
      written = off >= 0 ? 1u << off : 0u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) written |= __shfl_xor_sync(0xffffffffu, written, o);
      fresh = written & 1u;
    } else {
      written = rows_s[team][w];
      fresh = rows_s[team][0] & 1u;
    }
    // ---- the scale ----
    const int64_t bh = blk * num_kv_heads + h;
    float* scale_at = scales + bh * 2 + which;
    const float need = int8_scale(top);
    const float old = fresh ? 0.f : *scale_at;
    const float s = fresh ? need : int8_grown(need, old);
    const float r = int8_inverse(s);
    const float factor = old * r;   // <= 1; 0 for a fresh block and for NaN
    uint8_t* block = cache + bh * (kBs * 128);
    // every thread has read the scale, and the team's shared arrays, before one is written again
    team_sync();
    if (w == 0 && lane == 0 && (fresh || !(s == old))) *scale_at = s;
    // ---- the block's other rows ----
    if (fresh || !(s == old)) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 4 * i + (lane >> 3);
        if ((written >> row) & 1u) continue;
        uint4* p = reinterpret_cast<uint4*>(block + (w * kWarpRows + row) * 128) + (lane & 7);
        uint4 u = make_uint4(kInt8Zeros, kInt8Zeros, kInt8Zeros, kInt8Zeros);
        if (factor > 0.f) {
          u = *p;
          u = make_uint4(int8_rescaled(u.x, factor), int8_rescaled(u.y, factor),
                         int8_rescaled(u.z, factor), int8_rescaled(u.w, factor));
        }
        *p = u;
      }
    }
    // ---- the new rows ----
    if (any) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int o = __shfl_sync(0xffffffffu, off, 2 * i + odd);
        if (o >= 0) reinterpret_cast<uint2*>(block + o * 128)[c] = int8_codes(x[i], r);
      }
    }
    // ---- the keys' bounds: the least and the greatest new code are the codes of the least and
    // the greatest element ----
    if (bounds && which == 0 && w == 0) {
      uint4 e;
      if (W == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          lo[j] = __hmin2(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
          hi[j] = __hmax2(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
        }
        e = odd ? make_uint4(h2_bits(hi[0]), h2_bits(hi[1]), h2_bits(hi[2]), h2_bits(hi[3]))
                : make_uint4(h2_bits(lo[0]), h2_bits(lo[1]), h2_bits(lo[2]), h2_bits(lo[3]));
      } else {
        e = ends_s[team][0][lane];
#pragma unroll
        for (int i = 1; i < W; ++i) {
          const uint4 o = ends_s[team][i][lane];
          const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
          uint32_t ew[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ew[j] = h2_bits(odd ? __hmax2(as_h2(ew[j]), as_h2(ow[j]))
                                : __hmin2(as_h2(ew[j]), as_h2(ow[j])));
          e = make_uint4(ew[0], ew[1], ew[2], ew[3]);
        }
      }
      uint2 u = int8_codes(e, r);
      uint2* to = reinterpret_cast<uint2*>(bounds + bh * 256) + lane;   // least codes, then greatest
      if (!fresh && r != 0.f) {
        uint2 b = *to;
        if (!(s == old)) b = make_uint2(int8_rescaled(b.x, factor), int8_rescaled(b.y, factor));
        u = odd ? make_uint2(__vmaxu4(u.x, b.x), __vmaxu4(u.y, b.y))
                : make_uint2(__vminu4(u.x, b.x), __vminu4(u.y, b.y));
      }
      *to = u;
    }
    if (W > 1) team_sync();   // the shared arrays serve the next block
  }
}

// The grid enumerates (pair, K|V) and, within it, `parts` CTAs that stride over the block's rows, 16
// lanes a row, kWiden rows a thread with all of their loads in flight.
constexpr int kWiden = 4;
__global__ void __launch_bounds__(kThreads)
widen_blocks_int8_kernel(const uint8_t* k_cache, const uint8_t* v_cache, const float* scales,
                         const int32_t* src, const int32_t* dst, int num_blocks,
                         int num_blocks_out, int num_kv_heads, int parts, int bs_shift,
                         uint4* k_out, uint4* v_out, unsigned int* err) {
  griddep_wait();
  const int job = blockIdx.x / parts, part = blockIdx.x - job * parts;
  const int which = job & 1;
  const int32_t s = src[job >> 1], d = dst[job >> 1];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks_out) {
    if (part == 0 && threadIdx.x == 0) atomicOr(err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  constexpr int kRows = kThreads / 16;
  const int c = threadIdx.x & 15, r0 = threadIdx.x >> 4;
  const int block_rows = num_kv_heads << bs_shift;
  const uint2* from = reinterpret_cast<const uint2*>(which ? v_cache : k_cache) +
                      static_cast<int64_t>(s) * block_rows * 16 + c;
  uint4* to = (which ? v_out : k_out) + static_cast<int64_t>(d) * block_rows * 16 + c;
  const float* sc = scales + static_cast<int64_t>(s) * num_kv_heads * 2 + which;
  for (int r = part * (kRows * kWiden) + r0; r < block_rows; r += parts * (kRows * kWiden)) {
    uint2 u[kWiden];
    float f[kWiden];
#pragma unroll
    for (int i = 0; i < kWiden; ++i) {
      const int row = r + i * kRows;
      u[i] = make_uint2(0u, 0u);
      f[i] = 0.f;
      if (row < block_rows) {
        u[i] = from[static_cast<int64_t>(row) * 16];
        f[i] = sc[2 * (row >> bs_shift)];
      }
    }
#pragma unroll
    for (int i = 0; i < kWiden; ++i) {
      const int row = r + i * kRows;
      if (row >= block_rows) break;
      const uint32_t x = u[i].x, y = u[i].y;
      __stcs(to + static_cast<int64_t>(row) * 16,
             make_uint4(pack_half2(int8_value<0>(x) * f[i], int8_value<1>(x) * f[i]),
                        pack_half2(int8_value<2>(x) * f[i], int8_value<3>(x) * f[i]),
                        pack_half2(int8_value<0>(y) * f[i], int8_value<1>(y) * f[i]),
                        pack_half2(int8_value<2>(y) * f[i], int8_value<3>(y) * f[i])));
    }
  }
}

// (layer, pair) in grid x, parts of a block's bytes in grid y: K, V, bounds and scales of a block.
__global__ void __launch_bounds__(kThreads)
copy_blocks_int8_kernel(uint4* k_cache, uint4* v_cache, float2* scales, uint4* bounds,
                        const int32_t* src, const int32_t* dst, int n, int num_blocks,
                        int num_kv_heads, int bs, unsigned int* err) {
  griddep_wait();
  const int layer = blockIdx.x / n, pair = blockIdx.x - layer * n;
  const int32_t s = src[pair], d = dst[pair];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks) {
    if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  const int64_t from = static_cast<int64_t>(layer) * num_blocks + s,
                to = static_cast<int64_t>(layer) * num_blocks + d;
  const int per = num_kv_heads * bs * 8;   // 16-byte pieces of a block
  const int step = gridDim.y * kThreads, t = blockIdx.y * kThreads + threadIdx.x;
  for (int i = t; i < per; i += step) {
    const uint4 a = k_cache[from * per + i], b = v_cache[from * per + i];
    k_cache[to * per + i] = a;
    v_cache[to * per + i] = b;
  }
  for (int i = t; i < num_kv_heads; i += step)
    scales[to * num_kv_heads + i] = scales[from * num_kv_heads + i];
  if (bounds)
    for (int i = t; i < num_kv_heads * 16; i += step)
      bounds[to * num_kv_heads * 16 + i] = bounds[from * num_kv_heads * 16 + i];
}

int log2_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

int launch_status() { return cuda_status(cudaGetLastError()); }

template <int W, class... A>
int launch_append(int64_t jobs, pkv_stream_t stream, A... args) {
  constexpr int kTeams = W < 4 ? 4 / W : 1;
  return launch_waiting(&kv_append_int8_kernel<W>, static_cast<unsigned>((jobs + kTeams - 1) / kTeams),
                        W < 4 ? kThreads : W * 32, 0, stream, args...);
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_kv_append_int8(const void* k, const void* v, const int64_t* slot_mapping, int num_tokens,
                       void* k_cache, void* v_cache, float* kv_scales, void* k_bounds,
                       int num_blocks, int num_kv_heads, int head_dim, int block_size,
                       pkv_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 0 || num_kv_heads <= 0 || head_dim != 128 ||
      !valid_block_size(block_size))
    return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache || !kv_scales) return PKV_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(k_bounds) || (reinterpret_cast<uintptr_t>(kv_scales) & 7u))
    return PKV_EINVAL;
  // Few rows: a team for every token, so that a step's blocks are all taken at once. Many: a team
  // for kSpan tokens, most of which go to one block.
  const int64_t rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
  const int span = rows <= 4096 ? 1 : kSpan;
  const int64_t jobs = (static_cast<int64_t>(num_tokens) + span - 1) / span * num_kv_heads * 2;
  if (jobs > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  auto launch = [&](auto w) {
    return launch_append<decltype(w)::value>(
        jobs, stream, static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping,
        num_tokens, static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), kv_scales,
        static_cast<uint8_t*>(k_bounds), static_cast<int64_t>(num_blocks) * block_size,
        num_kv_heads, span, static_cast<unsigned>(jobs), err);
  };
  switch (block_size) {
    case 16: return launch(std::integral_constant<int, 1>());
    case 32: return launch(std::integral_constant<int, 2>());
    case 64: return launch(std::integral_constant<int, 4>());
    case 128: return launch(std::integral_constant<int, 8>());
    default: return launch(std::integral_constant<int, 16>());
  }
}

int pkv_widen_blocks_int8(const void* k_cache, const void* v_cache, const float* kv_scales,
                          const int32_t* src, const int32_t* dst, int n, int num_blocks,
                          void* k_out, void* v_out, int num_blocks_out, int num_kv_heads,
                          int head_dim, int block_size, pkv_stream_t stream) {
  if (n < 0 || num_blocks < 0 || num_blocks_out < 0 || num_kv_heads <= 0 || head_dim != 128 ||
      !valid_block_size(block_size))
    return PKV_EINVAL;
  if (n == 0) return PKV_OK;
  if (!k_cache || !v_cache || !kv_scales || !src || !dst || !k_out || !v_out) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out) ||
      (reinterpret_cast<uintptr_t>(kv_scales) & 7u))
    return PKV_EINVAL;
  const int64_t rows = static_cast<int64_t>(num_kv_heads) * block_size;
  const int64_t parts =
      std::min<int64_t>((rows * 16 + kThreads * kWiden - 1) / (kThreads * kWiden), 1024);
  if (rows * 16 > 0x3fffffff || 2LL * n * parts > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  return launch_waiting(&widen_blocks_int8_kernel, static_cast<unsigned>(2LL * n * parts), kThreads,
                        0, stream, static_cast<const uint8_t*>(k_cache),
                        static_cast<const uint8_t*>(v_cache), kv_scales, src, dst, num_blocks,
                        num_blocks_out, num_kv_heads, static_cast<int>(parts), log2_of(block_size),
                        static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), err);
}

int pkv_copy_blocks_int8(void* k_cache, void* v_cache, float* kv_scales, void* k_bounds,
                         const int32_t* src, const int32_t* dst, int n, int num_layers,
                         int num_blocks, int num_kv_heads, int head_dim, int block_size,
                         pkv_stream_t stream) {
  if (n < 0 || num_layers < 0 || num_blocks < 0 || num_kv_heads <= 0 || head_dim != 128 ||
      !valid_block_size(block_size))
    return PKV_EINVAL;
  if (n == 0 || num_layers == 0) return PKV_OK;
  if (!k_cache || !v_cache || !kv_scales || !src || !dst) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_bounds) ||
      (reinterpret_cast<uintptr_t>(kv_scales) & 7u))
    return PKV_EINVAL;
  const int64_t pieces = static_cast<int64_t>(num_kv_heads) * block_size * 8;
  const int64_t pairs = static_cast<int64_t>(n) * num_layers;
  if (pieces > 0x3fffffff || pairs > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  const int parts = static_cast<int>(std::min<int64_t>((pieces + 4 * kThreads - 1) / (4 * kThreads), 256));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs), static_cast<unsigned>(parts));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(
      &cfg, copy_blocks_int8_kernel, static_cast<uint4*>(k_cache), static_cast<uint4*>(v_cache),
      reinterpret_cast<float2*>(kv_scales), static_cast<uint4*>(k_bounds), src, dst, n, num_blocks,
      num_kv_heads, block_size, err));
}

}  // extern "C"
