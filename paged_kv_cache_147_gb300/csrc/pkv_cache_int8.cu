// pkv_cache_int8.cu -- the 8-bit cache's own edits: the append (quantise, scatter, and bring the
// touched blocks to their new scales), the widening of whole blocks to fp16, and the block copy.
//
// All move bytes. The append reads 256 and writes 128 per row; a block that rows are added to is
// read and written again only when its scale grows (its largest element doubles, so a few times
// in a block's life). A scale needs all of a block's new rows before the first code, so that the rows
// stay in registers between the two (16 rows a warp) and are read once: 8192 tokens of 8 heads in
// 16-token blocks take 13.2 us (50 MB, 3.8 TB/s: two waves of warps, none of which loads its next
// block's rows while it writes this one's codes), 64 tokens of 2 heads 2.9 (a launch and three
// dependent loads). Widening 8192 tokens: 9.6 us (5.3 TB/s). Copying 64 blocks of 8 heads and 16 tokens
// in each of 80 layers: 54 us (357 MB, 6.6 TB/s), 8 blocks of one layer 2.5 (a launch and two).
#include <algorithm>

#include "pkv_int8.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarpRows = 16;    // rows of a block that a warp holds in registers

__device__ __forceinline__ __half2 as_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }
__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ uint4 pick(bool second, const __half2 (&a)[4], const __half2 (&b)[4]) {
  return second ? make_uint4(h2_bits(b[0]), h2_bits(b[1]), h2_bits(b[2]), h2_bits(b[3]))
                : make_uint4(h2_bits(a[0]), h2_bits(a[1]), h2_bits(a[2]), h2_bits(a[3]));
}

struct AppendArgs {
  const uint4* k;
  const uint4* v;
  const int64_t* slots;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* scales;
  uint8_t* bounds;
  unsigned int* err;
  int64_t num_slots;
  int num_tokens, num_kv_heads, span;
  unsigned jobs;
};

// What the G warps that take a block's rows share.
template <int G, int BS>
struct Shared {
  float top[G];
  uint32_t rows[BS / kWarpRows];   // which rows of the block the call writes, 16 to a word
  uint4 ends[G][32];               // per channel least and greatest new element
};

// Where a token's row goes: its block (-1: nowhere) and its place there.
struct Slot {
  int blk, off;
};

// The rows of one call that go to one block (slots sl[0 ..], the block's first one first, all within
// BS tokens from t0 on; G = 1: within 16), for kv head h and K or V, by G warps: warp w has 16 tokens'
// rows in its registers between the pass that finds the scale and the one that writes codes.
template <int G, int BS, class Sync>
__device__ __forceinline__ void append_block(const AppendArgs& a, const Slot* sl, int64_t t0, int h,
                                             int which, int w, int lane, Shared<G, BS>& sh,
                                             Sync sync) {
  constexpr int kWords = BS / kWarpRows;
  const uint4* src = which ? a.v : a.k;
  const int c = lane & 15, odd = lane >> 4;
  const int blk = sl[0].blk;
  int off = -1;
  if (lane < kWarpRows) {
    const Slot s = sl[w * kWarpRows + lane];
    if (s.blk == blk) off = s.off;
  }
  // (a token that goes elsewhere counts as the block's first one, which changes no extreme)
  uint4 x[8];
  const unsigned live = __ballot_sync(0xffffffffu, off >= 0) >> odd;
  src += (t0 * a.num_kv_heads + h) * 16 + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = (live >> (2 * i)) & 1u ? w * kWarpRows + 2 * i + odd : 0;
    x[i] = src[static_cast<int64_t>(row) * a.num_kv_heads * 16];
  }
  const int64_t bh = static_cast<int64_t>(blk) * a.num_kv_heads + h;
  float* scale_at = a.scales + bh * 2 + which;
  const float had = *scale_at;
  const bool bounded = a.bounds && which == 0;

  // ---- largest element; for keys per channel least and greatest ----
  __half2 lo[4], hi[4], big = as_h2(0u);
#pragma unroll
  for (int j = 0; j < 4; ++j) lo[j] = hi[j] = as_h2(j == 0 ? x[0].x : j == 1 ? x[0].y : j == 2 ? x[0].z : x[0].w);
  if (bounded) {
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const __half2* p = reinterpret_cast<const __half2*>(&x[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = __hmin2_nan(lo[j], p[j]);
        hi[j] = __hmax2_nan(hi[j], p[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      big = __hmax2_nan(big, __hmax2_nan(__habs2(lo[j]), __habs2(hi[j])));
      lo[j] = __hmin2_nan(lo[j], __shfl_xor_sync(0xffffffffu, lo[j], 16));
      hi[j] = __hmax2_nan(hi[j], __shfl_xor_sync(0xffffffffu, hi[j], 16));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2* p = reinterpret_cast<const __half2*>(&x[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) big = __hmax2_nan(big, __habs2(p[j]));
    }
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
  float top = __half2float(__hmax_nan(__low2half(big), __high2half(big)));
  uint4 ends = pick(odd, lo, hi);   // of the channels 8 c ..: lanes 0-15 the least, 16-31 the greatest
  // ---- the group's ----
  uint32_t written[kWords];         // (G = 1, BS = 16: in registers; else in shared memory)
  bool fresh;
  if (kWords == 1) {
    uint32_t m = off >= 0 ? 1u << off : 0u;
    written[0] = __reduce_or_sync(0xffffffffu, m);
    fresh = written[0] & 1u;
  } else {
    for (int i = w * 32 + lane; i < kWords; i += G * 32) sh.rows[i] = 0u;
    if (G > 1) {
      if (lane == 0) sh.top[w] = top;
      if (bounded) sh.ends[w][lane] = ends;
    }
    sync();
    if (off >= 0) atomicOr(&sh.rows[off >> 4], 1u << (off & 15));
    sync();
    fresh = sh.rows[0] & 1u;
    if (G > 1) {
#pragma unroll
      for (int i = 0; i < G; ++i) {
        const float o = sh.top[i];
        top = o != o || top != top ? __uint_as_float(kNanBits) : fmaxf(top, o);
      }
      if (bounded && w == 0) {
#pragma unroll
        for (int i = 1; i < G; ++i) {
          const uint4 o = sh.ends[i][lane];
          const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
          uint32_t ew[4] = {ends.x, ends.y, ends.z, ends.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ew[j] = h2_bits(odd ? __hmax2(as_h2(ew[j]), as_h2(ow[j]))
                                : __hmin2(as_h2(ew[j]), as_h2(ow[j])));
          ends = make_uint4(ew[0], ew[1], ew[2], ew[3]);
        }
      }
    }
  }
  // ---- the scale ----
  const float need = int8_scale(top);
  const float old = fresh ? 0.f : had;
  const float s = fresh ? need : int8_grown(need, old);
  const Int8Mover move(old * int8_inverse(s));   // nothing stays in a fresh block, or of a NaN
  uint8_t* block = (which ? a.v_cache : a.k_cache) + bh * (BS * 128);
  const bool moved = fresh || !(s == old);
  sync();   // every thread has read the scale
  if (w == 0 && lane == 0 && moved) *scale_at = s;
  // ---- the new rows ----
  const Int8Quantiser quant(s);
  uint2* rows = reinterpret_cast<uint2*>(block) + c;
  if (quant.kind == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int o = __shfl_sync(0xffffffffu, off, 2 * i + odd);
      if (o >= 0) rows[o * 16] = quant.codes<true>(x[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int o = __shfl_sync(0xffffffffu, off, 2 * i + odd);
      if (o >= 0) rows[o * 16] = quant.codes(x[i]);
    }
  }
  // ---- the block's other rows ----
  if (moved && !(kWords == 1 && written[0] == 0xffffu)) {
    // 4 rows a warp, four times with the loads ahead of the first use
    constexpr int kPass = 4 * G;
    uint4* at = reinterpret_cast<uint4*>(block) + lane;   // (8 lanes a row)
    auto mine = [&](int row) {
      const uint32_t word = kWords == 1 ? written[0] : sh.rows[row >> 4];
      return !((word >> (row & 15)) & 1u);
    };
    if (!move.none) {
#pragma unroll 1
      for (int r0 = 4 * w; r0 < BS; r0 += 4 * kPass) {
        uint4 u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (r0 + i * kPass < BS) u[i] = at[(r0 + i * kPass) * 8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = r0 + i * kPass;
          if (row < BS && mine(row + (lane >> 3)))
            at[row * 8] = move(u[i]);
        }
      }
    } else {
      for (int row = 4 * w; row < BS; row += kPass)
        if (mine(row + (lane >> 3)))
          at[row * 8] = make_uint4(kInt8Zeros, kInt8Zeros, kInt8Zeros, kInt8Zeros);
    }
  }
  // ---- the keys' bounds: the least and the greatest new code are the codes of the least and
  // the greatest element ----
  if (bounded && w == 0) {
    uint2 u = quant.codes(ends);
    uint2* to = reinterpret_cast<uint2*>(a.bounds + bh * 256) + lane;   // least codes, then greatest
    if (!fresh && s == s) {
      uint2 b = *to;
      if (moved) b = make_uint2(move(b.x), move(b.y));
      u = odd ? make_uint2(__vmaxu4(u.x, b.x), __vmaxu4(u.y, b.y))
              : make_uint2(__vminu4(u.x, b.x), __vminu4(u.y, b.y));
    }
    *to = u;
  }
  if (kWords > 1) sync();   // the shared words serve the next block
}

// A team of W warps (W 16 rows make a block) takes, for one kv head and K or V, every block whose
// first row of the call is among its `span` tokens. Blocks that get rows of 16 consecutive tokens at
// most go to one warp each, the others to the whole team.
template <int W>
__global__ void __launch_bounds__(W < 4 ? kThreads : W * 32, W == 16 ? 2 : W == 8 ? 4 : W == 4 ? 8 : 7)
kv_append_int8_kernel(const AppendArgs a) {
  griddep_wait();
  constexpr int kTeams = W < 4 ? 4 / W : 1;
  constexpr int kBs = W * kWarpRows;
  constexpr int kShift = W == 1 ? 4 : W == 2 ? 5 : W == 4 ? 6 : W == 8 ? 7 : 8;
  constexpr int kSlots = 3 * kBs - 2, kMasks = (kBs + 31) / 32;
  __shared__ Slot slots_s[kTeams][kSlots];   // the span's, kBs - 1 before it and behind it
  __shared__ uint32_t first_s[kTeams][kMasks], wide_s[kTeams][kMasks];   // blocks' first tokens; for the team
  __shared__ Shared<1, kBs> warp_s[kTeams * W];
  __shared__ Shared<W, kBs> team_s[kTeams];
  const int lane = threadIdx.x & 31;
  const int team = threadIdx.x / (W * 32), w = (threadIdx.x >> 5) % W, t = threadIdx.x % (W * 32);
  const unsigned job = blockIdx.x * kTeams + team;
  if (job >= a.jobs) return;
  const unsigned which = job & 1;
  const unsigned part = (job >> 1) / a.num_kv_heads;
  const int h = static_cast<int>((job >> 1) - part * a.num_kv_heads);
  const int64_t first = static_cast<int64_t>(part) * a.span;
  auto team_sync = [&]() {
    if (W == 1) __syncwarp();
    else named_barrier_sync(1 + team, W * 32);
  };
  const Slot* sl = slots_s[team];
  // the span's rows start on their way while their slots are looked up (a row is two lines)
  if (a.span > 1)
    for (int i = t; i < 2 * a.span; i += W * 32)
      if (first + (i >> 1) < a.num_tokens)
        prefetch_l2((which ? a.v : a.k) + ((first + (i >> 1)) * a.num_kv_heads + h) * 16 + (i & 1) * 8);
  for (int i = t; i < 2 * (kBs - 1) + a.span; i += W * 32) {
    const int64_t at = first - (kBs - 1) + i;
    int64_t s = at >= 0 && at < a.num_tokens ? a.slots[at] : -1;
    if (s >= a.num_slots) {
      if (which == 0 && h == 0) atomicOr(a.err, PKV_DEVERR_SLOT);
      s = -1;
    }
    slots_s[team][i] = s < 0 ? Slot{-1, 0}
                             : Slot{static_cast<int>(s >> kShift), static_cast<int>(s & (kBs - 1))};
  }
  if (t < kMasks) first_s[team][t] = wide_s[team][t] = 0u;
  team_sync();
  // ---- the first tokens of blocks: no token of the kBs - 1 before goes there ----
  for (int i0 = 0; i0 < a.span; i0 += 32) {
    bool cand = false;
    if (i0 + lane < a.span) {
      const int b = sl[kBs - 1 + i0 + lane].blk;
      cand = b >= 0 && b != sl[kBs - 2 + i0 + lane].blk;
    }
    int turn = 0;
    for (unsigned m = __ballot_sync(0xffffffffu, cand); m; m &= m - 1, ++turn) {
      if (W > 1 && turn % W != w) continue;
      const int i = i0 + __ffs(m) - 1, at = kBs - 1 + i;
      const int blk = sl[at].blk;
      bool before = false, far = false;
#pragma unroll
      for (int j = 0; j < (kBs + 31) / 32; ++j) {
        const int d = 1 + 32 * j + lane;
        if (d < kBs) {
          before |= sl[at - d].blk == blk;
          far |= d >= kWarpRows && sl[at + d].blk == blk;
        }
      }
      before = __any_sync(0xffffffffu, before);
      far = __any_sync(0xffffffffu, far);
      if (lane == 0 && !before)
        atomicOr(far ? &wide_s[team][i0 >> 5] : &first_s[team][i0 >> 5], 1u << (i & 31));
    }
  }
  team_sync();
  int k = 0;
  for (int o = 0; o < kBs; o += 32)
    for (unsigned m = first_s[team][o >> 5]; m; m &= m - 1, ++k) {
      if (W > 1 && k % W != w) continue;
      const int i = o + __ffs(m) - 1;
      append_block<1, kBs>(a, sl + kBs - 1 + i, first + i, h, which, 0, lane,
                           warp_s[threadIdx.x >> 5], [] { __syncwarp(); });
    }
  if constexpr (W > 1) {
    for (int o = 0; o < kBs; o += 32)
      for (unsigned m = wide_s[team][o >> 5]; m; m &= m - 1) {
        const int i = o + __ffs(m) - 1;
        append_block<W, kBs>(a, sl + kBs - 1 + i, first + i, h, which, w, lane, team_s[team],
                             team_sync);
      }
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

template <int W>
int launch_append(const AppendArgs& args, pkv_stream_t stream) {
  constexpr int kTeams = W < 4 ? 4 / W : 1;
  return launch_waiting(&kv_append_int8_kernel<W>, (args.jobs + kTeams - 1) / kTeams,
                        W < 4 ? kThreads : W * 32, 0, stream, args);
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
  // Few rows: a team for every token, so that a step's blocks are all taken at once. Many: as many tokens
  // a team as leave 4096 warps, about as many as are resident, but a block's worth at most, so that
  // calls of 32768 tokens times heads and more have more than one wave. Measured, us: 8192 tokens of 8
  // heads in blocks of 16 with 1, 4, 8, 16 tokens a team 40.4, 17.9, 14.3, 13.2; 2048 tokens with 1, 4, 8,
  // 16: 10.0, 6.4, 5.2, 5.2; those in blocks of 256 with 64, 128, 256: 14.8, 12.5, 15.8; single tokens of
  // 512 sequences, blocks of 16, with 1, 2, 4: 7.4, 6.7, 8.5.
  const int64_t halves = static_cast<int64_t>(num_kv_heads) * 2;   // K and V of a head
  const int64_t warps = num_tokens * halves * (block_size / 16);
  const int span = static_cast<int>(std::min<int64_t>(std::max<int64_t>(warps / 4096, 1), block_size));
  const int64_t jobs = (static_cast<int64_t>(num_tokens) + span - 1) / span * halves;
  if (jobs > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  AppendArgs args = {};
  args.span = span;
  args.jobs = static_cast<unsigned>(jobs);
  args.k = static_cast<const uint4*>(k);
  args.v = static_cast<const uint4*>(v);
  args.slots = slot_mapping;
  args.k_cache = static_cast<uint8_t*>(k_cache);
  args.v_cache = static_cast<uint8_t*>(v_cache);
  args.scales = kv_scales;
  args.bounds = static_cast<uint8_t*>(k_bounds);
  args.err = err;
  args.num_slots = static_cast<int64_t>(num_blocks) * block_size;
  args.num_tokens = num_tokens;
  args.num_kv_heads = num_kv_heads;
  switch (block_size) {
    case 16: return launch_append<1>(args, stream);
    case 32: return launch_append<2>(args, stream);
    case 64: return launch_append<4>(args, stream);
    case 128: return launch_append<8>(args, stream);
    default: return launch_append<16>(args, stream);
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
