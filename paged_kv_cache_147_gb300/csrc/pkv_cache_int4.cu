// pkv_cache_int4.cu -- the 4-bit cache's own edits: the append (quantise and scatter) and the
// widening of whole blocks to fp16.
//
// Both move bytes: the append reads 256 and writes 80 per row, the widening the other way round.
// 16 lanes take a row, 8 elements (16 fp16 bytes, 4 bytes of codes) each, or, in large appends, 4
// lanes a group of 32 each. 8192 tokens of 8 heads (44 MB each way): append 10.1 us, widening 6.9
// (4.4 and 6.4 TB/s).
#include <algorithm>

#include "pkv_int4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kRowLanes = 16;

// Half-warp = one (token, kv head): its K row and its V row. The two half-warps of a warp take
// neighbouring tokens of one head, which usually are neighbouring rows of a block.
__global__ void __launch_bounds__(kThreads)
kv_append_int4_kernel(const uint4* k, const uint4* v, const int64_t* slots, int num_tokens,
                      uint8_t* k_cache, uint8_t* v_cache, int64_t num_slots, int num_kv_heads,
                      int bs_shift, unsigned int* err) {
  griddep_wait();
  const int lane = threadIdx.x & 31, c = lane & (kRowLanes - 1);
  const unsigned warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned pair = warp / num_kv_heads;
  const int h = static_cast<int>(warp - pair * num_kv_heads);
  const int64_t t = 2 * static_cast<int64_t>(pair) + (lane >> 4);
  const bool in = t < num_tokens;
  const int64_t slot = in ? slots[t] : -1;
  if (in && slot >= num_slots && c == 0 && h == 0) atomicOr(err, PKV_DEVERR_SLOT);
  const bool live = slot >= 0 && slot < num_slots;
  const int64_t src = (t * num_kv_heads + h) * kRowLanes + c;
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const uint4 x = live ? k[src] : zero, y = live ? v[src] : zero;
  uint32_t kc, kp, vc, vp;
  int4_quantise(x, kc, kp);
  int4_quantise(y, vc, vp);
  if (!live) return;
  const int64_t blk = slot >> bs_shift, off = slot & ((1 << bs_shift) - 1);
  const int64_t row = (((blk * num_kv_heads + h) << bs_shift) + off) * kInt4Row;
  uint32_t* kd = reinterpret_cast<uint32_t*>(k_cache + row);
  uint32_t* vd = reinterpret_cast<uint32_t*>(v_cache + row);
  kd[c] = kc;
  vd[c] = vc;
  if ((c & 3) == 0) {
    kd[kInt4Params / 4 + (c >> 2)] = kp;
    vd[kInt4Params / 4 + (c >> 2)] = vp;
  }
}

// Many rows: a thread takes a whole group (64 bytes in, 16 + 4 out), a warp the K or the V rows of
// eight neighbouring tokens of one head. The group's minimum, maximum and scale are then computed
// once instead of in four lanes, which is what a full GPU spends its time on otherwise: 65536 tokens
// of 8 heads 91 us against 66, 8192 tokens 14.2 against 10.6 (2048 tokens 4.8 against 4.2); below
// kGroupRows the longer chain per thread shows (512 tokens 2.75 against 3.0, 64 tokens of 2 heads
// 2.1 against 2.3).
constexpr int kGroupRows = 16384;
__global__ void __launch_bounds__(kThreads)
kv_append_int4_groups_kernel(const uint4* k, const uint4* v, const int64_t* slots, int num_tokens,
                             uint8_t* k_cache, uint8_t* v_cache, int64_t num_slots,
                             int num_kv_heads, int bs_shift, unsigned int* err) {
  griddep_wait();
  const int lane = threadIdx.x & 31, g = lane & 3;
  const unsigned warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  const unsigned job = warp >> 1, which = warp & 1;
  const unsigned oct = job / num_kv_heads;
  const int h = static_cast<int>(job - oct * num_kv_heads);
  const int64_t t = 8 * static_cast<int64_t>(oct) + (lane >> 2);
  if (t >= num_tokens) return;
  const int64_t slot = slots[t];
  if (slot >= num_slots && g == 0 && h == 0 && which == 0) atomicOr(err, PKV_DEVERR_SLOT);
  if (slot < 0 || slot >= num_slots) return;
  const uint4* src = (which ? v : k) + (t * num_kv_heads + h) * kRowLanes + 4 * g;
  const uint4 x[4] = {__ldcs(src), __ldcs(src + 1), __ldcs(src + 2), __ldcs(src + 3)};
  uint4 codes;
  uint32_t params;
  int4_quantise_group(x, codes, params);
  const int64_t blk = slot >> bs_shift, off = slot & ((1 << bs_shift) - 1);
  uint8_t* row = (which ? v_cache : k_cache) +
                 (((blk * num_kv_heads + h) << bs_shift) + off) * kInt4Row;
  reinterpret_cast<uint4*>(row)[g] = codes;
  reinterpret_cast<uint32_t*>(row + kInt4Params)[g] = params;
}

// The grid enumerates (pair, K|V) and, within it, `parts` CTAs that stride over the block's rows,
// 16 lanes a row. A thread takes kWiden rows at a time and has all of their loads in flight
// before the first use (with one row at a time the latency showed: 9.4 us for 44 MB). The fp16
// blocks are written past the caches' usual order (streaming): the pools stay in L2 (9.8 -> 7.5 us).
constexpr int kWiden = 4;
__global__ void __launch_bounds__(kThreads)
widen_blocks_int4_kernel(const uint8_t* k_cache, const uint8_t* v_cache, const int32_t* src,
                         const int32_t* dst, int num_blocks, int num_blocks_out, int parts,
                         int block_rows, uint4* k_out, uint4* v_out, unsigned int* err) {
  griddep_wait();
  const int job = blockIdx.x / parts, part = blockIdx.x - job * parts;
  const int which = job & 1;
  const int32_t s = src[job >> 1], d = dst[job >> 1];
  if (s < 0 || s >= num_blocks || d < 0 || d >= num_blocks_out) {
    if (part == 0 && threadIdx.x == 0) atomicOr(err, PKV_DEVERR_BLOCK_ID);
    return;
  }
  constexpr int kRows = kThreads / kRowLanes;   // rows the CTA takes at once
  const int c = threadIdx.x & (kRowLanes - 1), r0 = threadIdx.x / kRowLanes;
  const uint32_t* from = reinterpret_cast<const uint32_t*>(
      (which ? v_cache : k_cache) + static_cast<int64_t>(s) * block_rows * kInt4Row);
  uint4* to = (which ? v_out : k_out) + static_cast<int64_t>(d) * block_rows * kRowLanes + c;
  for (int r = part * (kRows * kWiden) + r0; r < block_rows; r += parts * (kRows * kWiden)) {
    uint32_t w[kWiden], sz[kWiden];
#pragma unroll
    for (int i = 0; i < kWiden; ++i) {
      const int row = r + i * kRows;
      w[i] = sz[i] = 0u;
      if (row < block_rows) {
        w[i] = from[row * (kInt4Row / 4) + c];
        sz[i] = from[row * (kInt4Row / 4) + kInt4Params / 4 + (c >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < kWiden; ++i) {
      const int row = r + i * kRows;
      if (row >= block_rows) break;
      const __half2 sc = __low2half2(as_half2(sz[i])), mn = __high2half2(as_half2(sz[i]));
      // (elements 0, 4), (1, 5), (2, 6), (3, 7), each s * code + z rounded once
      const uint32_t e04 = half2_bits(__hfma2(int4_lo(w[i]), sc, mn));
      const uint32_t e15 = half2_bits(__hfma2(int4_hi(w[i]), sc, mn));
      const uint32_t e26 = half2_bits(__hfma2(int4_lo(w[i] >> 8), sc, mn));
      const uint32_t e37 = half2_bits(__hfma2(int4_hi(w[i] >> 8), sc, mn));
      __stcs(to + static_cast<int64_t>(row) * kRowLanes,
             make_uint4(__byte_perm(e04, e15, 0x5410), __byte_perm(e26, e37, 0x5410),
                        __byte_perm(e04, e15, 0x7632), __byte_perm(e26, e37, 0x7632)));
    }
  }
}

int log2_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

int launch_status() { return cuda_status(cudaGetLastError()); }

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_kv_append_int4(const void* k, const void* v, const int64_t* slot_mapping, int num_tokens,
                       void* k_cache, void* v_cache, int num_blocks, int num_kv_heads,
                       int head_dim, int block_size, pkv_stream_t stream) {
  if (num_tokens < 0 || num_blocks < 0 || num_kv_heads <= 0 || head_dim != 128 ||
      !valid_block_size(block_size))
    return PKV_EINVAL;
  if (num_tokens == 0) return PKV_OK;
  if (!k || !v || !slot_mapping || !k_cache || !v_cache) return PKV_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return PKV_EINVAL;
  const int64_t rows = static_cast<int64_t>(num_tokens) * num_kv_heads;
  const bool groups = rows >= kGroupRows;
  const int64_t warps = groups ? (static_cast<int64_t>(num_tokens) + 7) / 8 * num_kv_heads * 2
                               : (static_cast<int64_t>(num_tokens) + 1) / 2 * num_kv_heads;
  const int64_t blocks = (warps * 32 + kThreads - 1) / kThreads;
  if (warps > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  const auto kernel = groups ? &kv_append_int4_groups_kernel : &kv_append_int4_kernel;
  return launch_waiting(kernel, static_cast<unsigned>(blocks), kThreads, 0, stream,
                        static_cast<const uint4*>(k), static_cast<const uint4*>(v), slot_mapping,
                        num_tokens, static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache),
                        static_cast<int64_t>(num_blocks) * block_size, num_kv_heads,
                        log2_of(block_size), err);
}

int pkv_widen_blocks_int4(const void* k_cache, const void* v_cache, const int32_t* src,
                          const int32_t* dst, int n, int num_blocks, void* k_out, void* v_out,
                          int num_blocks_out, int num_kv_heads, int head_dim, int block_size,
                          pkv_stream_t stream) {
  if (n < 0 || num_blocks < 0 || num_blocks_out < 0 || num_kv_heads <= 0 || head_dim != 128 ||
      !valid_block_size(block_size))
    return PKV_EINVAL;
  if (n == 0) return PKV_OK;
  if (!k_cache || !v_cache || !src || !dst || !k_out || !v_out) return PKV_EINVAL;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_out) || !aligned16(v_out))
    return PKV_EINVAL;
  const int64_t rows = static_cast<int64_t>(num_kv_heads) * block_size;
  const int64_t parts =
      std::min<int64_t>((rows * kRowLanes + kThreads * kWiden - 1) / (kThreads * kWiden), 1024);
  if (rows * kRowLanes > 0x3fffffff || 2LL * n * parts > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return launch_status();
  // Shared memory that it does not use keeps a small grid at four CTAs an SM: behind a fused decode,
  // which lets its successor in early, the first SMs to finish would take all of it (a fused step
  // of 64 ragged sequences and the widening 18.4 us -> 16.7, of 32 of 50 to 8000 tokens 51.2 -> 49.6;
  // on its own or behind an append a widening takes as long either way).
  const int64_t grid = 2LL * n * parts;
  const size_t smem = grid <= 4LL * sm_count() ? 46 * 1024 : 0;
  return launch_waiting(&widen_blocks_int4_kernel, static_cast<unsigned>(grid), kThreads, smem,
                        stream, static_cast<const uint8_t*>(k_cache),
                        static_cast<const uint8_t*>(v_cache), src, dst, num_blocks, num_blocks_out,
                        static_cast<int>(parts), static_cast<int>(rows), static_cast<uint4*>(k_out),
                        static_cast<uint4*>(v_out), err);
}

}  // extern "C"
