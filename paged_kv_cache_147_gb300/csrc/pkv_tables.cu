// pkv_tables.cu -- block tables and slot maps kept on the GPU: growing each sequence's table for
// a step's new tokens out of a stack of free blocks (and mapping those tokens to their slots),
// and cutting tables back.
//
// With old lengths n_b, new tokens m_b and block size s, sequence b needs
// ceil((n_b + m_b) / s) - ceil(n_b / s) blocks. An exclusive prefix sum over the sequences says
// which blocks of the stack it gets and where its tokens stand in the packed order; everything
// else is independent per token and per block.
//
// There is next to nothing to move (20 bytes per token, 8 per block): a launch and a few dependent
// round trips bound it. So one launch does it all: every CTA of one cluster scans all sequences
// by itself (at most kMaxTableSeqs, in shared memory), then takes its share of the tokens and
// blocks; the cluster barrier keeps the lengths and the stack's count, updated in place at the
// end, from changing under a CTA that has not read them yet. Past kClusterTokens tokens (or
// kClusterBlocks table entries to cut) one cluster's 8 SMs no longer write fast enough: a grid
// over the whole GPU does the tokens and blocks first and a second, one-CTA launch the rest; it
// starts beside the first (dependent launch), scans, and writes when the first is done (256 prompts
// of up to 4096 tokens, with the cut: 15.4 us one after the other, 11.8 so; a draft step of 64
// sequences, cut and extend: 8.8).
#include <algorithm>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

// Threads of a CTA: 256 while four sequences a thread suffice, or 1024 (an extend by 4 tokens and a
// cut in a row, us, against the other: 1024 sequences 9.8 / 13.7, 4096 sequences 18.3 / 27).
constexpr int kMaxThreads = 1024;
int threads_for(int num_seqs) { return num_seqs <= 1024 ? 256 : kMaxThreads; }
constexpr int kMaxTableSeqs = 4096;
constexpr int kMaxCluster = 8;
// An extend and a cut in a row, one cluster against the grid and the second launch, us: 4096 tokens
// 7.3 / 7.8, 8192 8.3 / 8.1, 16384 10.1 / 8.6, 32768 12.6 / 8.4, 262144 61 / 10.5. The cut's bound
// is the tables' capacity, of which most calls cut little (64 sequences whose tables hold 8320
// entries, a draft step: 8.8 / 9.1).
constexpr int kClusterTokens = 8192;
constexpr int kClusterBlocks = 16384;

struct TableArgs {
  int32_t* tables;
  int32_t* lens;
  const int32_t* arg;        // extend: new tokens per sequence; truncate: tokens to keep
  int32_t* free_blocks;
  int32_t* free_count;
  int64_t* slots;
  int32_t* seqs;
  int64_t* positions;
  int32_t* cu;
  int num_seqs, max_blocks, block_size, bs_shift, num_blocks, max_tokens;
  bool vec;                  // the token arrays are 16-byte aligned
  unsigned int* err;
};

__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}

// The scan of a call's second launch runs before its wait. What the kernels before the call wrote is
// in L2 by then (the first launch waited for them before it let the second one in), so it reads there.
template <bool BEFORE_WAIT>
__device__ __forceinline__ int scan_load(const int32_t* p) {
  return BEFORE_WAIT ? __ldcg(p) : *p;
}

// Exclusive sums of two 64-bit values over the CTA's threads, and their totals.
__device__ __forceinline__ void cta_scan(int64_t& x, int64_t& y, int64_t& total_x,
                                         int64_t& total_y, int64_t (*part)[2]) {
  const int warps = blockDim.x / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ux = __shfl_up_sync(0xffffffffu, ix, o);
    const int64_t uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) { ix += ux; iy += uy; }
  }
  if (lane == 31) { part[warp][0] = ix; part[warp][1] = iy; }
  __syncthreads();
  // every warp scans the warps' sums by itself
  int64_t px = lane < warps ? part[lane][0] : 0, py = lane < warps ? part[lane][1] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ux = __shfl_up_sync(0xffffffffu, px, o);
    const int64_t uy = __shfl_up_sync(0xffffffffu, py, o);
    if (lane >= o) { px += ux; py += uy; }
  }
  total_x = __shfl_sync(0xffffffffu, px, warps - 1);
  total_y = __shfl_sync(0xffffffffu, py, warps - 1);
  const int64_t bx = __shfl_sync(0xffffffffu, px, max(warp - 1, 0));
  const int64_t by = __shfl_sync(0xffffffffu, py, max(warp - 1, 0));
  x = ix - x + (warp ? bx : 0);
  y = iy - y + (warp ? by : 0);
}

// Largest b in [0, n) with first[b] <= x (first[0] = 0 <= x).
__device__ __forceinline__ int find(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int blocks_of(int64_t tokens, int shift) {
  return static_cast<int>((tokens + (1 << shift) - 1) >> shift);
}

// TOKENS: the token arrays and the new table entries; STATE: lengths, count and error bits.
// Shared memory: tok[n + 1], blk[n + 1], len[n].
template <bool TOKENS, bool STATE>
__global__ void __launch_bounds__(kMaxThreads) extend_kernel(const TableArgs a) {
  extern __shared__ int smem[];
  __shared__ int64_t part[kMaxThreads / 32][2];
  __shared__ int used_s;
  int* tok = smem;                       // first packed token of each sequence
  int* blk = tok + a.num_seqs + 1;       // first block (from the top of the stack)
  int* len = blk + a.num_seqs + 1;       // old length; -1: refused
  const int n = a.num_seqs, sh = a.bs_shift;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int rank = TOKENS && STATE ? cluster_rank() : blockIdx.x;
  const int ctas = TOKENS && STATE ? cluster_size() : gridDim.x;
  const int64_t cap = static_cast<int64_t>(a.max_blocks) << sh;
  unsigned int bad = 0;

  if (TOKENS) griddep_wait();                          // the launch before this call's
  if (TOKENS && !STATE) griddep_launch_dependents();   // the second launch scans meanwhile
  int count = scan_load<!TOKENS>(a.free_count);
  if (count < 0 || count > a.num_blocks) { bad |= PKV_DEVERR_SPACE; count = 0; }
  if (tid == 0) used_s = 0;

  // ---- the scan: each thread takes `per` neighbouring sequences ----
  const int per = (n + threads - 1) / threads;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  int64_t x = 0, y = 0;
  for (int b = b0; b < b1; ++b) {
    const int ctx = scan_load<!TOKENS>(a.lens + b), m = scan_load<!TOKENS>(a.arg + b);
    const bool ok = ctx >= 0 && ctx <= cap && m >= 0 && ctx + static_cast<int64_t>(m) <= cap;
    x += max(m, 0);
    if (ok) y += blocks_of(ctx + static_cast<int64_t>(m), sh) - blocks_of(ctx, sh);
  }
  int64_t total_x, total_y;
  cta_scan(x, y, total_x, total_y, part);
  int used = 0;
  for (int b = b0; b < b1; ++b) {
    const int ctx = scan_load<!TOKENS>(a.lens + b), m = scan_load<!TOKENS>(a.arg + b);
    bool ok = true;
    int need = 0;
    if (ctx < 0 || ctx > cap || m < 0) {
      bad |= PKV_DEVERR_CONTEXT;
      ok = false;
    } else if (ctx + static_cast<int64_t>(m) > cap) {
      bad |= PKV_DEVERR_POSITION;
      ok = false;
    } else {
      need = blocks_of(ctx + static_cast<int64_t>(m), sh) - blocks_of(ctx, sh);
    }
    tok[b] = static_cast<int>(min(x, static_cast<int64_t>(a.max_tokens)));
    blk[b] = static_cast<int>(min(y, static_cast<int64_t>(0x7fffffff)));
    x += max(m, 0);
    y += need;
    if (ok && (x > a.max_tokens || (need > 0 && y > count))) {
      bad |= PKV_DEVERR_SPACE;
      ok = false;
    }
    if (ok && need > 0) used = static_cast<int>(y);
    len[b] = ok ? ctx : -1;
  }
  if (used > 0) atomicMax(&used_s, used);
  const int live = static_cast<int>(min(total_x, static_cast<int64_t>(a.max_tokens)));
  if (tid == 0) {
    tok[n] = live;
    blk[n] = static_cast<int>(min(total_y, static_cast<int64_t>(count)));
  }
  __syncthreads();
  used = used_s;
  if (TOKENS && STATE) cluster_arrive();   // this CTA has read the lengths and the count

  if (TOKENS) {
    // ---- the new tokens, and the padding behind them, four neighbours a thread ----
    for (int64_t i0 = 4 * (static_cast<int64_t>(rank) * threads + tid); i0 < a.max_tokens;
         i0 += 4 * static_cast<int64_t>(ctas) * threads) {
      int64_t slot[4], pos[4];
      int seq[4];
      int b = i0 < live ? find(tok, n, static_cast<int>(i0)) : n;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int64_t i = i0 + e;
        slot[e] = pos[e] = -1;
        seq[e] = -1;
        if (i >= live) continue;
        while (tok[b + 1] <= i) ++b;
        const int ctx = len[b];
        if (ctx < 0) continue;
        seq[e] = b;
        pos[e] = ctx + (i - tok[b]);
        const int lb = static_cast<int>(pos[e] >> sh), held = blocks_of(ctx, sh);
        const int id = lb < held ? a.tables[static_cast<int64_t>(b) * a.max_blocks + lb]
                                 : a.free_blocks[count - 1 - (blk[b] + lb - held)];
        if (id >= 0 && id < a.num_blocks)
          slot[e] = (static_cast<int64_t>(id) << sh) + (pos[e] & ((1 << sh) - 1));
        else
          bad |= PKV_DEVERR_BLOCK_ID;
      }
      if (a.vec && i0 + 4 <= a.max_tokens) {
        longlong2* s2 = reinterpret_cast<longlong2*>(a.slots + i0);
        longlong2* p2 = reinterpret_cast<longlong2*>(a.positions + i0);
        s2[0] = make_longlong2(slot[0], slot[1]);
        s2[1] = make_longlong2(slot[2], slot[3]);
        p2[0] = make_longlong2(pos[0], pos[1]);
        p2[1] = make_longlong2(pos[2], pos[3]);
        *reinterpret_cast<int4*>(a.seqs + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      } else {
        for (int e = 0; e < 4 && i0 + e < a.max_tokens; ++e) {
          a.slots[i0 + e] = slot[e];
          a.seqs[i0 + e] = seq[e];
          a.positions[i0 + e] = pos[e];
        }
      }
    }
    // ---- the new table entries ----
    for (int k = rank * threads + tid; k < used; k += ctas * threads) {
      const int b = find(blk, n, k);
      if (len[b] < 0) continue;
      const int id = a.free_blocks[count - 1 - k];
      if (id < 0 || id >= a.num_blocks) bad |= PKV_DEVERR_BLOCK_ID;
      a.tables[static_cast<int64_t>(b) * a.max_blocks + blocks_of(len[b], sh) + (k - blk[b])] = id;
    }
    for (int b = rank * threads + tid; b <= n; b += ctas * threads) a.cu[b] = tok[b];
  }
  if (bad) atomicOr(a.err, bad);
  if (STATE) {
    if (TOKENS) cluster_wait(); else griddep_wait();
    for (int b = rank * threads + tid; b < n; b += ctas * threads)
      if (len[b] >= 0) a.lens[b] = len[b] + a.arg[b];
    if (rank == 0 && tid == 0 && used > 0) *a.free_count = count - used;
  }
}

// BLOCKS: the table entries and the stack; STATE: lengths and count. Shared memory: blk[n + 1],
// keep[n].
template <bool BLOCKS, bool STATE>
__global__ void __launch_bounds__(kMaxThreads) truncate_kernel(const TableArgs a) {
  extern __shared__ int smem[];
  __shared__ int64_t part[kMaxThreads / 32][2];
  int* blk = smem;                       // first freed block of each sequence
  int* keep = blk + a.num_seqs + 1;      // length kept; -1: as it is
  const int n = a.num_seqs, sh = a.bs_shift;
  const int tid = threadIdx.x, threads = blockDim.x;
  const int rank = BLOCKS && STATE ? cluster_rank() : blockIdx.x;
  const int ctas = BLOCKS && STATE ? cluster_size() : gridDim.x;
  const int64_t cap = static_cast<int64_t>(a.max_blocks) << sh;
  unsigned int bad = 0;

  if (BLOCKS) griddep_wait();
  if (BLOCKS && !STATE) griddep_launch_dependents();
  int count = scan_load<!BLOCKS>(a.free_count);
  if (count < 0 || count > a.num_blocks) { bad |= PKV_DEVERR_SPACE; count = a.num_blocks; }
  const int per = (n + threads - 1) / threads;
  const int b0 = min(n, tid * per), b1 = min(n, b0 + per);
  int64_t x = 0, unused = 0;
  for (int b = b0; b < b1; ++b) {
    const int ctx = scan_load<!BLOCKS>(a.lens + b), m = scan_load<!BLOCKS>(a.arg + b);
    if (ctx >= 0 && ctx <= cap && m >= 0 && m < ctx) x += blocks_of(ctx, sh) - blocks_of(m, sh);
  }
  int64_t total, total_unused;
  cta_scan(x, unused, total, total_unused, part);
  const bool fits = count + total <= a.num_blocks;
  if (!fits) bad |= PKV_DEVERR_SPACE;
  for (int b = b0; b < b1; ++b) {
    const int ctx = scan_load<!BLOCKS>(a.lens + b), m = scan_load<!BLOCKS>(a.arg + b);
    const bool known = ctx >= 0 && ctx <= cap;
    if (!known) bad |= PKV_DEVERR_CONTEXT;
    const bool cut = known && m >= 0 && m < ctx;
    blk[b] = fits ? static_cast<int>(x) : 0;
    if (cut) x += blocks_of(ctx, sh) - blocks_of(m, sh);
    keep[b] = cut && fits ? m : -1;
  }
  const int freed = fits ? static_cast<int>(total) : 0;
  if (tid == 0) blk[n] = freed;
  __syncthreads();
  if (BLOCKS && STATE) cluster_arrive();   // this CTA has read the lengths and the count

  if (BLOCKS) {
    for (int k = rank * threads + tid; k < freed; k += ctas * threads) {
      const int b = find(blk, n, k);
      int32_t* entry = a.tables + static_cast<int64_t>(b) * a.max_blocks +
                       blocks_of(keep[b], sh) + (k - blk[b]);
      const int id = *entry;
      if (id < 0 || id >= a.num_blocks) bad |= PKV_DEVERR_BLOCK_ID;
      a.free_blocks[count + freed - 1 - k] = id;
      *entry = -1;
    }
  }
  if (bad) atomicOr(a.err, bad);
  if (STATE) {
    if (BLOCKS) cluster_wait(); else griddep_wait();
    for (int b = rank * threads + tid; b < n; b += ctas * threads)
      if (keep[b] >= 0) a.lens[b] = keep[b];
    if (rank == 0 && tid == 0 && freed > 0) *a.free_count = count + freed;
  }
}

int launch_status() { return cuda_status(cudaGetLastError()); }

// The one number an extend of no sequences by no tokens writes: cu_new_lens[0] = 0. Such a call may
// come without outputs, so an address that CUDA does not know (or no device at all) is left alone.
int write_empty_total(int32_t* cu, cudaStream_t stream) {
  cudaPointerAttributes at = {};
  if (!cu) return PKV_OK;
  if (cudaPointerGetAttributes(&at, cu) != cudaSuccess) {
    cudaGetLastError();   // not this call's to report
    return PKV_OK;
  }
  if (at.type == cudaMemoryTypeUnregistered) return PKV_OK;
  return cuda_status(cudaMemsetAsync(cu, 0, sizeof(int32_t), stream));
}

// `cluster` > 0: one cluster of that many CTAs; 0: `ctas` CTAs on their own. May start while the
// launch before it ends: the first (or only) launch of a call waits for that before it reads
// anything, a second one before it writes.
int launch(const void* fn, const TableArgs& a, size_t smem, int cluster, int ctas,
           cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  if (smem > 47 * 1024)   // past the default limit, beside the kernels' own 528 bytes
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>((3 * kMaxTableSeqs + 2) * sizeof(int)));
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster ? cluster : ctas);
  cfg.blockDim = dim3(threads_for(a.num_seqs));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  void* params[1] = {const_cast<TableArgs*>(&a)};
  return cuda_status(cudaLaunchKernelExC(&cfg, fn, params));
}

int log2_of(int n) {
  int s = 0;
  while ((1 << s) < n) ++s;
  return s;
}

int cluster_for(int64_t items, int per_cta) {
  int c = 1;
  while (c < kMaxCluster && static_cast<int64_t>(c) * per_cta < items) c *= 2;
  return c;
}

bool valid_tables(int num_seqs, int max_blocks, int block_size, int num_blocks) {
  return num_seqs >= 0 && num_seqs <= kMaxTableSeqs && max_blocks >= 0 && num_blocks >= 0 &&
         valid_block_size(block_size) &&
         static_cast<int64_t>(max_blocks) * block_size <= 0x7fffffff;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_extend_tables(int32_t* block_tables, int32_t* context_lens, const int32_t* new_lens,
                      int num_seqs, int max_blocks_per_seq, int block_size, int32_t* free_blocks,
                      int32_t* free_count, int num_blocks, int64_t* slot_out, int32_t* seq_out,
                      int64_t* position_out, int32_t* cu_new_lens, int max_tokens,
                      pkv_stream_t stream) {
  if (!valid_tables(num_seqs, max_blocks_per_seq, block_size, num_blocks) || max_tokens < 0)
    return PKV_EINVAL;
  if (num_seqs == 0 && max_tokens == 0)
    return write_empty_total(cu_new_lens, static_cast<cudaStream_t>(stream));
  if ((num_seqs > 0 && (!context_lens || !new_lens)) ||
      (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) ||
      (num_blocks > 0 && !free_blocks) || !free_count || !cu_new_lens ||
      (max_tokens > 0 && (!slot_out || !seq_out || !position_out)))
    return PKV_EINVAL;
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  TableArgs a = {block_tables, context_lens, new_lens, free_blocks, free_count, slot_out, seq_out,
                 position_out, cu_new_lens, num_seqs, max_blocks_per_seq, block_size,
                 log2_of(block_size), num_blocks, max_tokens,
                 ((at(slot_out) | at(seq_out) | at(position_out)) & 15u) == 0, device_error_ptr()};
  if (!a.err) return launch_status();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = threads_for(num_seqs);
  const size_t smem = (3 * static_cast<size_t>(num_seqs) + 2) * sizeof(int);
  if (max_tokens <= kClusterTokens)
    return launch(reinterpret_cast<const void*>(&extend_kernel<true, true>), a, smem,
                  cluster_for(max_tokens, 4 * threads), 0, s);
  const int ctas = std::min(1024 / threads * sm_count(), (max_tokens / 4 + threads) / threads);
  if (ctas < 1) return launch_status();
  const int st =
      launch(reinterpret_cast<const void*>(&extend_kernel<true, false>), a, smem, 0, ctas, s);
  if (st != PKV_OK) return st;
  return launch(reinterpret_cast<const void*>(&extend_kernel<false, true>), a, smem, 0, 1, s);
}

int pkv_truncate_tables(int32_t* block_tables, int32_t* context_lens, const int32_t* keep_lens,
                        int num_seqs, int max_blocks_per_seq, int block_size,
                        int32_t* free_blocks, int32_t* free_count, int num_blocks,
                        pkv_stream_t stream) {
  if (!valid_tables(num_seqs, max_blocks_per_seq, block_size, num_blocks)) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if ((max_blocks_per_seq > 0 && !block_tables) || !context_lens || !keep_lens ||
      (num_blocks > 0 && !free_blocks) || !free_count)
    return PKV_EINVAL;
  TableArgs a = {block_tables, context_lens, keep_lens, free_blocks, free_count, nullptr, nullptr,
                 nullptr, nullptr, num_seqs, max_blocks_per_seq, block_size, log2_of(block_size),
                 num_blocks, 0, false, device_error_ptr()};
  if (!a.err) return launch_status();
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int threads = threads_for(num_seqs);
  const size_t smem = (2 * static_cast<size_t>(num_seqs) + 1) * sizeof(int);
  // at most this many entries leave the tables
  const int64_t most = std::min<int64_t>(static_cast<int64_t>(num_seqs) * max_blocks_per_seq,
                                         num_blocks);
  if (most <= kClusterBlocks)
    return launch(reinterpret_cast<const void*>(&truncate_kernel<true, true>), a, smem,
                  cluster_for(most, 4 * threads), 0, s);
  const int ctas =
      std::min<int64_t>(2 * sm_count(), (most + threads - 1) / threads);
  if (ctas < 1) return launch_status();
  const int st =
      launch(reinterpret_cast<const void*>(&truncate_kernel<true, false>), a, smem, 0, ctas, s);
  if (st != PKV_OK) return st;
  return launch(reinterpret_cast<const void*>(&truncate_kernel<false, true>), a, smem, 0, 1, s);
}

}  // extern "C"
