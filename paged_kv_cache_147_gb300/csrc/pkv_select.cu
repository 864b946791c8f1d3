// pkv_select.cu -- the blocks of a long context that each kv head's queries attend to, by a bound on
// their scores (sm_103a).
//
// What it computes: for a sequence and kv head with query rows r (new tokens x heads of the group),
// rounded to whole numbers p_r in -127 .. 127 times a power of two 2^(e_r), and a block j whose key
// codes lie in [lo_d, hi_d] per channel at the scale s_j:
//   score_j = max_r 2^(e_r) s_j sum_d max(p_rd lo_d, p_rd hi_d),
// no less than any rounded query's product with any key of the block. The first and last blocks are
// kept, and those of the largest scores up to the budget.
//
// The sum is one product of 256 terms, min(p, 0) against lo and max(p, 0) against hi: whole numbers
// below 2^22 times powers of two, exact in fp32 whatever the order, so that the choice (ties to the
// lower block) is the definition's. Codes go to the tensor cores as fp16 subnormals u 2^-24 with
// their offset taken off in the accumulator (as in pkv_decode_int8.cu), straight from global memory: a
// dot's terms may come in any order, so 16 bytes of a row are four operands of a lane.
//
// What bounds it: 256 bytes of bounds per block and head, and for few of them latency. One cluster
// per (sequence, kv head): its CTAs share the blocks, keep their scores in shared memory as ordered
// integers, and find the budget's smallest score by four rounds of 256-bin counts added up through
// distributed shared memory. One launch, no workspace.
#include <cuda_fp16.h>

#include <algorithm>
#include <map>
#include <mutex>

#include "pkv_decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_int8.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kAlways = 0xffffffffu;     // key of a block that is kept whatever its score
constexpr uint32_t kNanKey = 0xfffffffeu;     // a NaN scale: before every number

struct SelectArgs {
  const __half* q;
  const float* scales;
  const uint8_t* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* tables_out;
  int32_t* lens_out;
  unsigned int* err;
  int num_blocks, max_blocks, q_len, Hq, Hkv, G, R;
  int block_size, bs_shift;   // bs_shift = log2(block_size)
  int budget, keep_first, keep_last;
  int C, cap;                 // CTAs per cluster, keys a CTA has room for
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// a word in CTA `rank`'s copy of this CTA's shared variable p
__device__ __forceinline__ uint32_t ld_cluster_u32(const uint32_t* p, uint32_t rank) {
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// Larger numbers have larger keys; -0 does not come here.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t b = __float_as_uint(s);
  return s == s ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : kNanKey;
}

// Exclusive scan of one value per thread; `total` gets the sum.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* sh, uint64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  uint64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < warp) before += sh[i];
    total += sh[i];
  }
  return before + incl - v;
}

// NT: tiles of 8 query rows.
template <int NT>
__global__ void __launch_bounds__(kThreads)
select_blocks_kernel(const SelectArgs a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t smem[];
  uint2* frag = reinterpret_cast<uint2*>(smem);                   // [NT][16][32]
  float4* col = reinterpret_cast<float4*>(frag + NT * 512);       // [8 NT] offset, factor, bias, -
  uint32_t* hist = reinterpret_cast<uint32_t*>(col + 8 * NT);     // [4][256]
  uint32_t* keys = hist + 1024;                                   // [cap]
  __shared__ uint64_t scan_s[kWarps];
  __shared__ uint32_t found_s[2];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const uint32_t rank = a.C > 1 ? cluster_rank() : 0;
  const int unit = blockIdx.x / a.C;
  const int b = unit / a.Hkv, h = unit - b * a.Hkv;
  int ctx = a.context_lens[b];
  if (ctx < 0 || ctx > a.max_blocks * a.block_size) {
    if (rank == 0 && h == 0 && tid == 0) atomicOr(a.err, PKV_DEVERR_CONTEXT);
    ctx = ctx < 0 ? 0 : a.max_blocks * a.block_size;
  }
  const int nblk = (ctx + a.block_size - 1) >> a.bs_shift;
  const int n = min(nblk, a.budget);
  const int32_t* table = a.block_tables + static_cast<int64_t>(b) * a.max_blocks;
  int32_t* out = a.tables_out + static_cast<int64_t>(unit) * a.budget;
  if (h == 0 && rank == 0 && tid == 0) a.lens_out[b] = ctx - (nblk - n) * a.block_size;
  // entries without a block, and all of a context within the budget
  for (int i = rank * kThreads + tid; i < a.budget; i += a.C * kThreads) {
    if (i >= n) out[i] = -1;
    else if (nblk == n) out[i] = table[i];
  }
  if (nblk == n) return;

  // ---- the queries: whole numbers as the products' B operands ----
  for (int i = tid; i < 1024; i += kThreads) hist[i] = 0u;
  for (int r = warp; r < 8 * NT; r += kWarps) {
    const int qi = r / a.G;
    uint2 v = make_uint2(0u, 0u);
    const bool sees = r < a.R && ctx - a.q_len + qi >= 0;
    if (sees)
      v = reinterpret_cast<const uint2*>(
          a.q + ((static_cast<int64_t>(b) * a.q_len + qi) * a.Hq + h * a.G + r - qi * a.G) * kD)[lane];
    const __half2 x = *reinterpret_cast<const __half2*>(&v.x);
    const __half2 y = *reinterpret_cast<const __half2*>(&v.y);
    __half2 big = __hmax2_nan(__habs2(x), __habs2(y));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
    const float s = int8_scale(__half2float(__hmax_nan(__low2half(big), __high2half(big))));
    const float inv = int8_inverse(s);
    const float2 fx = __half22float2(x), fy = __half22float2(y);
    float p[4] = {fx.x, fx.y, fy.x, fy.y};
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (a row with a NaN or an infinity counts for nothing)
      p[i] = s == s ? fminf(fmaxf(rintf(p[i] * inv), -127.f), 127.f) : 0.f;
      sum += p[i];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // dims 4 lane .. + 3: word `lane & 3` of 16-byte piece (lane >> 2) & 3 of 64-byte part lane >> 4
    uint2* to = frag + (r >> 3) * 512 + ((lane >> 4) * 4 + (lane & 3)) * 32 + (r & 7) * 4 +
                ((lane >> 2) & 3);
    to[0] = make_uint2(pack_half2(fminf(p[0], 0.f), fminf(p[2], 0.f)),
                       pack_half2(fminf(p[1], 0.f), fminf(p[3], 0.f)));
    to[8 * 32] = make_uint2(pack_half2(fmaxf(p[0], 0.f), fmaxf(p[2], 0.f)),
                            pack_half2(fmaxf(p[1], 0.f), fmaxf(p[3], 0.f)));
    if (lane == 0) {
      const bool counts = sees && s == s;
      col[r] = make_float4(sum * -0x1p-17f, counts ? 0x1p24f * s : 0.f, counts ? 0.f : kNegInf, 0.f);
    }
  }
  __syncthreads();

  // ---- scores of this CTA's blocks, 16 a warp at a time ----
  const int per = ((nblk + a.C - 1) / a.C + 15) & ~15;
  const int lo = min(nblk, static_cast<int>(rank) * per), count = min(nblk, lo + per) - lo;
  const int tail = nblk - max(a.keep_last, nblk - (max(ctx - a.q_len, 0) >> a.bs_shift));
  auto id_of = [&](int j) { return j < count ? table[lo + j] : -1; };
  int next[2] = {id_of(16 * warp + g), id_of(16 * warp + g + 8)};
#pragma unroll 1
  for (int j0 = 16 * warp; j0 < count; j0 += 16 * kWarps) {
    uint4 w[2][4];
    float sc[2];
    bool good[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      good[o] = next[o] >= 0 && next[o] < a.num_blocks;
      const int64_t bh = static_cast<int64_t>(good[o] ? next[o] : 0) * a.Hkv + h;
      const uint4* src = reinterpret_cast<const uint4*>(a.bounds + bh * 256) + t4;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[o][i] = good[o] ? src[4 * i] : make_uint4(0, 0, 0, 0);
      sc[o] = good[o] ? a.scales[bh * 2] : 0.f;
      if (!good[o] && j0 + g + 8 * o < count && t4 == 0) atomicOr(a.err, PKV_DEVERR_BLOCK_ID);
      next[o] = id_of(j0 + 16 * kWarps + g + 8 * o);
    }
    float best[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 c0 = col[8 * nt + 2 * t4], c1 = col[8 * nt + 2 * t4 + 1];
      float acc[4] = {c0.x, c1.x, c0.x, c1.x};
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint2 f = frag[nt * 512 + (4 * i + e) * 32 + lane];
          const uint32_t u0 = u4_word(w[0][i], e), u1 = u4_word(w[1][i], e);
          mma_f16(acc, u0 & 0x00ff00ffu, u1 & 0x00ff00ffu, __byte_perm(u0, 0u, 0x4341),
                  __byte_perm(u1, 0u, 0x4341), f.x, f.y);
        }
#pragma unroll
      for (int o = 0; o < 2; ++o)
        best[o] = fmaxf(best[o], fmaxf(fmaf(acc[2 * o], c0.y, c0.z), fmaf(acc[2 * o + 1], c1.y, c1.z)));
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      best[o] = fmaxf(best[o], __shfl_xor_sync(0xffffffffu, best[o], 1));
      best[o] = fmaxf(best[o], __shfl_xor_sync(0xffffffffu, best[o], 2));
      const int j = j0 + g + 8 * o;
      if (t4 == 0 && j < count) {
        // (+ 0 turns -0 into 0; a scale of 0 must not meet -infinity)
        float s = best[o] == kNegInf ? kNegInf : best[o] * sc[o] + 0.f;
        if (!good[o]) s = kNegInf;
        keys[j] = lo + j < a.keep_first || lo + j >= tail ? kAlways : key_of(s);
      }
    }
  }
  __syncthreads();

  // ---- the n-th largest key: a byte of it per round ----
  uint32_t prefix = 0, need = n;
  uint32_t gt_before = 0, eq_before = 0;   // larger keys (this thread's share), equal ones: lower ranks
#pragma unroll 1
  for (int round = 0; round < 4; ++round) {
    const int shift = 24 - 8 * round;
    uint32_t* hr = hist + 256 * round;
    for (int j = tid; j < count; j += kThreads) {
      const uint32_t key = keys[j];
      if (round == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(hr + ((key >> shift) & 255u), 1u);
    }
    if (a.C > 1) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    const uint32_t bin = 255 - tid;        // the largest first
    uint32_t all = 0, before = 0;
    if (a.C > 1) {
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= a.C) break;
        const uint32_t v = ld_cluster_u32(hr + bin, c);
        all += v;
        if (c < static_cast<int>(rank)) before += v;
      }
    } else {
      all = hr[bin];
    }
    uint64_t total;
    const uint32_t above = static_cast<uint32_t>(block_scan(all, scan_s, total));
    if (above < need && need <= above + all) {
      found_s[0] = bin;
      found_s[1] = need - above;
    }
    if (round == 3) keys[a.cap + tid] = before;   // by bin, for the equal ones
    __syncthreads();
    const uint32_t digit = found_s[0];
    need = found_s[1];
    prefix |= digit << shift;
    if (bin > digit) gt_before += before;
    if (round == 3) eq_before = keys[a.cap + 255 - digit];
  }
  if (a.C > 1) cluster_arrive();   // this CTA has read the others' counts

  // ---- the chosen blocks in their order ----
  uint64_t sum;
  block_scan(gt_before, scan_s, sum);
  gt_before = static_cast<uint32_t>(sum);
  const int run = (count + kThreads - 1) / kThreads;
  const int k0 = min(count, tid * run), k1 = min(count, k0 + run);
  uint64_t mine = 0;   // larger keys in the upper half, equal ones in the lower
  for (int j = k0; j < k1; ++j) {
    const uint32_t key = keys[j];
    mine += key > prefix ? 1ull << 32 : (key == prefix ? 1ull : 0ull);
  }
  const uint64_t ahead = block_scan(mine, scan_s, sum);
  uint32_t gt = gt_before + static_cast<uint32_t>(ahead >> 32);
  uint32_t eq = eq_before + static_cast<uint32_t>(ahead);
  for (int j = k0; j < k1; ++j) {
    const uint32_t key = keys[j];
    if (key > prefix) {
      out[gt + min(eq, need)] = table[lo + j];
      ++gt;
    } else if (key == prefix) {
      if (eq < need) out[gt + eq] = table[lo + j];
      ++eq;
    }
  }
  if (a.C > 1) cluster_wait();     // the others have read this CTA's
}

// ---------------------------------------------------------------------------------------------
// Host side.

const void* kernel_for(int R) {
  return R <= 8    ? reinterpret_cast<const void*>(&select_blocks_kernel<1>)
         : R <= 16 ? reinterpret_cast<const void*>(&select_blocks_kernel<2>)
         : R <= 24 ? reinterpret_cast<const void*>(&select_blocks_kernel<3>)
                   : reinterpret_cast<const void*>(&select_blocks_kernel<4>);
}

// CTAs per cluster: at least as many in all as fill the SMs, while each has 128 blocks and more.
int cluster_for(int64_t units, int max_blocks) {
  int c = 1;
  while (c < kMaxCluster && units * c < 2LL * sm_count() && max_blocks >= 256 * c) c *= 2;
  return c;
}

// Raises the kernel's limit of dynamic shared memory to the device's, once per device and kernel.
cudaError_t allow_smem(const void* fn) {
  static std::mutex mu;
  static std::map<std::pair<int, const void*>, bool> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (done.count({dev, fn})) return cudaSuccess;
  int limit = 0;
  e = cudaDeviceGetAttribute(&limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaFuncAttributes fa;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             limit - static_cast<int>(fa.sharedSizeBytes));
  if (e == cudaSuccess) done[{dev, fn}] = true;
  return e;
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" int pkv_select_blocks(int32_t* tables_out, int32_t* lens_out, const void* q,
                                 const float* kv_scales, const void* k_bounds, int num_blocks,
                                 const int32_t* block_tables, int max_blocks_per_seq,
                                 const int32_t* context_lens, int num_seqs, int q_len,
                                 int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                 int budget, int keep_first, int keep_last, pkv_stream_t stream) {
  if (num_seqs < 0 || q_len < 1 || num_q_heads < 1 || num_kv_heads < 1 ||
      num_q_heads % num_kv_heads != 0 || head_dim != kD || !valid_block_size(block_size) ||
      num_blocks < 1 || max_blocks_per_seq < 0 || max_blocks_per_seq > kMaxCluster * 32768 ||
      budget < 1 || keep_first < 0 || keep_last < 0)
    return PKV_EINVAL;
  const int G = num_q_heads / num_kv_heads;
  if (static_cast<int64_t>(G) * q_len > 32) return PKV_EINVAL;
  const int ends = std::max(keep_last, 1 + (q_len - 1 + block_size - 1) / block_size);
  if (static_cast<int64_t>(keep_first) + ends > budget) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (!tables_out || !lens_out || !q || !kv_scales || !k_bounds || !block_tables || !context_lens)
    return PKV_EINVAL;
  if (!aligned16(q) || !aligned16(k_bounds) || (reinterpret_cast<uintptr_t>(kv_scales) & 7u))
    return PKV_EINVAL;
  const int64_t units = static_cast<int64_t>(num_seqs) * num_kv_heads;
  if (units * kMaxCluster > 0x7fffffff) return PKV_EINVAL;
  unsigned int* err = device_error_ptr();
  if (!err) return cuda_status(cudaGetLastError());
  SelectArgs a = {};
  a.q = static_cast<const __half*>(q);
  a.scales = kv_scales;
  a.bounds = static_cast<const uint8_t*>(k_bounds);
  a.block_tables = block_tables;
  a.context_lens = context_lens;
  a.tables_out = tables_out;
  a.lens_out = lens_out;
  a.err = err;
  a.num_blocks = num_blocks;
  a.max_blocks = max_blocks_per_seq;
  a.q_len = q_len;
  a.Hq = num_q_heads;
  a.Hkv = num_kv_heads;
  a.G = G;
  a.R = G * q_len;
  a.block_size = block_size;
  while ((1 << a.bs_shift) < block_size) ++a.bs_shift;
  a.budget = budget;
  a.keep_first = keep_first;
  a.keep_last = keep_last;
  a.C = cluster_for(units, max_blocks_per_seq);
  if (max_blocks_per_seq > a.C * 32768) a.C = kMaxCluster;
  a.cap = ((max_blocks_per_seq + a.C - 1) / a.C + 15) & ~15;
  const void* fn = kernel_for(a.R);
  const int nt = (a.R + 7) / 8;
  const size_t smem = static_cast<size_t>(nt) * (4096 + 8 * 16) + 4096 + (a.cap + 256) * 4;
  const cudaError_t e = allow_smem(fn);
  if (e != cudaSuccess) return cuda_status(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * a.C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = a.C;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.C > 1 ? 2 : 1;
  void* params[1] = {&a};
  return cuda_status(cudaLaunchKernelExC(&cfg, fn, params));
}
