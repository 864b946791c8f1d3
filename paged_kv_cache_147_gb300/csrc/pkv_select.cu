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
// per (sequence, kv head): its CTAs share the blocks and keep their scores in shared memory as
// ordered integers. The budget's smallest score is found by counting the scores in up to 1024 equal
// intervals between the least and the greatest, the CTAs' counts added up through distributed
// shared memory; the few scores in the interval where the budget ends are compared with each other
// one by one (more of them: counted again in finer intervals). One launch, no workspace.
// Measured: 256 heads of 1024 blocks 19.2 us (67 MB of bounds at 3.5 TB/s: a gather of 256-byte pieces
// behind a table; its start and the choice, about 5 us, are not hidden), 8 heads of 2048 blocks 8.2,
// 128 heads of up to 128 blocks 4.9, with 16 rows of 512 to 1024 blocks 12.9 (above 8 rows no next
// bounds are on their way while a tile is scored).
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "pkv_decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_int8.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;   // as many as rows in a tile of queries
constexpr int kMaxCluster = 8;
constexpr int kGather = 16384;    // blocks whose keys a CTA takes all of
constexpr int kBinBits = 10, kBins = 1 << kBinBits;   // 4 a thread
constexpr int kCands = kThreads;
constexpr uint32_t kAlways = 0xffffffffu;     // key of a block that is kept whatever its score
constexpr uint32_t kNanKey = 0xfffffffeu;     // a NaN scale: before every number
constexpr uint32_t kUnknownKey = 1u;          // an id outside the pool: behind every number (0: not chosen)

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

__device__ __forceinline__ uint4 ld_cluster_v4(const uint32_t* p, uint32_t rank) {
  uint32_t remote;
  uint4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(remote) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(const uint64_t* p, uint32_t rank) {
  uint32_t remote;
  uint64_t v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(remote) : "memory");
  return v;
}

// Larger numbers have larger keys; -0 does not come here.
__device__ __forceinline__ uint32_t key_of(float s) {
  const uint32_t b = __float_as_uint(s);
  return s == s ? b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u) : kNanKey;
}

// Exclusive scan of one value per thread.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i)
    if (i < warp) before += sh[i];
  return before + incl - v;
}

// CTAs of an SM that the registers are shared out for.
constexpr int kCtas = 2;

// NT: tiles of 8 query rows.
template <int NT>
__global__ void __launch_bounds__(kThreads, kCtas)
select_blocks_kernel(const SelectArgs a) {
  griddep_wait();
  extern __shared__ __align__(16) uint8_t smem[];
  uint2* frag = reinterpret_cast<uint2*>(smem);                   // [NT][16][32]
  float4* col = reinterpret_cast<float4*>(frag + NT * 512);       // [8 NT] offset, factor, bias, -
  uint32_t* hist = reinterpret_cast<uint32_t*>(col + 8 * NT);     // [2][kBins], taken in turn
  uint32_t* keys = hist + 2 * kBins;                              // [cap]
  __shared__ uint64_t cand_s[kCands];        // this CTA's scores in the interval where the budget ends
  __shared__ uint64_t all_s[kCands];         // the cluster's
  __shared__ uint32_t scan_s[4 * kWarps], found_s[3];
  __shared__ uint32_t ends_s[2], taken_s[2], ncand_s;

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
  // entries without a block, and all of a context within the budget (which may be any int)
  for (int64_t i = rank * kThreads + tid; i < a.budget; i += a.C * kThreads) {
    if (i >= n) out[i] = -1;
    else if (nblk == n) out[i] = table[i];
  }
  if (nblk == n) return;
  // A context whose keys all fit in a CTA's shared memory: every CTA copies the others' there and
  // goes on as if it were alone, but for the blocks it writes out.
  const bool gather = a.C > 1 && a.cap >= a.max_blocks;
  const bool joint = a.C > 1 && !gather;   // the CTAs keep their own keys and add up their counts
  auto everyone = [&]() {   // a barrier of those that work together
    if (joint) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  };
  auto theirs = [&](const uint32_t* p, int c) { return joint ? ld_cluster_u32(p, c) : *p; };

  // ---- this CTA's blocks: their ids on the way ----
  const int per = ((nblk + a.C - 1) / a.C + 15) & ~15;
  const int from = min(nblk, static_cast<int>(rank) * per), to = min(nblk, from + per);
  uint32_t* own = keys + (gather ? from : 0);
  // blocks before `head` and from `tail` on are kept
  const int head = a.keep_first;
  const int tail = nblk - max(a.keep_last, nblk - (max(ctx - a.q_len, 0) >> a.bs_shift));
  auto id_of = [&](int j) { return j < to ? table[j] : -1; };
  constexpr int kStep = 16 * kWarps;
  int j0 = from + 16 * warp;
  int next[2] = {id_of(j0 + g), id_of(j0 + g + 8)};   // ids of the warp's next 16 blocks

  // ---- the queries: whole numbers as the products' B operands ----
  for (int i = tid; i < 2 * kBins; i += kThreads) hist[i] = 0u;
  if (tid == 0) {
    ends_s[0] = 0xffffffffu;
    ends_s[1] = 0u;
    ncand_s = 0u;
  }
  // (a warp has row `warp` of each tile; all of its loads go out first)
  uint2 qv[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + warp, qi = r / a.G;
    qv[nt] = make_uint2(0u, 0u);
    if (r < a.R && ctx - a.q_len + qi >= 0)
      qv[nt] = reinterpret_cast<const uint2*>(
          a.q + ((static_cast<int64_t>(b) * a.q_len + qi) * a.Hq + h * a.G + r - qi * a.G) * kD)[lane];
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = 8 * nt + warp;
    const bool sees = r < a.R && ctx - a.q_len + r / a.G >= 0;
    const uint2 v = qv[nt];
    const __half2 x = *reinterpret_cast<const __half2*>(&v.x);
    const __half2 y = *reinterpret_cast<const __half2*>(&v.y);
    __half2 big = __hmax2_nan(__habs2(x), __habs2(y));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, o));
    const float s = int8_scale(__half2float(__hmax_nan(__low2half(big), __high2half(big))));
    const float inv = int8_inverse(s);
    const float2 fx = __half22float2(x), fy = __half22float2(y);
    float p[4] = {fx.x, fx.y, fy.x, fy.y};
    int sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // (a row with a NaN or an infinity counts for nothing)
      p[i] = s == s ? fminf(fmaxf(rintf(p[i] * inv), -127.f), 127.f) : 0.f;
      sum += static_cast<int>(p[i]);
    }
    sum = __reduce_add_sync(0xffffffffu, sum);
    // dims 4 lane .. + 3: word `lane & 3` of 16-byte piece (lane >> 2) & 3 of 64-byte part lane >> 4
    uint2* at = frag + nt * 512 + ((lane >> 4) * 4 + (lane & 3)) * 32 + warp * 4 + ((lane >> 2) & 3);
    at[0] = make_uint2(pack_half2(fminf(p[0], 0.f), fminf(p[2], 0.f)),
                       pack_half2(fminf(p[1], 0.f), fminf(p[3], 0.f)));
    at[8 * 32] = make_uint2(pack_half2(fmaxf(p[0], 0.f), fmaxf(p[2], 0.f)),
                            pack_half2(fmaxf(p[1], 0.f), fmaxf(p[3], 0.f)));
    if (lane == 0) {
      const bool counts = sees && s == s;
      col[r] = make_float4(static_cast<float>(sum) * -0x1p-17f, counts ? 0x1p24f * s : 0.f,
                           counts ? 0.f : kNegInf, 0.f);
    }
  }
  __syncthreads();

  // ---- scores, 16 blocks a warp at a time ----
  uint32_t least = 0xffffffffu, most = 0u;
  struct Tile {
    uint4 w[2][4];
    float sc[2];
    bool good[2];
  };
  auto fetch = [&](Tile& t, int j0) {
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      const int id = next[o];
      t.good[o] = id >= 0 && id < a.num_blocks;
      const int64_t bh = static_cast<int64_t>(t.good[o] ? id : 0) * a.Hkv + h;
      const uint4* src = reinterpret_cast<const uint4*>(a.bounds + bh * 256) + t4;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.w[o][i] = t.good[o] ? src[4 * i] : make_uint4(0, 0, 0, 0);
      t.sc[o] = t.good[o] ? a.scales[bh * 2] : 0.f;
      if (!t.good[o] && j0 + g + 8 * o < to && t4 == 0) atomicOr(a.err, PKV_DEVERR_BLOCK_ID);
      next[o] = id_of(j0 + kStep + g + 8 * o);
    }
  };
  auto score = [&](const Tile& t, int j0) {
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      acc[nt][0] = acc[nt][2] = col[8 * nt + 2 * t4].x;
      acc[nt][1] = acc[nt][3] = col[8 * nt + 2 * t4 + 1].x;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t u0 = u4_word(t.w[0][i], e), u1 = u4_word(t.w[1][i], e);
        const uint32_t l0 = u0 & 0x00ff00ffu, l1 = u1 & 0x00ff00ffu;
        const uint32_t h0 = __byte_perm(u0, 0u, 0x4341), h1 = __byte_perm(u1, 0u, 0x4341);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 f = frag[nt * 512 + (4 * i + e) * 32 + lane];
          mma_f16(acc[nt], l0, l1, h0, h1, f.x, f.y);
        }
      }
    float best[2] = {kNegInf, kNegInf};
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float4 c0 = col[8 * nt + 2 * t4], c1 = col[8 * nt + 2 * t4 + 1];
#pragma unroll
      for (int o = 0; o < 2; ++o)
        best[o] = fmaxf(best[o], fmaxf(fmaf(acc[nt][2 * o], c0.y, c0.z),
                                       fmaf(acc[nt][2 * o + 1], c1.y, c1.z)));
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      best[o] = fmaxf(best[o], __shfl_xor_sync(0xffffffffu, best[o], 1));
      best[o] = fmaxf(best[o], __shfl_xor_sync(0xffffffffu, best[o], 2));
      const int j = j0 + g + 8 * o;
      if (t4 == 0 && j < to) {
        // (+ 0 turns -0 into 0; a scale of 0 must not meet -infinity, which a NaN one outranks)
        float s = best[o] * t.sc[o] + 0.f;
        if (best[o] == kNegInf && t.sc[o] == t.sc[o]) s = kNegInf;
        const uint32_t key = j < head || j >= tail ? kAlways : t.good[o] ? key_of(s) : kUnknownKey;
        if (key != kAlways) {
          least = min(least, key);
          most = max(most, key);
        }
        own[j - from] = key;
      }
    }
  };
  if constexpr (NT == 1) {
    // the next 16 blocks' bounds on the way (more rows leave no registers for that)
    Tile t[2];
    if (j0 < to) fetch(t[0], j0);
    while (j0 < to) {
      if (j0 + kStep < to) fetch(t[1], j0 + kStep);
      score(t[0], j0);
      j0 += kStep;
      if (j0 >= to) break;
      if (j0 + kStep < to) fetch(t[0], j0 + kStep);
      score(t[1], j0);
      j0 += kStep;
    }
  } else {
#pragma unroll 1
    for (; j0 < to; j0 += kStep) {
      Tile t;
      fetch(t, j0);
      score(t, j0);
    }
  }
  if (gather) {
    cluster_arrive();
    cluster_wait();
    // four keys a load (`per` is a multiple of 16), four loads in flight
    constexpr int kPass = 4 * kThreads;
    for (int j0 = 4 * tid; j0 < nblk; j0 += 4 * kPass) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kPass;
        if (j < nblk) v[i] = ld_cluster_v4(keys + j, j / per);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = j0 + i * kPass;
        if (j >= nblk || (j >= from && j < to)) continue;
        *reinterpret_cast<uint4*>(keys + j) = v[i];
        const uint32_t vw[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (j + e < nblk && vw[e] != kAlways) {
            least = min(least, vw[e]);
            most = max(most, vw[e]);
          }
      }
    }
    cluster_arrive();   // this CTA has read the others' keys
  }
  bool copying = gather;   // the others may still be reading this CTA's
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0 && least <= most) {
    atomicMin(&ends_s[0], least);
    atomicMax(&ends_s[1], most);
  }
  everyone();
  {
    // (lane c: CTA c's; a CTA without such blocks has the neutral ends)
    const bool there = lane < (joint ? a.C : 1);
    least = __reduce_min_sync(0xffffffffu, there ? theirs(&ends_s[0], lane) : 0xffffffffu);
    most = __reduce_max_sync(0xffffffffu, there ? theirs(&ends_s[1], lane) : 0u);
  }
  // the keys this CTA looks through from here on: `count` of them, of blocks `lo` on
  const int lo = joint ? from : 0, count = joint ? to - from : nblk;

  // ---- where the budget ends: keys above `edge` are taken, and the first `need` equal to it ----
  uint32_t need = n - min(head, nblk) - (nblk - tail);
  uint32_t edge = kAlways - 1;     // (nothing but the kept ones)
  for (int round = 0; need > 0 && round < 4; ++round) {   // (32 bits, 10 a round)
    const int shift = max(0, 32 - __clz(most - least) - kBinBits);
    uint32_t* hr = hist + (round & 1) * kBins;
#pragma unroll 4
    for (int j = tid; j < count; j += kThreads) {
      const uint32_t key = keys[j];
      if (key >= least && key <= most) atomicAdd(hr + ((key - least) >> shift), 1u);
    }
    everyone();
    // four bins a thread, the greatest first
    const int b0 = kBins - 4 - 4 * tid;
    uint32_t in[4] = {0u, 0u, 0u, 0u};
    if (joint) {
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (c >= a.C) break;
        const uint4 v = ld_cluster_v4(hr + b0, c);
        in[0] += v.w; in[1] += v.z; in[2] += v.y; in[3] += v.x;
      }
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(hr + b0);
      in[0] = v.w; in[1] = v.z; in[2] = v.y; in[3] = v.x;
    }
    uint32_t above = block_scan(in[0] + in[1] + in[2] + in[3], scan_s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (above < need && need <= above + in[i]) {
        found_s[0] = b0 + 3 - i;
        found_s[1] = need - above;
        found_s[2] = in[i];
      }
      above += in[i];
    }
    // the other counters are ready for the next round (no one reads them: this round's barrier is
    // behind everyone's last use)
    for (int i = tid; i < kBins; i += kThreads) hist[((round + 1) & 1) * kBins + i] = 0u;
    __syncthreads();
    const uint32_t bottom = least + (found_s[0] << shift);
    most = bottom + min((1u << shift) - 1u, most - bottom);
    least = bottom;
    need = found_s[1];
    const uint32_t inside = found_s[2];
    edge = most;
    if (shift == 0) break;
    if (inside == need) {          // all of the interval
      edge = least - 1;
      need = 0;
    } else if (inside <= kCands) {
      // ---- few: each is compared with all, the lower block first among equal ones ----
      for (int j = tid; j < count; j += kThreads) {
        const uint32_t key = keys[j];
        if (key >= least && key <= most)
          cand_s[atomicAdd(&ncand_s, 1u)] =
              static_cast<uint64_t>(key) << 32 | (0xffffffffu - static_cast<uint32_t>(lo + j));
      }
      everyone();
      uint64_t x = 0;
      uint32_t c = rank;
      if (joint) {
        // (lane c: how many CTA c has; they come one CTA's behind the other's)
        uint32_t end = lane < a.C ? ld_cluster_u32(&ncand_s, lane) : 0u, first = 0;
#pragma unroll
        for (int o = 1; o < kMaxCluster; o <<= 1) {
          const uint32_t y = __shfl_up_sync(0xffffffffu, end, o);
          if (lane >= o) end += y;
        }
        c = 0;
#pragma unroll
        for (int i = 0; i < kMaxCluster; ++i) {
          const uint32_t e = __shfl_sync(0xffffffffu, end, i);
          if (i < a.C && static_cast<uint32_t>(tid) >= e) {
            first = e;
            c = i + 1;
          }
        }
        if (static_cast<uint32_t>(tid) < inside) x = ld_cluster_u64(cand_s + (tid - first), c);
      } else if (static_cast<uint32_t>(tid) < inside) {
        x = cand_s[tid];
      }
      all_s[tid] = x;
      if (copying) {   // (the marks below go into this CTA's own keys, too)
        cluster_wait();
        copying = false;
      }
      __syncthreads();
      if (static_cast<uint32_t>(tid) < inside && c == rank) {
        uint32_t better = 0;
#pragma unroll 8
        for (uint32_t i = 0; i < inside; ++i) better += all_s[i] > x;
        keys[0xffffffffu - static_cast<uint32_t>(x) - lo] = better < need ? kAlways : 0u;
      }
      need = 0;
      __syncthreads();
    }
  }

  // ---- the chosen blocks in their order ----
  // taken blocks and equal keys ahead of this CTA's (gather: counted here)
  uint32_t gt = 0, eq = 0;
  if (gather) {
    for (int j = 4 * tid; j < from; j += 4 * kThreads) {   // (`from` is a multiple of 16)
      const uint4 v = *reinterpret_cast<const uint4*>(keys + j);
      gt += (v.x > edge) + (v.y > edge) + (v.z > edge) + (v.w > edge);
      eq += (v.x == edge) + (v.y == edge) + (v.z == edge) + (v.w == edge);
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
  }
  // a warp takes a run of this CTA's, 32 at a time
  const int cnt = to - from, run = ((cnt + kThreads - 1) / kThreads) * 32;
  const int k0 = min(cnt, warp * run), k1 = min(cnt, k0 + run);
  uint32_t gt_run = 0, eq_run = 0;
  for (int j = k0 + lane; j - lane < k1; j += 32) {
    const uint32_t key = j < k1 ? own[j] : 0u;
    gt_run += __popc(__ballot_sync(0xffffffffu, key > edge));
    eq_run += __popc(__ballot_sync(0xffffffffu, j < k1 && key == edge));
  }
  if (lane == 0) {
    scan_s[warp] = gt_run;
    scan_s[kWarps + warp] = eq_run;
    scan_s[2 * kWarps + warp] = gt;
    scan_s[3 * kWarps + warp] = eq;
  }
  __syncthreads();
  gt = eq = 0;
  gt_run = eq_run = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    gt += scan_s[2 * kWarps + i] + (i < warp ? scan_s[i] : 0u);
    eq += scan_s[3 * kWarps + i] + (i < warp ? scan_s[kWarps + i] : 0u);
    gt_run += scan_s[i];
    eq_run += scan_s[kWarps + i];
  }
  if (joint) {
    if (tid == 0) {
      taken_s[0] = gt_run;
      taken_s[1] = eq_run;
    }
    everyone();
    const bool before = lane < static_cast<int>(rank);
    gt += __reduce_add_sync(0xffffffffu, before ? ld_cluster_u32(&taken_s[0], lane) : 0u);
    eq += __reduce_add_sync(0xffffffffu, before ? ld_cluster_u32(&taken_s[1], lane) : 0u);
    cluster_arrive();   // this CTA has read what the others counted
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int j = k0 + lane; j - lane < k1; j += 32) {
    const uint32_t key = j < k1 ? own[j] : 0u;
    const bool is_eq = j < k1 && key == edge;
    const uint32_t gts = __ballot_sync(0xffffffffu, key > edge);
    const uint32_t eqs = __ballot_sync(0xffffffffu, is_eq);
    const uint32_t e = eq + __popc(eqs & below);    // equal ones before this
    if (key > edge || (is_eq && e < need))
      out[gt + __popc(gts & below) + min(e, need)] = table[from + j];
    gt += __popc(gts);
    eq += __popc(eqs);
  }
  if (joint || copying) cluster_wait();   // the others have read this CTA's
}

// ---------------------------------------------------------------------------------------------
// Host side.

const void* kernel_for(int R) {
  return R <= 8    ? reinterpret_cast<const void*>(&select_blocks_kernel<1>)
         : R <= 16 ? reinterpret_cast<const void*>(&select_blocks_kernel<2>)
         : R <= 24 ? reinterpret_cast<const void*>(&select_blocks_kernel<3>)
                   : reinterpret_cast<const void*>(&select_blocks_kernel<4>);
}

// CTAs per cluster: as many as are resident at once, with at least kMinBlocks columns of the table each
// (the lengths are on the GPU), where the table has room for contexts that are worth it: a cluster costs
// 1 us more than a CTA alone, its barriers and the copying of the keys. Measured with 1, 2, 4, 8 CTAs,
// contexts as long as the table, us:
//   8 heads     of 128 blocks 4.9, 5.7, 5.7, 5.8   of 256 6.1, 6.3, 5.9, 5.9   of 384 7.3, 7.0, 6.2, 6.1
//               of 1024 12.4, 9.9, 7.7, 6.8        of 2048 19.5, 14.0, 10.3, 8.3
//   64 heads    of 128 blocks 5.1, 6.2, 6.2        of 384 7.5, 7.2, 6.9        of 1024 12.7, 10.1, 8.9
//   128 heads   of 128 blocks 5.1, 6.5             of 512 8.7, 8.8             of 1024 15.1, 13.1
//   (16 rows)                 5.2, 6.7                    8.8, 9.3                     16.8, 14.4
constexpr int kMinBlocks = 64;
constexpr int kWide = 384, kWidePair = 768;   // columns from which on a cluster, and one of two, pays
int cluster_for(int64_t units, int max_blocks) {
  int c = 1;
  while (c < kMaxCluster && units * 2 * c <= static_cast<int64_t>(kCtas) * sm_count() &&
         max_blocks >= 2 * c * kMinBlocks)
    c *= 2;
  return max_blocks >= (c > 2 ? kWide : kWidePair) ? c : 1;
}

// Raises the limit of dynamic shared memory of the kernel for `nt` tiles to the device's, once per
// device (of the first 64; two threads at once both do it).
cudaError_t allow_smem(const void* fn, int nt) {
  static std::atomic<unsigned> done[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && (done[dev].load(std::memory_order_acquire) >> nt & 1u)) return cudaSuccess;
  int limit = 0;
  e = cudaDeviceGetAttribute(&limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  cudaFuncAttributes fa;
  if (e == cudaSuccess) e = cudaFuncGetAttributes(&fa, fn);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             limit - static_cast<int>(fa.sharedSizeBytes));
  if (e == cudaSuccess && dev < 64) done[dev].fetch_or(1u << nt, std::memory_order_release);
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
      num_blocks < 1 || max_blocks_per_seq < 0 || max_blocks_per_seq > 8 * 32768 ||
      budget < 1 || keep_first < 0 || keep_last < 0)
    return PKV_EINVAL;
  const int G = num_q_heads / num_kv_heads;
  if (static_cast<int64_t>(G) * q_len > 32) return PKV_EINVAL;
  const int ends = std::max(keep_last, 1 + (q_len - 1 + block_size - 1) / block_size);
  if (static_cast<int64_t>(keep_first) + ends > budget) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (!tables_out || !lens_out || !q || !kv_scales || !k_bounds || !context_lens ||
      (!block_tables && max_blocks_per_seq > 0))   // (a table without columns has no address)
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
  const int nt = (a.R + 7) / 8;
  a.C = cluster_for(units, max_blocks_per_seq);
  // (what shared memory has room for)
  while (max_blocks_per_seq > a.C * 32768) a.C *= 2;
  const int share = max_blocks_per_seq <= kGather ? 1 : a.C;
  a.cap = ((max_blocks_per_seq + share - 1) / share + 15) & ~15;
  const void* fn = kernel_for(a.R);
  const size_t smem = static_cast<size_t>(nt) * (4096 + 8 * 16) + (2 * kBins + a.cap) * 4;
  const cudaError_t e = allow_smem(fn, nt);
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
