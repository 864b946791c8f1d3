// pkv_decode_int4.cu -- paged decode attention over a 4-bit cache (pkv_int4.cuh's rows) for
// sm_103a.
//
// What it computes: pkv_paged_attn_decode's operation with K_t[d] = s_K code_K + z_K and
// V_t[d] = s_V code_V + z_V, (s, z) of the 32 elements that d belongs to.
//
// What bounds it: 160 bytes per (token, kv head) against 512 of the fp16 cache, so the widening of
// the codes, not the loads, is what the loop has to keep short. It is written so that a step of
// 16 keys takes a warp about 300 issue slots for up to 8 query rows:
//  * Stream, slices, split units and their merge are those of pkv_decode.cu (shared in
//    pkv_decode_common.cuh). A stage holds two 16-token chunks: K of both, V of both, four boxes
//    of 16 rows x 80 bytes (rows 20 words apart: any 8 rows x 4 words touch all 32 banks, so
//    the tiles need no swizzle).
//  * Transposed tile: S^T = K Q^T and O^T = V^T P^T on mma.sync m16n8k16, keys (and output dims)
//    on the 16-row side, query rows in NT tiles of 8 columns. A code is widened once for all NT.
//  * Keys: sum_d q_d (s c_d + z) = s sum_d q_d c_d + z sum_d q_d per group of 32 dims. The codes
//    go to the tensor cores as they stand: four bits at bits 4-7 of a 16-bit half are the fp16
//    (subnormal) number c 2^-20, exactly, and one AND of a shifted word makes two of them. The
//    group's two products (32 dims) are scaled by s in fp32; 2^20 joins the score scale. z times
//    the group's query sum is one more product per 16 keys: a row's four (s, z) pairs as they
//    stand against (0, mean of q over the group), the mean split in two fp16 numbers (it is
//    held as sum / 32 so that no sum of finite fp16 queries overflows).
//  * Values: s varies with the key, the summed dimension, so V is widened: pairs of neighbouring
//    keys' codes by byte permutes, code = (1024 + code) - 1024 in fp16, then s code + z by one
//    fused multiply-add: rounded once to fp16 (2^-12 relative, as a cached fp16 V would be).
//    A thread's 16 output dims lie in one group, so it needs one (s, z) pair per key.
//  * Softmax as in pkv_decode.cu (fp32, exp2 domain, lazy running maximum); weights in fp16.
//  * Tokens past the context hold anything: their scores are masked and their (s, z) of V set
//    to zero before the widening.
#include <cuda_fp16.h>

#include "pkv_decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_int4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kTile = kChunk * kInt4Row;     // one chunk's K (or V): 1280 bytes
constexpr int kStage4 = 4 * kTile;           // K of two chunks, V of two chunks
constexpr int kSeg4 = 4;                     // per-segment cost in chunks (see kSegCost)

// Shared-memory layout (offsets from a 1024-byte aligned base); the names are those the shared
// helpers use.
template <int NCW, int NST, int NT>
struct Smem4 {
  static constexpr int kNST = NST;
  static constexpr int kQHalf = NT * 1024;            // 8 NT rows x 128 B
  static constexpr int kQBuf = 2 * kQHalf;
  static constexpr int kQ = NST * kStage4;
  static constexpr int kBars = kQ + 2 * kQBuf;        // full, empty, qfull, qempty, sdone, sfree
  static constexpr int kFlags = kBars + (2 * NST + 8) * 8;
  static constexpr int kSrow = kFlags + 64;           // TMA rows of each stage's two chunks
  static constexpr int kState = kSrow + ((NST * 8 + 15) & ~15);
  __host__ __device__ static int state_floats(int R) { return 2 * NCW * R * (kSt + 2); }
  __host__ __device__ static int seq_off(int R) { return kState + state_floats(R) * 4; }
  __host__ __device__ static int newkv_off(int R, int B) {
    return (seq_off(R) + (2 * B + 1) * 4 + 127) & ~127;
  }
  __host__ static size_t bytes(int R, int B, int newkv_bytes) {
    return 1024 + static_cast<size_t>(newkv_off(R, B)) + static_cast<size_t>(newkv_bytes);
  }
  static_assert(kStage4 % 1024 == 0 && kQHalf % 1024 == 0, "swizzle atoms of the query tiles");
  // the merge of split units stages at least two partials in the stage memory
  static_assert(kQ >= 8 * NT * ((kD + 8) * 4 + 2 * (kD + 4) * 4), "merge staging");
};

// (x & m), the four bits of each half at bits 4-7: c 2^-20 as fp16.
__device__ __forceinline__ uint32_t nibs(uint32_t x) { return x & 0x00f000f0u; }

// Warp roles as in decode_kernel: warps 0..NCW-1 consume stages, warp NCW produces, warp NCW+1 is
// the epilogue.
template <int NCW, int NST, int NT, int MINB, bool APPEND>
__global__ void __launch_bounds__((NCW + 2) * 32, MINB)
decode_int4_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                   const __grid_constant__ CUtensorMap tmQ, const DecodeArgs a) {
  using L = Smem4<NCW, NST, NT>;
  static_assert(NST % NCW == 0, "pipeline stages must be a multiple of the consumer warps");
  // more than two row tiles: the query fragments do not fit the registers and are read from the
  // (permuted) query tile, which then stays in use for the whole segment
  constexpr bool kQSmem = NT > 2;
  constexpr bool kHoldQ = APPEND || kQSmem;
  constexpr int kNC = NCW * 32;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_full = sbase + L::kBars;
  const uint32_t bar_empty = bar_full + NST * 8;
  const uint32_t bar_qfull = bar_empty + NST * 8;
  const uint32_t bar_qempty = bar_qfull + 2 * 8;
  const uint32_t bar_sdone = bar_qempty + 2 * 8;
  const uint32_t bar_sfree = bar_sdone + 2 * 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kFlags);
  int* srow_s = reinterpret_cast<int*>(smem + L::kSrow);
  int* npend_s = reinterpret_cast<int*>(smem + L::kFlags) + 1;   // then 2 x (b, h, nb)
  volatile int* fast_s = reinterpret_cast<volatile int*>(smem + L::kFlags) + 8;
  float* stO = reinterpret_cast<float*>(smem + L::kState);       // [2][NCW][R][kSt]
  float* stM = stO + 2 * NCW * a.R * kSt;                         // [2][NCW][R]
  float* stL = stM + 2 * NCW * a.R;                               // [2][NCW][R]
  int* pre = reinterpret_cast<int*>(smem + L::seq_off(a.R));
  int* slen = pre + a.num_seqs + 1;

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int B = a.num_seqs;

  // ---- per-sequence lengths and chunk counts -------------------------------------------------
  for (int b = tid; b < B; b += blockDim.x) {
    int ctx = a.context_lens[b];
    const int lim = a.max_blocks * a.block_size;
    if (ctx < 0 || ctx > lim) {
      atomicOr(a.err, PKV_DEVERR_CONTEXT);
      ctx = ctx < 0 ? 0 : lim;
    }
    const int nchunks = (ctx + kChunk - 1) / kChunk;
    slen[b] = ctx;
    pre[b + 1] = nchunks > 0 ? nchunks + kSeg4 : 0;
  }
  // zero both Q buffers so rows past R are finite; TMA overwrites rows < R
  for (int i = tid; i < L::kQBuf * 2 / 16; i += blockDim.x)
    reinterpret_cast<uint4*>(smem + L::kQ)[i] = make_uint4(0, 0, 0, 0);
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(bar_full + s * 8, 1);
      mbar_init(bar_empty + s * 8, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_qfull + s * 8, 1);
      mbar_init(bar_qempty + s * 8, NCW);
      mbar_init(bar_sdone + s * 8, NCW);
      mbar_init(bar_sfree + s * 8, 1);
    }
    *abort = 0;
    *npend_s = 0;
    pre[0] = 0;
  }
  fence_barrier_init();
  __syncthreads();
  if (warp == 0) scan_chunks(pre, B, lane);
  __syncthreads();

  const int total = pre[B] * a.Hkv;
  const int per = (total + gridDim.x - 1) / gridDim.x;
  const int begin = blockIdx.x * per;
  const CursorT<kSeg4> cur{pre, B, a.Hkv, min(total, begin + per)};

  // let the next kernel on the stream launch as SM resources free up (it waits for this one
  // before it reads anything this kernel writes)
  if (tid == 0) griddep_launch_dependents();

  if (warp == NCW) {
    // =================================== producer ============================================
    const int chunk_mask = (1 << a.bs_shift) - 1;
    const uint64_t kv_policy = l2_policy_evict_first();
    int j = 0, k = 0;
    Seg s;
    bool has = cur.first(begin, s);
    auto load_ids = [&](const Seg& sg, int cb) -> int32_t {
      const int cc = cb + lane;
      return cc < sg.c1 ? __ldg(a.block_tables + static_cast<int64_t>(sg.b) * a.max_blocks +
                                (cc >> a.bs_shift))
                        : -1;
    };
    int32_t ids = has ? load_ids(s, s.c0) : -1;
    if (lane == 0) {
      prefetch_tensormap(&tmK);
      prefetch_tensormap(&tmV);
      prefetch_tensormap(&tmQ);
    }
    // An early-started launch (APPEND) requests its first stages at once and waits for the
    // preceding kernel before the queries; the epilogue warp requests the first segment's.
    bool waited = false;
    while (has) {
      if (!APPEND || k > 0) {
        if (!waited) { griddep_wait(); waited = true; }
        if (lane == 0) issue_queries<L, APPEND>(a, &tmQ, sbase, B, s, k, abort);
      }
      Seg nx = s;
      const bool has_next = cur.next(nx);
      for (int cb = s.c0; cb < s.c1; cb += 32) {
        const int32_t cur_ids = ids;
        if (cb + 32 < s.c1) ids = load_ids(s, cb + 32);
        else if (has_next) ids = load_ids(nx, nx.c0);
        const int cc = cb + lane;
        int row = -kChunk;  // an out-of-range box: TMA fills it with zeros
        if (cc < s.c1) {
          if (cur_ids >= 0 && cur_ids < a.num_blocks)
            row = (cur_ids * a.Hkv + s.h) * a.block_size + ((cc & chunk_mask) << 4);
          else
            atomicOr(a.err, PKV_DEVERR_BLOCK_ID);
        }
        const int n = min(32, s.c1 - cb);
        for (int l = 0; l < n; l += 2, ++j) {
          if (APPEND && !waited && j == NST) {
            griddep_wait();   // every stage is requested; none frees before the dependency is met
            waited = true;
          }
          const int r = __shfl_sync(0xffffffffu, row, l);
          const int r2 = __shfl_sync(0xffffffffu, row, (l + 1) & 31);   // l + 1 < n, or out of range
          const int st = j % NST;
          const uint32_t fb = bar_full + st * 8;
          if (lane == 0) {
            if (j >= NST && !mbar_wait(bar_empty + st * 8, ((j / NST) - 1) & 1, abort))
              flag_timeout(a, abort);
            if (APPEND) {
              srow_s[2 * st] = r;
              srow_s[2 * st + 1] = r2;
            }
            mbar_arrive_expect_tx(fb, kStage4);
          }
          __syncwarp();
          if (lane < 4)
            tma_load_2d_hint(sbase + st * kStage4 + lane * kTile, (lane >> 1) ? &tmV : &tmK, 0,
                             (lane & 1) ? r2 : r, fb, kv_policy);
        }
      }
      ++k;
      s = nx;
      has = has_next;
    }
    if (!waited) griddep_wait();
    // sequences without any chunk get zeros (their units are in no CTA's slice)
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      if (pre[b + 1] != pre[b]) continue;
      const int n = a.q_len * a.Hq * kD;
      for (int i = lane; i < n; i += 32)
        a.out[static_cast<int64_t>(b) * n + i] = __float2half_rn(0.f);
    }
    // no TMA write into this CTA's shared memory may be pending when it exits
    if (lane == 0) {
      for (int jj = max(0, j - NST); jj < j; ++jj)
        if (!mbar_wait(bar_full + (jj % NST) * 8, (jj / NST) & 1, nullptr)) flag_timeout(a, abort);
      for (int kk = max(0, k - 2); kk < k; ++kk)
        if (!mbar_wait(bar_qfull + (kk & 1) * 8, (kk >> 1) & 1, nullptr)) flag_timeout(a, abort);
    }
    return;
  }

  const LastSeg last = LastSeg::of(cur, begin);

  if (warp == NCW + 1) {
    // =================================== epilogue ============================================
    int k = 0, npend = 0;
    Seg s;
    bool has = cur.first(begin, s);
    if (APPEND && has) {
      griddep_wait();
      if (lane == 0) issue_queries<L, APPEND>(a, &tmQ, sbase, B, s, 0, abort);
    }
    while (has && k < last.k) {
      const int sb = k & 1;
      if (!mbar_wait(bar_sdone + sb * 8, (k >> 1) & 1, abort)) flag_timeout(a, abort);
      const bool complete = (s.c0 == 0 && s.c1 == s.nb);
      const int slot = 2 * blockIdx.x + (k == 0 ? 0 : 1);
      merge_segment<NCW, 32>(a, stO + sb * NCW * a.R * kSt, stM + sb * NCW * a.R,
                             stL + sb * NCW * a.R, s.b, s.h, complete,
                             a.part_o + static_cast<int64_t>(slot) * a.R * kD,
                             a.part_ml + static_cast<int64_t>(slot) * a.R * 4, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sfree + sb * 8);
      if (!complete && lane == 0) {
        // announce the partial (release) and see who else has arrived (acquire)
        const int ua = unit_first<kSeg4>(pre, a.Hkv, s.b, s.h, s.nb);
        const int parts = (ua + s.nb - 1) / per - ua / per + 1;
        if (atomic_add_acq_rel(a.counters + s.b * a.Hkv + s.h, 1) == parts - 1) {
          npend_s[1 + 3 * npend] = s.b;
          npend_s[2 + 3 * npend] = s.h;
          npend_s[3 + 3 * npend] = s.nb;
          ++npend;
        }
      }
      ++k;
      has = cur.next(s);
    }
    if (lane == 0) *npend_s = npend;
  } else {
    // =================================== consumers ===========================================
    const int w = warp;
    const int g = lane >> 2, t4 = lane & 3;
    const float score_l2 = a.scale_log2 * 1048576.f;   // the codes come in as c 2^-20
    int j = 0, k = 0;
    Seg s;
    bool has = cur.first(begin, s);
    while (has) {
      const int qs = k & 1;
      const uint32_t qb = sbase + L::kQ + qs * L::kQBuf;
      if (!mbar_wait(bar_qfull + qs * 8, (k >> 1) & 1, abort)) flag_timeout(a, abort);
      const int Lc = slen[s.b];

      // ---- Q^T fragments (B operands): thread (g, t4) holds row g of each tile and, of group
      // gr, dims d0 = 32 gr + 8 t4 .. d0 + 7, paired as the codes of a word come out of the
      // masks: (d0 + i, d0 + i + 4) for i = 0 .. 3. And the group means, for the minima: t4's
      // group, as two fp16 numbers in the upper halves (the lower ones meet the scales). ----
      uint32_t qf[kQSmem ? 1 : NT][kQSmem ? 1 : 4][4], qzh[NT], qzl[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mean_own = 0.f;
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
          const int ch = 4 * gr + t4;
          const uint4 v = ld_shared_v4(qb + (ch >> 3) * L::kQHalf + swz128(8 * nt + g, ch & 7));
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u = u4_word(v, i);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
            sum += f.x + f.y;
          }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (gr == t4) mean_own = sum * 0.03125f;
          if constexpr (!kQSmem) {
            qf[nt][gr][0] = __byte_perm(v.x, v.z, 0x5410);
            qf[nt][gr][1] = __byte_perm(v.x, v.z, 0x7632);
            qf[nt][gr][2] = __byte_perm(v.y, v.w, 0x5410);
            qf[nt][gr][3] = __byte_perm(v.y, v.w, 0x7632);
          }
        }
        const __half hi = __float2half_rn(mean_own);
        const __half lo = __float2half_rn(mean_own - __half2float(hi));
        qzh[nt] = static_cast<uint32_t>(__half_as_ushort(hi)) << 16;
        qzl[nt] = static_cast<uint32_t>(__half_as_ushort(lo)) << 16;
      }
      if constexpr (kQSmem) {
        // every 16-byte piece of the tile into its fragment order, in place
        named_barrier_sync(1, kNC);                   // all warps have read the plain tile
        for (int i = tid; i < L::kQBuf / 16; i += kNC) {
          const uint4 v = ld_shared_v4(qb + i * 16);
          st_shared_v4(qb + i * 16, make_uint4(__byte_perm(v.x, v.z, 0x5410),
                                               __byte_perm(v.x, v.z, 0x7632),
                                               __byte_perm(v.y, v.w, 0x5410),
                                               __byte_perm(v.y, v.w, 0x7632)));
        }
        named_barrier_sync(1, kNC);
      }
      if (!kHoldQ) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_qempty + qs * 8);
      }

      float tm[NT][2], tl[NT][2], ot[NT][8][4];
      int tlim[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          tm[nt][e] = kNegInf;
          tl[nt][e] = 0.f;
          const int r = 8 * nt + 2 * t4 + e;
          const int qi = r < a.R ? r / a.G : a.q_len - 1;
          tlim[nt][e] = Lc - a.q_len + qi + 1;
        }
#pragma unroll
        for (int dt = 0; dt < 8; ++dt)
          ot[nt][dt][0] = ot[nt][dt][1] = ot[nt][dt][2] = ot[nt][dt][3] = 0.f;
      }

      const int nchunk = s.c1 - s.c0;
      const int npair = (nchunk + 1) >> 1;
      for (int jp = ((w - j) % NCW + NCW) % NCW; jp < npair; jp += NCW) {
        const int gj = j + jp;
        const int st = gj % NST;
        if (!mbar_wait(bar_full + st * 8, (gj / NST) & 1, abort)) flag_timeout(a, abort);
        const uint32_t stK = sbase + st * kStage4;
        const uint32_t stV = stK + 2 * kTile;
        const int c = s.c0 + 2 * jp;
        const bool two = c + 1 < s.c1;
        const int nk = two ? 2 * kChunk : kChunk;
        const bool full = two && (c + 2) * kChunk <= Lc - a.q_len + 1;
        bool patched = false;
        if (APPEND && (c * kChunk + nk > Lc - a.q_len)) {
          // new rows of these chunks: lanes 0-15 quantise the K row, 16-31 the V row, into the
          // stage's tiles and into the pool
          const int first_new = Lc - a.q_len;
          const uint32_t nkv = sbase + L::newkv_off(a.R, B) + qs * a.q_len * 512;
          const int which = lane >> 4, p = lane & 15;
          for (int i = 0; i < a.q_len; ++i) {
            const int pos = first_new + i;
            const int tk = pos - c * kChunk;
            if (pos < 0 || tk < 0 || tk >= nk) continue;
            uint32_t codes, params;
            int4_quantise(ld_shared_v4(nkv + i * 512 + which * 256 + p * 16), codes, params);
            const uint32_t row = stK + which * 2 * kTile + tk * kInt4Row;
            st_shared_u32(row + 4 * p, codes);
            if ((p & 3) == 0) st_shared_u32(row + kInt4Params + p, params);
            const int srow = srow_s[2 * st + (tk >> 4)];
            if (srow >= 0) {
              uint32_t* pool = reinterpret_cast<uint32_t*>(
                  reinterpret_cast<uint8_t*>(which ? a.v_pool : a.k_pool) +
                  (static_cast<int64_t>(srow) + (tk & 15)) * kInt4Row);
              pool[p] = codes;
              if ((p & 3) == 0) pool[(kInt4Params + p) / 4] = params;
            }
          }
          __syncwarp();
          patched = true;
        }

        // ---- S^T = K Q^T, 16 keys at a time ----
        float x[NT][2][2][2];   // [tile][row e][chunk h][key g, g + 8]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t kb0 = stK + h * kTile + g * kInt4Row, kb1 = kb0 + 8 * kInt4Row;
          const uint4 p0 = ld_shared_v4(kb0 + kInt4Params), p1 = ld_shared_v4(kb1 + kInt4Params);
          const uint32_t z0 = ld_shared_u32(kb0 + kInt4Params + 4 * t4);
          const uint32_t z1 = ld_shared_u32(kb1 + kInt4Params + 4 * t4);
          float acc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
            mma_16816(acc[nt], z0, z1, z0, z1, qzh[nt], qzl[nt]);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nt][i] *= 0x1p-15f;   // x 32, in units of 2^-20
          }
#pragma unroll
          for (int gr = 0; gr < 4; ++gr) {
            const uint32_t w0 = ld_shared_u32(kb0 + 16 * gr + 4 * t4);
            const uint32_t w1 = ld_shared_u32(kb1 + 16 * gr + 4 * t4);
            const uint32_t u0 = u4_word(p0, gr), u1 = u4_word(p1, gr);
            const float s0 = __low2float(*reinterpret_cast<const __half2*>(&u0));
            const float s1 = __low2float(*reinterpret_cast<const __half2*>(&u1));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t q0, q1, q2, q3;
              if constexpr (kQSmem) {
                const int ch = 4 * gr + t4;
                const uint4 v =
                    ld_shared_v4(qb + (ch >> 3) * L::kQHalf + swz128(8 * nt + g, ch & 7));
                q0 = v.x; q1 = v.y; q2 = v.z; q3 = v.w;
              } else {
                q0 = qf[nt][gr][0]; q1 = qf[nt][gr][1]; q2 = qf[nt][gr][2]; q3 = qf[nt][gr][3];
              }
              float t[4] = {0.f, 0.f, 0.f, 0.f};
              mma_16816(t, nibs(w0 << 4), nibs(w1 << 4), nibs(w0), nibs(w1), q0, q1);
              mma_16816(t, nibs(w0 >> 4), nibs(w1 >> 4), nibs(w0 >> 8), nibs(w1 >> 8), q2, q3);
              acc[nt][0] = fmaf(s0, t[0], acc[nt][0]);
              acc[nt][1] = fmaf(s0, t[1], acc[nt][1]);
              acc[nt][2] = fmaf(s1, t[2], acc[nt][2]);
              acc[nt][3] = fmaf(s1, t[3], acc[nt][3]);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              x[nt][e][h][0] = acc[nt][e] * score_l2;
              x[nt][e][h][1] = acc[nt][2 + e] * score_l2;
            }
        }

        // ---- mask, online softmax (exp2 domain, lazy running maximum) ----
        uint32_t pb[NT][2][2];   // P^T of chunk h as the B operand
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            if (!full) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int p0 = (c + h) * kChunk + g;
                const int lim = h == 0 || two ? tlim[nt][e] : 0;
                if (p0 >= lim) x[nt][e][h][0] = kNegInf;
                if (p0 + 8 >= lim) x[nt][e][h][1] = kNegInf;
              }
            }
            const float lm = fmaxf(fmaxf(x[nt][e][0][0], x[nt][e][0][1]),
                                   fmaxf(x[nt][e][1][0], x[nt][e][1][1]));
            grow |= lm > tm[nt][e] + kLazyLog2;
          }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(x[nt][e][0][0], x[nt][e][0][1]),
                               fmaxf(x[nt][e][1][0], x[nt][e][1][1]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float m_new = fmaxf(tm[nt][e], mx);
              alpha[e] = fast_exp2(tm[nt][e] - (m_new == kNegInf ? 0.f : m_new));
              tm[nt][e] = m_new;
              tl[nt][e] *= alpha[e];
            }
#pragma unroll
            for (int dt = 0; dt < 8; ++dt) {
              ot[nt][dt][0] *= alpha[0];
              ot[nt][dt][1] *= alpha[1];
              ot[nt][dt][2] *= alpha[0];
              ot[nt][dt][3] *= alpha[1];
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float pv[2][2][2];   // [chunk h][key half][row e]
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float m_use = tm[nt][e] == kNegInf ? 0.f : tm[nt][e];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i) pv[h][i][e] = fast_exp2(x[nt][e][h][i] - m_use);
            tl[nt][e] += (pv[0][0][e] + pv[0][1][e]) + (pv[1][0][e] + pv[1][1][e]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              pb[nt][h][i] = movmatrix_trans(pack_half2(pv[h][i][0], pv[h][i][1]));
        }

        // ---- O^T += V^T P^T. Row g of tile dt is output dim 16 g + dt, row g + 8 dim
        // 16 g + 8 + dt (undone at the hand-off): a thread's operands are its own 8 bytes of
        // keys 2 t4, 2 t4 + 1, 2 t4 + 8 and 2 t4 + 9 ----
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t vb = stV + h * kTile + 2 * t4 * kInt4Row;
          uint2 v[4];
          uint32_t p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t r = vb + ((i & 1) + 8 * (i >> 1)) * kInt4Row;
            v[i] = ld_shared_v2(r + 8 * g);
            p[i] = ld_shared_u32(r + kInt4Params + 4 * (g >> 1));
          }
          uint32_t sc[2], mn[2];   // scales, minima of the two key pairs
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            sc[i] = __byte_perm(p[2 * i], p[2 * i + 1], 0x5410);
            mn[i] = __byte_perm(p[2 * i], p[2 * i + 1], 0x7632);
            if (!full) {   // keys that no query may see may hold anything
              const int t0 = (c + h) * kChunk + 2 * t4 + 8 * i;
              const int lim = h == 0 || two ? Lc : 0;
              const uint32_t m = (t0 < lim ? 0x0000ffffu : 0u) | (t0 + 1 < lim ? 0xffff0000u : 0u);
              sc[i] &= m;
              mn[i] &= m;
            }
          }
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t sel = hf ? 0x7632u : 0x5410u;
            uint32_t u[2][2];   // [word][key pair]: four codes of each of the pair's keys
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              u[0][i] = __byte_perm(v[2 * i].x, v[2 * i + 1].x, sel);
              u[1][i] = __byte_perm(v[2 * i].y, v[2 * i + 1].y, sel);
            }
#pragma unroll
            for (int jn = 0; jn < 4; ++jn) {
              uint32_t f[2][2];
#pragma unroll
              for (int wd = 0; wd < 2; ++wd)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t y = jn < 2 ? u[wd][i] : u[wd][i] >> 8;
                  const __half2 code = (jn & 1) ? int4_hi(y) : int4_lo(y);
                  f[wd][i] = half2_bits(__hfma2(code, *reinterpret_cast<const __half2*>(&sc[i]),
                                                *reinterpret_cast<const __half2*>(&mn[i])));
                }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816(ot[nt][4 * hf + jn], f[0][0], f[1][0], f[0][1], f[1][1], pb[nt][h][0],
                          pb[nt][h][1]);
            }
          }
        }
        // a patched tile was written through the generic proxy; order that before the next TMA
        // write into this stage
        if (APPEND && patched) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_empty + st * 8);
      }
      if (kHoldQ) {
        if (kQSmem) fence_proxy_async_smem();   // the tile was permuted in place
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_qempty + qs * 8);
      }
      j += npair;

      // ---- hand this warp's state to the epilogue ----
      const int sb = k & 1;
      if (k >= 2 && !mbar_wait(bar_sfree + sb * 8, ((k >> 1) - 1) & 1, abort)) flag_timeout(a, abort);
      float* o_d = stO + sb * NCW * a.R * kSt;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lv = tl[nt][e];
          lv += __shfl_xor_sync(0xffffffffu, lv, 4);
          lv += __shfl_xor_sync(0xffffffffu, lv, 8);
          lv += __shfl_xor_sync(0xffffffffu, lv, 16);
          const int r = 8 * nt + 2 * t4 + e;
          if (r < a.R) {
            float4* dst = reinterpret_cast<float4*>(o_d + (w * a.R + r) * kSt + 16 * g);
            dst[0] = make_float4(ot[nt][0][e], ot[nt][1][e], ot[nt][2][e], ot[nt][3][e]);
            dst[1] = make_float4(ot[nt][4][e], ot[nt][5][e], ot[nt][6][e], ot[nt][7][e]);
            dst[2] = make_float4(ot[nt][0][2 + e], ot[nt][1][2 + e], ot[nt][2][2 + e],
                                 ot[nt][3][2 + e]);
            dst[3] = make_float4(ot[nt][4][2 + e], ot[nt][5][2 + e], ot[nt][6][2 + e],
                                 ot[nt][7][2 + e]);
            if (g == 0) {
              stM[(sb * NCW + w) * a.R + r] = tm[nt][e];
              stL[(sb * NCW + w) * a.R + r] = lv;
            }
          }
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sdone + (k & 1) * 8);
      ++k;
      has = cur.next(s);
    }
  }

  // ---- end of the slice (the producer has left; t: dense index over consumers + epilogue)
  if (warp != NCW && last.k >= 0)
    finish_slice<NCW, kSeg4>(a, last, pre, per, smem, L::kQ, stO, stM, stL, npend_s, fast_s,
                             warp < NCW ? tid : tid - 32);
}

// ---------------------------------------------------------------------------------------------
// Host side.

template <int NCW, int NST, int NT>
size_t smem4_of(int R, int B, int newkv_bytes) {
  return Smem4<NCW, NST, NT>::bytes(R, B, newkv_bytes);
}

template <int NCW, int NST, int NT, int MINB>
Variant variant4(bool append) {
  const void* fn =
      append ? reinterpret_cast<const void*>(&decode_int4_kernel<NCW, NST, NT, MINB, true>)
             : reinterpret_cast<const void*>(&decode_int4_kernel<NCW, NST, NT, MINB, false>);
  return Variant{fn, NT, false, (NCW + 2) * 32, &smem4_of<NCW, NST, NT>};
}

int launch_decode_int4(void* out, const void* q, const void* k_new, const void* v_new,
                       const void* k_cache, const void* v_cache, int num_blocks,
                       const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                       int num_seqs, int q_len, int Hq, int Hkv, int head_dim, int block_size,
                       float scale, void* workspace, size_t workspace_bytes, bool append,
                       pkv_stream_t stream) {
  if (num_seqs < 0 || q_len < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || head_dim != kD ||
      !valid_block_size(block_size) || num_blocks < 0 || max_blocks < 0)
    return PKV_EINVAL;
  const int G = Hq / Hkv;
  if (static_cast<int64_t>(G) * q_len > 32) return PKV_EINVAL;
  if (num_seqs == 0) return PKV_OK;
  if (num_seqs > kMaxSeqs) return PKV_EINVAL;
  const int R = G * q_len;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !workspace)
    return PKV_EINVAL;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return PKV_EINVAL;
  if (append && (!k_new || !v_new || !aligned16(k_new) || !aligned16(v_new))) return PKV_EINVAL;
  // all chunk indices and TMA rows fit in int32
  const int64_t rows = static_cast<int64_t>(num_blocks) * Hkv * block_size;
  const int64_t max_ctx = static_cast<int64_t>(max_blocks) * block_size;
  if (rows >= (1ll << 31) || max_ctx >= (1ll << 31) ||
      static_cast<int64_t>(num_seqs) * Hkv * ((max_ctx + kChunk - 1) / kChunk + kSeg4) >=
          (1ll << 30))
    return PKV_EINVAL;
  if (num_blocks == 0) return PKV_EINVAL;
  const WsLayout ws = ws_layout(num_seqs, Hkv, R);
  if (workspace_bytes < ws.total) return PKV_ENOSPC;

  const Variant v = R <= 8 ? variant4<4, 8, 1, 2>(append)
                    : R <= 16 ? variant4<4, 8, 2, 1>(append) : variant4<4, 12, 4, 1>(append);
  const int newkv_bytes = append ? 2 * q_len * 512 : 0;
  const size_t smem = v.smem(R, num_seqs, newkv_bytes);
  if (smem > 227 * 1024) return PKV_EINVAL;
  int status = PKV_OK;
  const int grid = grid_size(v, smem, &status);
  if (!grid) return status != PKV_OK ? status : PKV_EINVAL;

  CUtensorMap tmK, tmV, tmQ;
  const cuuint64_t kv_dims[2] = {kInt4Row, static_cast<cuuint64_t>(rows)};
  const cuuint64_t kv_strides[1] = {kInt4Row};
  const cuuint32_t kv_box[2] = {kInt4Row, kChunk};
  int st = encode(&tmK, k_cache, 2, kv_dims, kv_strides, kv_box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                  CU_TENSOR_MAP_SWIZZLE_NONE);
  if (st == PKV_OK)
    st = encode(&tmV, v_cache, 2, kv_dims, kv_strides, kv_box, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                CU_TENSOR_MAP_SWIZZLE_NONE);
  const cuuint64_t q_dims[3] = {static_cast<cuuint64_t>(kD), static_cast<cuuint64_t>(Hq),
                                static_cast<cuuint64_t>(num_seqs) * q_len};
  const cuuint64_t q_strides[2] = {kD * 2, static_cast<cuuint64_t>(Hq) * kD * 2};
  const cuuint32_t q_box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(q_len)};
  if (st == PKV_OK) st = encode(&tmQ, q, 3, q_dims, q_strides, q_box);
  if (st != PKV_OK) return st;

  unsigned int* err = device_error_ptr();
  if (!err) return cuda_status(cudaGetLastError());
  DecodeArgs args = {};
  args.out = static_cast<__half*>(out);
  args.block_tables = block_tables;
  args.context_lens = context_lens;
  uint8_t* wsb = static_cast<uint8_t*>(workspace);
  args.counters = reinterpret_cast<int*>(wsb + ws.counters);
  args.part_ml = reinterpret_cast<float*>(wsb + ws.part_ml);
  args.part_o = reinterpret_cast<float*>(wsb + ws.part_o);
  args.err = err;
  args.num_blocks = num_blocks;
  args.max_blocks = max_blocks;
  args.num_seqs = num_seqs;
  args.q_len = q_len;
  args.Hq = Hq;
  args.Hkv = Hkv;
  args.G = G;
  args.R = R;
  args.block_size = block_size;
  int shift = 0;
  while ((kChunk << shift) < block_size) ++shift;
  args.bs_shift = shift;
  args.scale_log2 = scale * 1.4426950408889634f;
  args.k_new = static_cast<const __half*>(k_new);
  args.v_new = static_cast<const __half*>(v_new);
  args.k_pool = static_cast<__half*>(const_cast<void*>(k_cache));
  args.v_pool = static_cast<__half*>(const_cast<void*>(v_cache));

  void* params[4] = {&tmK, &tmV, &tmQ, &args};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(v.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = (append && early_start_enabled()) ? 1 : 0;
  return cuda_status(cudaLaunchKernelExC(&cfg, v.fn, params));
}

}  // namespace
}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_paged_attn_decode_int4(void* out, const void* q, const void* k_cache,
                               const void* v_cache, int num_blocks, const int32_t* block_tables,
                               int max_blocks_per_seq, const int32_t* context_lens, int num_seqs,
                               int q_len, int num_q_heads, int num_kv_heads, int head_dim,
                               int block_size, float scale, void* workspace,
                               size_t workspace_bytes, pkv_stream_t stream) {
  return launch_decode_int4(out, q, nullptr, nullptr, k_cache, v_cache, num_blocks, block_tables,
                            max_blocks_per_seq, context_lens, num_seqs, q_len, num_q_heads,
                            num_kv_heads, head_dim, block_size, scale, workspace,
                            workspace_bytes, false, stream);
}

int pkv_paged_attn_decode_append_int4(void* out, const void* q, const void* k_new,
                                      const void* v_new, void* k_cache, void* v_cache,
                                      int num_blocks, const int32_t* block_tables,
                                      int max_blocks_per_seq, const int32_t* context_lens,
                                      int num_seqs, int q_len, int num_q_heads, int num_kv_heads,
                                      int head_dim, int block_size, float scale, void* workspace,
                                      size_t workspace_bytes, pkv_stream_t stream) {
  return launch_decode_int4(out, q, k_new, v_new, k_cache, v_cache, num_blocks, block_tables,
                            max_blocks_per_seq, context_lens, num_seqs, q_len, num_q_heads,
                            num_kv_heads, head_dim, block_size, scale, workspace,
                            workspace_bytes, true, stream);
}

}  // extern "C"
