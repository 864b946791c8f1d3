// pkv_decode_int4.cu -- paged decode attention over a 4-bit cache (pkv_int4.cuh's rows) for
// sm_103a.
//
// What it computes: pkv_paged_attn_decode's operation with K_t[d] = s_K code_K + z_K and
// V_t[d] = s_V code_V + z_V, (s, z) of the 32 elements that d belongs to.
//
// What bounds it: 160 bytes per (token, kv head) against 512 of the fp16 cache, so the work per
// key, not the loads, is what the loop has to keep short: at the copy rate an SM has ~109 cycles
// for 16 keys of one kv head. Codes go to the tensor cores as they stand; nothing is widened
// per element:
//  * Stream, slices, split units and their merge are those of pkv_decode.cu (shared in
//    pkv_decode_common.cuh). A stage is two 16-token chunks: K of both, V of both, four runs of
//    1280 contiguous bytes. Rows are 20 words apart: any 8 rows x 16 bytes touch all 32 banks
//    without a swizzle.
//  * No producer: every consumer warp keeps a ring of its own stages in flight with cp.async (10
//    copies of 512 bytes a stage), waits for its own copies and needs no barrier. One producer
//    warp for all (tensor tiles or bulk copies, an mbarrier pair per stage) took ~450 ns a stage
//    whatever its size, which bounded the kernel at 3 TB/s.
//  * Transposed tile: S^T = K Q^T and O^T = V^T P^T, keys (and output dims) on the mma's 16-row
//    side, 8 query rows on its 8 columns.
//  * Four bits at bits 2-5 (6-9) of a 16-bit half are the fp16 subnormal c 2^-22 (c 2^-18),
//    exactly, and the products' sums are fp32: one AND of the word shifted left by 2 or right by 6
//    makes an mma operand of two codes. (The tensor cores count a subnormal's exponent as -14 when
//    they align products, and cut below 2^-25 of the largest: at bits 0-3, without the left shift,
//    a product loses up to 2^-15 of a code step times the largest weight, always downwards, here
//    2^-17. The shifts cost 0 to 3 % of the time.)
//  * Keys: sum_d q_d (s c_d + z) = s sum_d q_d c_d + z sum_d q_d per group of 32 dims. The
//    queries are scaled by a power of two that puts the row's largest between 2^10 and 2^11, those
//    that meet codes at bits 2-5 by 16 more (both exact: what falls below fp16's smallest is
//    under 2^-34 of the row's largest). The group's sum is scaled by s in fp32; z times the
//    group's query sum is one more product per 16 keys, the (s, z) words as they stand against
//    (0, sum), the sum split in two fp16 numbers.
//  * Values: O[d] = sum_k (p_k s_k) c_kd + sum_k p_k z_k. ldmatrix.trans brings, per group, a
//    register with four codes of two neighbouring keys. The weights take the group's scales as
//    packed fp16 products, each with what its rounding left over as a second operand (s c and z
//    nearly cancel for values near zero, so an error of 2^-11 of s c would show). The minima's
//    sum is one product per 16 keys with the (s, z) halves as its rows; it is added when the
//    segment ends.
//  * Softmax as in pkv_decode.cu (fp32, exp2 domain, a reference that follows the running
//    maximum lazily). p and p s are fp16: the reference stays kShift = 11 powers of two below
//    the maximum while every scale is below 2 (p < 2^13, p s < 2^14, and values of 1e-6 still
//    count); the first scale of 2 or more (values over a range of 30) moves it up to the maximum
//    (p <= 4, p s <= 4 x 8736) for the rest of the segment. That one rounding of a weight (2^-11 of
//    it at most; the weights' sum takes them unrounded) is what the error has over attention in
//    fp32 with the same fp16 output: 2.4e-4 to 3.0e-4 of the output's norm against 2.1e-4.
//  * Tokens past the context hold anything: their scores are masked and their (s, z) of V set
//    to zero.
//  * More than 8 rows: two to four warps take a stage, 8 rows each (and a copy of their own; all
//    but the first come from L2). Two row tiles in one warp save the second masking of the codes
//    but not the registers: with two, four drafts of 6 heads took 36 us, with one 25.
//  * Fused append: the warp that prepares the queries also quantises the segment's new rows, into
//    the pool and for the consumers, which copy them over their stage's stale ones (done by the
//    consumers, 128 ragged sequences took 57 us instead of 54).
// Where it stands: 32 sequences of 16384 tokens, 8 kv heads, 8 queries each take 134 us (5.0 TB/s,
// 73 % of the copy rate). The loads alone take 104, the arithmetic alone 106; together they share
// the SM's issue slots (50 % used, ALU 47 %, tensor 34 %, shared memory 34 %), and neither 12
// warps instead of 8 (130) nor fewer instructions (the queries' operands loaded half as often: 140)
// change much.
#include <cuda_fp16.h>

#include "pkv_decode_common.cuh"
#include "pkv_device.cuh"
#include "pkv_int4.cuh"
#include "pkv_internal.h"

namespace pkv {
namespace {

constexpr int kTile = kChunk * kInt4Row;     // one chunk's K (or V): 1280 bytes
constexpr int kStage4 = 4 * kTile;           // K of two chunks, V of two chunks
constexpr int kNewRow = 2 * kInt4Row;        // a new token's K and V
// Per-segment cost in chunks (see kSegCost): queries, hand-off and merge of a segment take a CTA
// ~1.5 us, the time of a dozen chunks (70B mixed lengths: 62 us with 4, 55 with 8, 51 with 12).
constexpr int kSeg4 = 12;
// A unit of n chunks cut into slices of T costs about T chunks' time and a merge of n / T partials,
// each kPartCost chunks' worth: least at T = sqrt(kPartCost n), so no slice is cut finer. One
// sequence of 4096 tokens and 2 kv heads (all 304 CTAs otherwise) 44 -> 14 us, of 1536 36 -> 11;
// with a cost of 1.5, 2.5, 4, 6 the lengths from 256 to 131072 stay within 8 % of each other.
constexpr float kPartCost = 3.f;
// Few short units: a whole unit for each CTA, when its warps then take at most kAlone rounds of
// stages more than an equal share has; that costs less than writing and merging partials (one
// sequence of 256 tokens 9.4 -> 7.2 us, 32 of 1024 with 8 kv heads 18.6 -> 16.3).
constexpr int kAlone = 3;
constexpr size_t kMaxSmem = 227 * 1024;
// How far the softmax's reference stays below the running maximum (see above), and how far a
// weight may grow past the maximum it was taken at before the reference moves.
constexpr float kShift = 11.f, kGrow = 2.f;
// Stages after which a warp's sums move to its state buffer. The tensor cores' fp32 sums truncate,
// and the two large sums that make a value's (of p s c and of p z) do not lose alike: over 100
// stages a warp (16384 tokens) their difference was off by 6.9e-4 relative, over 64 by 5.2e-4, over
// 32 by 3.6e-4, over 16 by 2.9e-4, near what the rounded weights and output alone cost (2.7e-4).
// With 16 a sum takes 64 products (two chunks, weights and what they lost); moving the sums costs
// at most 3 % of the time (134.0 us against 130.5 without).
constexpr int kFlush = 16;

// Shared-memory layout (offsets from a 128-byte aligned base). NCS: warps that share the stages
// among them, RS: warps that take one stage, 8 query rows each, ND: stages in flight per warp.
template <int NCS, int RS, int ND>
struct Smem4 {
  static constexpr int kQTile = 5 * 512;              // 8 rows: fragments of 4 groups, constants
  static constexpr int kQBuf = RS * kQTile;
  static constexpr int kQ = NCS * RS * ND * kStage4;
  static constexpr int kBars = kQ + 2 * kQBuf;        // qfull[2], qempty[2], sdone, sfree, nfull[2]
  static constexpr int kFlags = kBars + 8 * 8;
  static constexpr int kState = (kFlags + 64 + 15) & ~15;   // [NCS] segment states
  __host__ __device__ static int state_floats(int R) { return NCS * R * (kSt + 2); }
  __host__ __device__ static int seq_off(int R) { return kState + state_floats(R) * 4; }
  __host__ __device__ static int newkv_off(int R, int B) {
    return (seq_off(R) + (2 * B + 1) * 4 + 127) & ~127;
  }
  __host__ static size_t bytes(int R, int B, int newkv_bytes) {
    return 128 + static_cast<size_t>(newkv_off(R, B)) + static_cast<size_t>(newkv_bytes);
  }
  // the merge of split units stages at least two partials in the stage memory
  static_assert(kQ >= 8 * RS * ((kD + 8) * 4 + 2 * (kD + 4) * 4), "merge staging");
};

// A warp's walk over the stages it loads: stage jp of a segment goes to warp (jp + stages before
// the segment) mod NCS. Pool rows are fetched for up to 16 of the warp's stages at once (lane l:
// chunk l & 1 of the (l / 2)-th), one group ahead of their use.
template <int NCS>
struct StageWalk {
  Seg s;
  int j, jp;        // stages of the slice before the segment; the warp's next stage in it
  bool has;
  int rows, n, i;   // current group: pool rows per lane, stages, position
  int ids, at, nn;  // group ahead: block ids, (h << 16 | first row in the block) per lane, stages

  __device__ __forceinline__ static int npair(const Seg& s) { return (s.c1 - s.c0 + 1) >> 1; }
  __device__ __forceinline__ void enter(int w) { jp = ((w - j) % NCS + NCS) % NCS; }

  // requests the block ids of the next group
  __device__ __forceinline__ void fetch(const DecodeArgs& a, const CursorT<kSeg4>& cur, int w,
                                        int lane) {
    nn = 0;
    ids = -1;
    at = -1;
    while (has && jp >= npair(s)) {
      j += npair(s);
      has = cur.next(s);
      enter(w);
    }
    if (!has) return;
    const int np = npair(s);
    nn = min(16, (np - jp + NCS - 1) / NCS);
    const int c = s.c0 + 2 * (jp + (lane >> 1) * NCS) + (lane & 1);
    if ((lane >> 1) < nn && c < s.c1) {
      ids = a.block_tables[static_cast<int64_t>(s.b) * a.max_blocks + (c >> a.bs_shift)];
      at = (s.h << 8) | ((c & ((1 << a.bs_shift) - 1)) << 4);
    }
    jp += nn * NCS;
  }
  // makes it the current one: rows (-1: no chunk, -2: bad block id)
  __device__ __forceinline__ void take(const DecodeArgs& a) {
    rows = -1;
    if (at >= 0) {
      if (ids >= 0 && ids < a.num_blocks) {
        rows = (ids * a.Hkv + (at >> 8)) * a.block_size + (at & 255);
      } else {
        atomicOr(a.err, PKV_DEVERR_BLOCK_ID);
        rows = -2;
      }
    }
    n = nn;
    i = 0;
  }
  __device__ __forceinline__ void start(const DecodeArgs& a, const CursorT<kSeg4>& cur, int begin,
                                        int w, int lane) {
    j = 0;
    has = cur.first(begin, s);
    enter(w);
    fetch(a, cur, w, lane);
    take(a);
    fetch(a, cur, w, lane);
  }
  // requests the warp's next stage into buffer `dst`, if there is one; one group of copies
  __device__ __forceinline__ void load(const DecodeArgs& a, const CursorT<kSeg4>& cur, int w,
                                       int lane, uint32_t dst, uint64_t policy) {
    if (i == n) {
      take(a);
      fetch(a, cur, w, lane);
    }
    if (i < n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = __shfl_sync(0xffffffffu, rows, 2 * i + h);
        const uint32_t kd = dst + h * kTile, vd = kd + 2 * kTile;
        if (r >= 0) {
          // 80 pieces of 16 bytes each of K and V: 64 + 64, and the last 16 of both together
          const int64_t off = static_cast<int64_t>(r) * kInt4Row + lane * 16;
          const uint8_t* ks = reinterpret_cast<const uint8_t*>(a.k_pool) + off;
          const uint8_t* vs = reinterpret_cast<const uint8_t*>(a.v_pool) + off;
          cp_async_16_hint(kd + lane * 16, ks, policy);
          cp_async_16_hint(kd + lane * 16 + 512, ks + 512, policy);
          cp_async_16_hint(vd + lane * 16, vs, policy);
          cp_async_16_hint(vd + lane * 16 + 512, vs + 512, policy);
          const bool k16 = lane < 16;
          cp_async_16_hint((k16 ? kd : vd - 256) + lane * 16 + 1024, (k16 ? ks : vs - 256) + 1024,
                           policy);
        } else if (r == -2) {   // a chunk behind a bad block id reads as zeros
          for (int x = lane; x < kTile / 16; x += 32) {
            st_shared_v4(kd + x * 16, make_uint4(0, 0, 0, 0));
            st_shared_v4(vd + x * 16, make_uint4(0, 0, 0, 0));
          }
        }
      }
      ++i;
    }
    cp_async_commit();
  }
};

// 0xffff in the halves of w that are NaN, 0 in the others.
__device__ __forceinline__ uint32_t nan_halves(uint32_t w) {
  return __hneu2_mask(as_half2(w), as_half2(w));
}

// Warps 0 .. NCS RS - 1 consume; the next one prepares the queries, the last one is the epilogue
// (merges each segment's per-warp states, writes outputs and split units' partials).
template <int NCS, int RS, int ND, int MINB, bool APPEND>
__global__ void __launch_bounds__((NCS * RS + 2) * 32, MINB)
decode_int4_kernel(const DecodeArgs a, const __half* q_in) {
  using L = Smem4<NCS, RS, ND>;
  constexpr int NCW = NCS * RS;
  if (!APPEND) griddep_wait();   // (the fused form reads ahead; see the early-start contract)
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_qfull = sbase + L::kBars;
  const uint32_t bar_qempty = bar_qfull + 2 * 8;
  const uint32_t bar_sdone = bar_qempty + 2 * 8;
  const uint32_t bar_sfree = bar_sdone + 8;
  const uint32_t bar_nfull = bar_sfree + 8;
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kFlags);
  int* npend_s = reinterpret_cast<int*>(smem + L::kFlags) + 1;   // then 2 x (b, h, nb)
  volatile int* fast_s = reinterpret_cast<volatile int*>(smem + L::kFlags) + 8;
  int* longest_s = reinterpret_cast<int*>(smem + L::kFlags) + 9;
  float* stO = reinterpret_cast<float*>(smem + L::kState);       // [NCS][R][kSt]
  float* stM = stO + NCS * a.R * kSt;                             // [NCS][R]
  float* stL = stM + NCS * a.R;                                   // [NCS][R]
  int* pre = reinterpret_cast<int*>(smem + L::seq_off(a.R));
  int* slen = pre + a.num_seqs + 1;

  const int tid = threadIdx.x;
  const int warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int B = a.num_seqs;

  // ---- per-sequence lengths and chunk counts -------------------------------------------------
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_qfull + s * 8, 1);
      mbar_init(bar_qempty + s * 8, NCW);
      mbar_init(bar_nfull + s * 8, 1);
    }
    mbar_init(bar_sdone, NCW);
    mbar_init(bar_sfree, 1);
    *abort = 0;
    *npend_s = 0;
    *longest_s = 0;
    pre[0] = 0;
  }
  int longest = 0;
  for (int b = tid; b < B; b += blockDim.x) {
    int ctx = a.context_lens[b];
    const int lim = a.max_blocks * a.block_size;
    if (ctx < 0 || ctx > lim) {
      atomicOr(a.err, PKV_DEVERR_CONTEXT);
      // no position of such a context is where the caller thinks: a fused call writes nothing of it
      ctx = APPEND || ctx < 0 ? 0 : lim;
    }
    const int nchunks = (ctx + kChunk - 1) / kChunk;
    longest = max(longest, nchunks);
    slen[b] = ctx;
    pre[b + 1] = nchunks > 0 ? nchunks + kSeg4 : 0;
  }
  fence_barrier_init();
  __syncthreads();
  if (longest > 0) atomicMax(longest_s, longest);
  if (warp == 0) scan_chunks(pre, B, lane);
  __syncthreads();

  // ---- this CTA's slice of the stream --------------------------------------------------------
  const int total = pre[B] * a.Hkv;
  const int per = max(static_cast<int>((total + gridDim.x - 1) / gridDim.x),
                      static_cast<int>(sqrtf(kPartCost * *longest_s)));
  int begin = blockIdx.x * per, end = min(total, begin + per);
  if (B * a.Hkv <= gridDim.x && *longest_s <= 2 * NCS * ((per + 2 * NCS - 1) / (2 * NCS) + kAlone)) {
    const int b = blockIdx.x / a.Hkv;
    const int len = b < B ? pre[b + 1] - pre[b] : 0;
    begin = len > 0 ? pre[b] * a.Hkv + (blockIdx.x - b * a.Hkv) * len : 0;
    end = begin + len;
  }
  const CursorT<kSeg4> cur{pre, B, a.Hkv, end};

  // let the next kernel on the stream launch as SM resources free up (it waits for this one
  // before it reads anything this kernel writes)
  if (tid == 0) griddep_launch_dependents();

  LastSeg last{-1, 0, 0, 0, 0, true, false};
  auto set_last = [&](const Seg& s, int k) {
    last = LastSeg{k, s.b, s.h, s.nb, 2 * static_cast<int>(blockIdx.x) + (k == 0 ? 0 : 1),
                   s.c0 == 0 && s.c1 == s.nb, s.c0 == 0};
  };

  if (warp == NCW) {
    // =================================== queries =============================================
    // An early-started launch (APPEND) has its first stages on the way already; queries, new
    // rows, outputs and the workspace are touched only after the preceding kernel completed.
    griddep_wait();
    // Queries of segment kk into buffer kk & 1 as the products' B operands: for lane (g, t4), row
    // g of each tile, the dims d0 = 32 gr + 8 t4 .. d0 + 7 of group gr (the codes of its key
    // words), paired as the masks pair them. And per lane: the sum of group t4 as two fp16 numbers
    // in the upper halves (the lower ones meet the scales), and what makes scores of rows 2 t4,
    // 2 t4 + 1 from the products.
    auto prepare = [&](const Seg& sg, int kk) {
      const uint32_t qb = sbase + L::kQ + (kk & 1) * L::kQBuf;
#pragma unroll 1
      for (int tile = 0; 8 * tile < a.R; ++tile) {
        const int row = 8 * tile + g;
        uint4 v[4];
        __half2 big = as_half2(0u);
        const int qi = row / a.G;
        // a query before its sequence's first token sees nothing, whatever it holds: taken as zeros, it
        // keeps a NaN from its scores, which are all masked
        const bool sees = row < a.R && slen[sg.b] - a.q_len + qi >= 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            q_in +
            ((static_cast<int64_t>(sg.b) * a.q_len + qi) * a.Hq + sg.h * a.G + row - qi * a.G) * kD);
#pragma unroll
        for (int gr = 0; gr < 4; ++gr)
          v[gr] = sees ? src[4 * gr + t4] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int gr = 0; gr < 4; ++gr)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            big = __hmax2_nan(big, __habs2(as_half2(u4_word(v[gr], i))));
        big = __hmax2_nan(big, __lowhigh2highlow(big));
        big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = __hmax2_nan(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const float top = __low2float(big);
        // 2^(10 - exponent of the row's largest), which comes to lie in [2^10, 2^11); a negative
        // score scale turns the queries' signs instead, so that a larger product is a larger score
        const int ex = top > 0.f ? static_cast<int>(__float_as_uint(top) >> 23) : 127;
        float f = __uint_as_float(static_cast<uint32_t>(264 - ex) << 23);
        // codes come in as c 2^-18; a NaN or an infinity among the queries makes the scores NaN
        float unit = top <= 65504.f
                         ? fabsf(a.scale_log2) *
                               (262144.f * __uint_as_float(static_cast<uint32_t>(ex - 10) << 23))
                         : __uint_as_float(0x7fffffffu);
        if (a.scale_log2 < 0.f) f = -f;
        if (unit == 0.f) unit = 0x1p-100f;   // so that masked scores stay -infinity
        float own = 0.f;
#pragma unroll
        for (int gr = 0; gr < 4; ++gr) {
          float sum = 0.f;
          float2 u[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            u[i] = __half22float2(as_half2(u4_word(v[gr], i)));
            u[i].x *= f;
            u[i].y *= f;
            sum += u[i].x + u[i].y;
          }
          st_shared_v4(qb + tile * L::kQTile + gr * 512 + lane * 16,
                       make_uint4(pack_half2(u[0].x * 16.f, u[2].x * 16.f),    // dims 0, 4
                                  pack_half2(u[1].x * 16.f, u[3].x * 16.f),    // dims 2, 6
                                  pack_half2(u[0].y, u[2].y),                  // dims 1, 5
                                  pack_half2(u[1].y, u[3].y)));                // dims 3, 7
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          if (gr == t4) own = sum * 0x1p-18f;   // in the products' units; at most 2^-2
        }
        const __half hi = __float2half_rn(own);
        const __half lo = __float2half_rn(own - __half2float(hi));
        const float r0 = __shfl_sync(0xffffffffu, unit, 8 * t4);
        const float r1 = __shfl_sync(0xffffffffu, unit, 8 * t4 + 4);
        st_shared_v4(qb + tile * L::kQTile + 2048 + lane * 16,
                     make_uint4(static_cast<uint32_t>(__half_as_ushort(hi)) << 16,
                                static_cast<uint32_t>(__half_as_ushort(lo)) << 16,
                                __float_as_uint(r0), __float_as_uint(r1)));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_qfull + (kk & 1) * 8);
      if (!APPEND) return;
      // the segment's new rows, K in lanes 0-15, V in 16-31: quantised once, into the pool and for
      // the consumers, who need them when they come to the rows' chunks
      const uint32_t nkv = sbase + L::newkv_off(a.R, B) + (kk & 1) * a.q_len * kNewRow;
      const int which = lane >> 4, p = lane & 15;
      const __half* src = which ? a.v_new : a.k_new;
      for (int i = 0; i < a.q_len; ++i) {
        const int pos = slen[sg.b] - a.q_len + i;
        const int c = pos >> 4;
        if (pos < 0 || c < sg.c0 || c >= sg.c1) continue;
        const int id = a.block_tables[static_cast<int64_t>(sg.b) * a.max_blocks + (c >> a.bs_shift)];
        const int64_t row = (static_cast<int64_t>(sg.b) * a.q_len + i) * a.Hkv + sg.h;
        uint32_t codes, params;
        int4_quantise(reinterpret_cast<const uint4*>(src + row * kD)[p], codes, params);
        const uint32_t to = nkv + i * kNewRow + which * kInt4Row;
        st_shared_u32(to + 4 * p, codes);
        if ((p & 3) == 0) st_shared_u32(to + kInt4Params + p, params);
        if (id >= 0 && id < a.num_blocks) {
          const int64_t prow = (static_cast<int64_t>(id) * a.Hkv + sg.h) * a.block_size +
                               (pos & (a.block_size - 1));
          uint32_t* pool = reinterpret_cast<uint32_t*>(
              reinterpret_cast<uint8_t*>(which ? a.v_pool : a.k_pool) + prow * kInt4Row);
          pool[p] = codes;
          if ((p & 3) == 0) pool[(kInt4Params + p) / 4] = params;
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_nfull + (kk & 1) * 8);
    };
    Seg s;
    bool has = cur.first(begin, s);
    for (int k = 0; has; ++k) {
      if (k >= 2 && !mbar_wait(bar_qempty + (k & 1) * 8, ((k >> 1) - 1) & 1, abort))
        flag_timeout(a, abort);
      prepare(s, k);
      has = cur.next(s);
    }
    // sequences without any chunk get zeros (their units are in no CTA's slice)
    for (int b = blockIdx.x; b < B; b += gridDim.x) {
      if (pre[b + 1] != pre[b]) continue;
      const int n = a.q_len * a.Hq * kD;
      for (int i = lane; i < n; i += 32)
        a.out[static_cast<int64_t>(b) * n + i] = __float2half_rn(0.f);
    }
    return;
  }
  if (warp == NCW + 1) {
    // =================================== epilogue ============================================
    griddep_wait();
    Seg s;
    if (cur.first(begin, s)) {
      int npend = 0, k = 0;
      Seg nx = s;
      while (cur.next(nx)) {
        if (!mbar_wait(bar_sdone, k & 1, abort)) flag_timeout(a, abort);
        const bool complete = (s.c0 == 0 && s.c1 == s.nb);
        const int slot = 2 * blockIdx.x + (k == 0 ? 0 : 1);
        merge_rows<NCS>(a, stO, stM, stL, s, complete,
                        a.part_o + static_cast<int64_t>(slot) * a.R * kD,
                        a.part_ml + static_cast<int64_t>(slot) * a.R * 4, lane);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_sfree);
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
        s = nx;
        ++k;
      }
      if (lane == 0) *npend_s = npend;
      set_last(s, k);
    }
  } else {
    // =================================== consumers ===========================================
    const int w = warp % NCS, rs = warp / NCS;   // share of the stages, query rows 8 rs .. + 7
    // ldmatrix row addresses: matrices 0, 1 the two key octets of 16 bytes, 2, 3 of the next 16
    // (codes), or the two octets of the next chunk (scales and minima)
    const uint32_t lm_row = ((lane >> 3) & 1) * 8 * kInt4Row + (lane & 7) * kInt4Row;
    const uint32_t lm_codes = lm_row + (lane >> 4) * 16;
    const uint32_t lm_par = lm_row + (lane >> 4) * kTile + kInt4Params;
    const uint64_t kv_policy = l2_policy_evict_first();
    const uint32_t ring = sbase + warp * (ND * kStage4);
    StageWalk<NCS> walk;
    walk.start(a, cur, begin, w, lane);
    for (int i = 0; i < ND; ++i) walk.load(a, cur, w, lane, ring + i * kStage4, kv_policy);
    const uint32_t wide_mask = (g & 1) ? 0u : 0x40004000u;
    int slot = 0;   // ring position of the warp's next stage
    int j = 0, k = 0;
    Seg s;
    bool has = cur.first(begin, s);
    while (has) {
      const int qs = k & 1;
      const uint32_t qb = sbase + L::kQ + qs * L::kQBuf + rs * L::kQTile + lane * 16;
      if (!mbar_wait(bar_qfull + qs * 8, (k >> 1) & 1, abort)) flag_timeout(a, abort);
      const int Lc = slen[s.b];
      // the sums of group t4; what makes scores of rows 2 t4, 2 t4 + 1 from the products
      const uint4 qc = ld_shared_v4(qb + 2048);
      const float rsc[2] = {__uint_as_float(qc.z), __uint_as_float(qc.w)};

      // per row: the reference's negative (0 before the first score), the product above which it
      // moves, the sum of the weights
      float nm[2] = {0.f, 0.f}, thr[2] = {kNegInf, kNegInf}, tl[2] = {0.f, 0.f};
      float ot[4][2][4], oz[4];
      const int r0 = 8 * rs + 2 * t4;
      // query tokens of rows 2 t4 (low half), 2 t4 + 1
      const int qis = min(r0 / a.G, a.q_len - 1) | (min((r0 + 1) / a.G, a.q_len - 1) << 16);
      float shift = kShift;   // the same for all lanes

      const int nchunk = s.c1 - s.c0;
      const int npair = (nchunk + 1) >> 1;
      int jp = ((w - j) % NCS + NCS) % NCS;
      bool held = false;      // the state buffer holds what this segment's earlier stages gave
      do {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          oz[i] = 0.f;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr) ot[gr][0][i] = ot[gr][1][i] = 0.f;
        }
        for (int left = kFlush; left > 0 && jp < npair; --left, jp += NCS) {
          cp_async_wait<ND - 1>();
          __syncwarp();                        // every lane's copies of this stage are in
          const uint32_t stK = ring + slot * kStage4;
          const uint32_t stV = stK + 2 * kTile;
          const int c = s.c0 + 2 * jp;
          const bool two = c + 1 < s.c1;
          const int nk = two ? 2 * kChunk : kChunk;
          const bool full = two && (c + 2) * kChunk <= Lc - a.q_len + 1;
          if (APPEND && (c * kChunk + nk > Lc - a.q_len)) {
            // new rows of these chunks go into the stage's tiles
            const int first_new = Lc - a.q_len;
            const uint32_t nkv = sbase + L::newkv_off(a.R, B) + qs * a.q_len * kNewRow;
            if (!mbar_wait(bar_nfull + qs * 8, (k >> 1) & 1, abort)) flag_timeout(a, abort);
            for (int i = 0; i < a.q_len; ++i) {
              const int tk = first_new + i - c * kChunk;
              if (first_new + i < 0 || tk < 0 || tk >= nk || lane >= kInt4Row / 4) continue;
              const uint32_t from = nkv + i * kNewRow + 4 * lane, to = stK + tk * kInt4Row + 4 * lane;
              st_shared_u32(to, ld_shared_u32(from));
              st_shared_u32(to + 2 * kTile, ld_shared_u32(from + kInt4Row));
            }
            __syncwarp();
          }

          // ---- S^T = K Q^T, 16 keys (g, g + 8) at a time ----
          float x[2][4];       // [chunk h][key g: rows 2 t4, + 1; key g + 8: the same]
          uint32_t kz[4];      // (s, z) of group t4: keys g, g + 8 of both chunks
          ldsm_x4(stK + lm_par, kz[0], kz[1], kz[2], kz[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t kb = stK + h * kTile;
            uint32_t kw[4][2];
            ldsm_x4(kb + lm_codes, kw[0][0], kw[0][1], kw[1][0], kw[1][1]);
            ldsm_x4(kb + lm_codes + 32, kw[2][0], kw[2][1], kw[3][0], kw[3][1]);
            const uint4 p0 = ld_shared_v4(kb + g * kInt4Row + kInt4Params);
            const uint4 p1 = ld_shared_v4(kb + (g + 8) * kInt4Row + kInt4Params);
            x[h][0] = x[h][1] = x[h][2] = x[h][3] = 0.f;
            mma_f16(x[h], kz[2 * h], kz[2 * h + 1], kz[2 * h], kz[2 * h + 1], qc.x, qc.y);
            // all groups at a time: their products do not wait on each other
            float t[4][4];
#pragma unroll
            for (int part = 0; part < 2; ++part) {
              const uint32_t m = part ? 0x03c003c0u : 0x003c003cu;
#pragma unroll
              for (int gr = 0; gr < 4; ++gr) {
                const uint32_t w0 = kw[gr][0], w1 = kw[gr][1];
                const uint2 b = ld_shared_v2(qb + gr * 512 + part * 8);
                if (part == 0) t[gr][0] = t[gr][1] = t[gr][2] = t[gr][3] = 0.f;
                mma_f16(t[gr], (w0 << 2) & m, (w1 << 2) & m, (w0 >> 6) & m, (w1 >> 6) & m, b.x, b.y);
              }
            }
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) {
              const float s0 = __low2float(as_half2(u4_word(p0, gr)));
              const float s1 = __low2float(as_half2(u4_word(p1, gr)));
              x[h][0] = fmaf(s0, t[gr][0], x[h][0]);
              x[h][1] = fmaf(s0, t[gr][1], x[h][1]);
              x[h][2] = fmaf(s1, t[gr][2], x[h][2]);
              x[h][3] = fmaf(s1, t[gr][3], x[h][3]);
            }
          }

          // ---- V's scales and minima: half g of each key's eight, for keys 2 t4, 2 t4 + 1 of the
          // two octets of both chunks ----
          uint32_t vp[2][2];
          ldsm_x4_trans(stV + lm_par, vp[0][0], vp[0][1], vp[1][0], vp[1][1]);
          if (!full) {   // keys that no query may see may hold anything
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                const int t0 = (c + h) * kChunk + 8 * o;
                const int lim = h == 0 || two ? Lc : 0;
                vp[h][o] &= (t0 + 2 * t4 < lim ? 0x0000ffffu : 0u) |
                            (t0 + 2 * t4 + 1 < lim ? 0xffff0000u : 0u);
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (t0 + g >= lim - a.q_len + 1 + ((qis >> (16 * e)) & 0xffff))
                    x[h][2 * o + e] = kNegInf;
              }
            // A NaN row of V is for the queries that see it only (a weight of 0 would not keep
            // it from the others): its parameters become 0, and the minima's sums of the rows that
            // see it NaN. Lane (g, t4) finds the first such key of half g, and holds the sums.
            uint32_t nan = 0;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int o = 0; o < 2; ++o) nan |= nan_halves(vp[h][o]);
            if (__any_sync(0xffffffffu, nan != 0)) {
              int at = 2 * kChunk;
#pragma unroll
              for (int h = 1; h >= 0; --h)
#pragma unroll
                for (int o = 1; o >= 0; --o) {
                  const uint32_t b = nan_halves(vp[h][o]);
                  if (b) at = h * kChunk + 8 * o + 2 * t4 + ((b & 0xffffu) ? 0 : 1);
                  vp[h][o] &= ~b;
                }
              at = min(at, __shfl_xor_sync(0xffffffffu, at, 1));
              at = min(at, __shfl_xor_sync(0xffffffffu, at, 2));
              at = min(at, __shfl_xor_sync(0xffffffffu, at, 4));   // scale or minimum
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (at < 2 * kChunk &&
                    c * kChunk + at < Lc - a.q_len + 1 + ((qis >> (16 * e)) & 0xffff))
                  oz[e] = __uint_as_float(0x7fffffffu);
            }
          }
          // even g: scales; bit 14 says 2 or more
          const bool wide = ((vp[0][0] | vp[0][1] | vp[1][0] | vp[1][1]) & wide_mask) != 0;

          // ---- softmax weights against the reference (exp2 domain) ----
          bool move = wide && shift != 0.f;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            move |= fmaxf(fmaxf(x[0][e], x[0][2 + e]), fmaxf(x[1][e], x[1][2 + e])) > thr[e];
          if (__any_sync(0xffffffffu, move)) {
            const float to = __any_sync(0xffffffffu, wide) ? 0.f : shift;
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(fmaxf(x[0][e], x[0][2 + e]), fmaxf(x[1][e], x[1][2 + e]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
              const float m_old = thr[e] == kNegInf ? kNegInf : -nm[e];
              const float m_new = fmaxf(m_old + (shift - to), mx * rsc[e] - to);
              alpha[e] = m_old == kNegInf ? 0.f : fast_exp2(m_old - m_new);
              if (m_new != kNegInf) {
                nm[e] = -m_new;
                thr[e] = (m_new + (to + kGrow)) / rsc[e];
              }
              tl[e] *= alpha[e];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              oz[i] *= alpha[i & 1];
#pragma unroll
              for (int gr = 0; gr < 4; ++gr) {
                ot[gr][0][i] *= alpha[i & 1];
                ot[gr][1][i] *= alpha[i & 1];
              }
            }
            shift = to;
          }
          uint32_t pb[2][2];   // P^T of chunk h as the B operand
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[h][e] = fast_exp2(fmaf(x[h][e], rsc[e], nm[e]));
              x[h][2 + e] = fast_exp2(fmaf(x[h][2 + e], rsc[e], nm[e]));
            }
            tl[e] += (x[0][e] + x[0][2 + e]) + (x[1][e] + x[1][2 + e]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int o = 0; o < 2; ++o)
              pb[h][o] = movmatrix_trans(pack_half2(x[h][2 * o], x[h][2 * o + 1]));

          // ---- O^T += V^T (P s)^T and the minima's sums ----
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t vb = stV + h * kTile;
            uint32_t vw[4][2];
            ldsm_x4_trans(vb + lm_codes, vw[0][0], vw[0][1], vw[1][0], vw[1][1]);
            ldsm_x4_trans(vb + lm_codes + 32, vw[2][0], vw[2][1], vw[3][0], vw[3][1]);
            mma_f16(oz, vp[h][0], 0u, vp[h][1], 0u, pb[h][0], pb[h][1]);
            const __half2 p0 = as_half2(pb[h][0]), p1 = as_half2(pb[h][1]);
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) {
              const __half2 s0 = as_half2(__shfl_sync(0xffffffffu, vp[h][0], 8 * gr + t4));
              const __half2 s1 = as_half2(__shfl_sync(0xffffffffu, vp[h][1], 8 * gr + t4));
              const uint32_t l0 = vw[gr][0] << 2, l1 = vw[gr][1] << 2;
              const uint32_t u0 = vw[gr][0] >> 6, u1 = vw[gr][1] >> 6;
              const __half2 b0 = __hmul2(p0, s0), b1 = __hmul2(p1, s1);
              // what the products' rounding left over (exact)
              const __half2 d0 = __hfma2(p0, s0, __hneg2(b0)), d1 = __hfma2(p1, s1, __hneg2(b1));
#pragma unroll
              for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const uint32_t m = i ? 0x03c003c0u : 0x003c003cu;
                  mma_f16(ot[gr][i], l0 & m, u0 & m, l1 & m, u1 & m,
                          half2_bits(part ? d0 : b0), half2_bits(part ? d1 : b1));
                }
            }
          }
          __syncwarp();                        // every lane has read the stage
          walk.load(a, cur, w, lane, stK, kv_policy);
          slot = slot + 1 == ND ? 0 : slot + 1;
        }
        // ---- the sums go to the warp's state buffer: row g of tile (gr, i) is dim 32 gr + 4 g + i,
        // row g + 8 dim 32 gr + 4 g + 2 + i ----
        if (!held && k >= 1 && !mbar_wait(bar_sfree, (k - 1) & 1, abort)) flag_timeout(a, abort);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float lv = tl[e];
          if (jp >= npair) {
            lv += __shfl_xor_sync(0xffffffffu, lv, 4);
            lv += __shfl_xor_sync(0xffffffffu, lv, 8);
            lv += __shfl_xor_sync(0xffffffffu, lv, 16);
          }
          float z[4];
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
            z[gr] = __shfl_sync(0xffffffffu, oz[e], 8 * gr + 4 + t4);
          const int r = r0 + e;
          const int at = w * a.R + r;
          const float m = thr[e] == kNegInf ? kNegInf : -nm[e];
          float keep = 0.f;   // what the earlier sums are worth against the present reference
          if (held && r < a.R && stM[at] != kNegInf) keep = fast_exp2(stM[at] - m);
          __syncwarp();
          if (r < a.R) {
            float4* row = reinterpret_cast<float4*>(stO + at * kSt + 4 * g);
#pragma unroll
            for (int gr = 0; gr < 4; ++gr) {
              float4 o = make_float4(fmaf(ot[gr][0][e], 0x1p22f, z[gr]),
                                     fmaf(ot[gr][1][e], 0x1p18f, z[gr]),
                                     fmaf(ot[gr][0][2 + e], 0x1p22f, z[gr]),
                                     fmaf(ot[gr][1][2 + e], 0x1p18f, z[gr]));
              if (held) {
                const float4 b = row[8 * gr];
                o.x = fmaf(b.x, keep, o.x);
                o.y = fmaf(b.y, keep, o.y);
                o.z = fmaf(b.z, keep, o.z);
                o.w = fmaf(b.w, keep, o.w);
              }
              row[8 * gr] = o;
            }
            if (g == 0) {
              stM[at] = m;
              stL[at] = lv;
            }
          }
        }
        __syncwarp();
        held = true;
      } while (jp < npair);
      j += npair;
      if (lane == 0) mbar_arrive(bar_qempty + qs * 8);
      if (lane == 0) mbar_arrive(bar_sdone);
      set_last(s, k);
      ++k;
      has = cur.next(s);
    }
    cp_async_wait<0>();
  }

  // ---- end of the slice ----
  if (last.k >= 0)
    finish_slice<NCS, kSeg4, NCW, 1>(a, last, pre, per, smem, L::kQ, stO, stM, stL, npend_s,
                                      fast_s, warp < NCW ? tid : tid - 32);
}

// ---------------------------------------------------------------------------------------------
// Host side.

template <int NCS, int RS, int ND, int MINB, bool APPEND>
Variant variant4() {
  return Variant{reinterpret_cast<const void*>(&decode_int4_kernel<NCS, RS, ND, MINB, APPEND>), RS,
                 false, (NCS * RS + 2) * 32, &Smem4<NCS, RS, ND>::bytes};
}

// The variant for R query rows. Four consumer warps a CTA and two CTAs for up to 16 rows, one CTA
// of 12 beyond (a multiple of four of them per SM: one of its four schedulers takes every fourth
// warp). Measured against others that fit, us (64 sequences of 16 to 2048 tokens, 2 kv heads; 16 of
// 4096 tokens, 8 kv heads):
//   16 rows   <2, 2, 3, 2> 20.4 / 43.4, <4, 2, 3, 1> 20.7 / 46.8, <6, 2, 2, 1> 22.3 / 43.3
//   24 rows   <4, 3, 2, 1> 25.2 / 59.6, <3, 3, 3, 1> 27.5 / 69.6
//   32 rows   <3, 4, 2, 1> 29.6 / 73.7, <2, 4, 3, 1> 30.8 / 78.6
// Up to 8 rows, 12 warps in one CTA keep more in flight than two CTAs of 4, but hand a segment over
// only once per SM and merge 12 states for it. That pays where a CTA has a segment or two, of many
// stages: no more units than SMs, tables for 4096 tokens or more (the lengths are on the GPU; a few
// short contexts in tables as wide as a server's capacity pay for that). <12, 1, 2, 1> against
// <4, 1, 3, 2>: 16 sequences of 4096 tokens with 8 kv heads 25.7 against 27.0, one of 65536 30.8
// against 35.8, two of 131072 with one kv head 34.1 against 41.1; but two of about 70 tokens 7.3
// against 6.5, and 512 units of mixed lengths 65 against 51.
template <bool APPEND>
Variant choose4(int R, bool few_long) {
  return R <= 8    ? (few_long ? variant4<12, 1, 2, 1, APPEND>() : variant4<4, 1, 3, 2, APPEND>())
         : R <= 16 ? variant4<2, 2, 3, 2, APPEND>()
         : R <= 24 ? variant4<4, 3, 2, 1, APPEND>()
                   : variant4<3, 4, 2, 1, APPEND>();
}

int launch_decode_int4(void* out, const void* q, const void* k_new, const void* v_new,
                       const void* k_cache, const void* v_cache, int num_blocks,
                       const int32_t* block_tables, int max_blocks, const int32_t* context_lens,
                       int num_seqs, int q_len, int Hq, int Hkv, int head_dim, int block_size,
                       float scale, void* workspace, size_t workspace_bytes, bool append,
                       pkv_stream_t stream) {
  if (num_seqs < 0 || q_len < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || head_dim != kD ||
      !valid_block_size(block_size) || num_blocks < 0 || max_blocks < 0 ||
      Hkv > (1 << 20))   // a stage's place is packed as head << 8 | row
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
  // all chunk indices and pool rows fit in int32
  const int64_t rows = static_cast<int64_t>(num_blocks) * Hkv * block_size;
  const int64_t max_ctx = static_cast<int64_t>(max_blocks) * block_size;
  if (rows >= (1ll << 31) || max_ctx >= (1ll << 31) ||
      static_cast<int64_t>(num_seqs) * Hkv * ((max_ctx + kChunk - 1) / kChunk + kSeg4) >=
          (1ll << 30))
    return PKV_EINVAL;
  if (num_blocks == 0) return PKV_EINVAL;
  const WsLayout ws = ws_layout(num_seqs, Hkv, R, workspace_bytes);
  if (workspace_bytes < ws.total) return PKV_ENOSPC;

  const int newkv_bytes = append ? 2 * q_len * kNewRow : 0;
  const bool few_long = num_seqs * Hkv <= sm_count() && max_ctx >= 4096;
  Variant v = append ? choose4<true>(R, few_long) : choose4<false>(R, few_long);
  size_t smem = v.smem(R, num_seqs, newkv_bytes);
  if (append && smem > kMaxSmem) {   // thousands of sequences with 8 and more new tokens each
    v = variant4<2, 4, 2, 1, true>();
    smem = v.smem(R, num_seqs, newkv_bytes);
  }
  if (smem > kMaxSmem) return PKV_EINVAL;
  int status = PKV_OK;
  const int grid = grid_size(v, smem, &status);
  if (!grid) return status != PKV_OK ? status : PKV_EINVAL;

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

  const __half* q_in = static_cast<const __half*>(q);
  void* params[2] = {&args, &q_in};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(v.threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // The plain form waits for the kernel before it as its first step: its CTAs only take their places
  // early (one sequence of 101 tokens 6.5 -> 5.8 us in a row, 16 of 4096 25.4 -> 24.9).
  cfg.numAttrs = (!append || early_start_enabled()) ? 1 : 0;
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
