// pkv_decode_common.cuh -- what the paged decode kernels share (fp16, E4M3 and 4-bit caches): the
// stream of 16-token chunks and its slices, the merges of per-warp states and of split units'
// partials, the query loads, and the host side's workspace, grid and tensor-map helpers. The
// design notes are at the top of pkv_decode.cu.
#pragma once

#include <cuda_fp16.h>

#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>

#include "pkv_device.cuh"
#include "pkv_internal.h"

namespace pkv {

// Whether the fused-append calls may start while the kernel before them finishes
// (programmatic dependent launch); process-wide, read at each launch.
bool early_start_enabled();

namespace {

constexpr int kD = 128;                       // head_dim
constexpr int kChunk = 16;                    // tokens per pipeline stage
constexpr int kMaxCtasPerSm = 4;              // bounds the grid, hence the workspace
constexpr int kMaxSeqs = 4096;
// Per-segment cost in chunk equivalents: in the stream that is cut into equal slices, every
// non-empty unit is preceded by this many empty positions, so a CTA whose slice holds many
// short units (each one a segment: queries, hand-off, merge) gets fewer chunks.
#ifndef PKV_SEGMENT_COST
#define PKV_SEGMENT_COST 2
#endif
constexpr int kSegCost = PKV_SEGMENT_COST;
// Row stride (floats) of the per-warp output states in shared memory: 8 floats of padding put
// the 8 rows a warp's float2 stores touch at once in different banks.
constexpr int kSt = kD + 8;
constexpr float kNegInf = -__builtin_huge_valf();
// How long the CTA that merges a split unit waits for the unit's other partials before it
// falls back to announcing its own (normally they are in within microseconds).
#ifndef PKV_MERGE_WAIT_NS
#define PKV_MERGE_WAIT_NS 200000
#endif
constexpr uint64_t kMergeWaitNs = PKV_MERGE_WAIT_NS;

struct DecodeArgs {
  __half* out;
  const int32_t* block_tables;
  const int32_t* context_lens;  // paged
  const int64_t* logical_len;   // ring: L
  const int64_t* high_water;    // ring: hw
  const float* rope;            // ring: [sink + window][64][2] (cos, sin)
  float* part_o;                // [2 * grid][R][128]
  float* part_ml;               // [2 * grid][R][4]: m, l, 0, 0 (16-byte rows)
  int* counters;                // [num_seqs * Hkv]
  unsigned int* err;
  int num_blocks, max_blocks, num_seqs, q_len, Hq, Hkv, G, R;
  int block_size, bs_shift;     // bs_shift = log2(block_size / 16)
  int sink, window;
  float scale_log2;             // scale * log2(e)
  // fused append: this step's new K/V rows [B*q_len][Hkv][128] and the layer's pools
  const __half* k_new;
  const __half* v_new;
  __half* k_pool;
  __half* v_pool;
  // FP8 (E4M3) cache: per kv head scales of K and V (value = code * scale)
  const float* k_scale;
  const float* v_scale;
};

__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Seg {
  int b, h, c0, c1, nb;  // chunks [c0, c1) of unit (b, h), which has nb chunks
  int x;                 // global stream index of chunk c0
};

// The stream: unit (b, h) of a sequence with nb > 0 chunks per kv head occupies nb + kSegCost
// positions, kSegCost empty ones and then its chunks; pre[b] is the length (per kv head) of the
// sequences before b, so the unit starts at pre[b] * Hkv + h * (nb + kSegCost). A CTA's slice
// [a, end) of the stream gives it segments: the runs of chunks of one unit inside the slice.
// (SEG: the kernel's kSegCost.)
template <int SEG = kSegCost>
__device__ __forceinline__ int unit_first(const int* pre, int Hkv, int b, int h, int nb) {
  return pre[b] * Hkv + h * (nb + SEG) + SEG;   // position of the unit's chunk 0
}

template <int SEG = kSegCost>
struct CursorT {
  const int* pre;
  int B, Hkv, end;

  __device__ __forceinline__ bool first(int a, Seg& s) const {
    if (a >= end) return false;
    int lo = 0, hi = B - 1;  // largest b with pre[b] * Hkv <= a (a sequence with chunks)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * Hkv <= a) lo = mid; else hi = mid - 1;
    }
    const int vl = pre[lo + 1] - pre[lo];
    const int off = a - pre[lo] * Hkv;
    const int h = off / vl, o = off - h * vl;
    const int ustart = a - o;
    const int x0 = ustart + SEG + max(o - SEG, 0);   // first chunk in the slice
    if (x0 >= end) return false;   // the slice ends before the unit's first chunk
    s.b = lo;
    s.h = h;
    s.nb = vl - SEG;
    s.c0 = x0 - ustart - SEG;
    s.c1 = min(s.nb, end - ustart - SEG);
    s.x = x0;
    return true;
  }
  __device__ __forceinline__ bool next(Seg& s) const {
    // the next unit's first chunk, if the slice reaches it (then this segment ended its unit)
    const int u2 = s.x - s.c0 + s.nb;
    if (u2 + SEG >= end) return false;
    if (++s.h == Hkv) {
      s.h = 0;
      do { ++s.b; } while (pre[s.b + 1] == pre[s.b]);
    }
    s.nb = pre[s.b + 1] - pre[s.b] - SEG;
    s.c0 = 0;
    s.c1 = min(s.nb, end - (u2 + SEG));
    s.x = u2 + SEG;
    return true;
  }
};
using Cursor = CursorT<>;

__device__ __forceinline__ void flag_timeout(const DecodeArgs& a, volatile int* abort) {
  atomicOr(a.err, PKV_DEVERR_TIMEOUT);
  *abort = 1;
}

// Inclusive scan of pre[1 .. B] in place by one warp (contiguous slices per lane + shuffle scan).
__device__ __forceinline__ void scan_chunks(int* pre, int B, int lane) {
  const int per_lane = (B + 31) / 32;
  const int lo = min(B, lane * per_lane), hi = min(B, lo + per_lane);
  int sum = 0;
  for (int b = lo; b < hi; ++b) sum += pre[b + 1];
  int incl = sum;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  int run = incl - sum;
  for (int b = lo; b < hi; ++b) {
    run += pre[b + 1];
    pre[b + 1] = run;
  }
}

// Sync of the threads taking part in a merge: one warp, or a named barrier over NT threads.
template <int NT>
__device__ __forceinline__ void merge_sync() {
  if (NT == 32) __syncwarp();
  else named_barrier_sync(2, NT);
}

// Output row r (= query token qi, head g of the group) of unit (b, h): pointer to its 128 halves.
__device__ __forceinline__ __half* out_row(const DecodeArgs& a, int b, int h, int r) {
  const int qi = r / a.G, gg = r - qi * a.G;
  return a.out + ((static_cast<int64_t>(b) * a.q_len + qi) * a.Hq + h * a.G + gg) * kD;
}

__device__ __forceinline__ void store_half4(__half* dst, float4 v) {
  uint2 u;
  u.x = pack_half2(v.x, v.y);
  u.y = pack_half2(v.z, v.w);
  *reinterpret_cast<uint2*>(dst) = u;
}

// Weights of one row of a segment's per-warp states: w[ww] = 2^(m_ww - m) / l, with m the
// row's max and l = sum_ww l_ww 2^(m_ww - m); returns m and l for the partial.
template <int NCW>
__device__ __forceinline__ void row_weights(const float* m_s, const float* l_s, int R, int r,
                                            float (&w)[NCW], float& row_m, float& row_l) {
  row_m = kNegInf;
#pragma unroll
  for (int ww = 0; ww < NCW; ++ww) {
    w[ww] = m_s[ww * R + r];
    row_m = fmaxf(row_m, w[ww]);
  }
  row_l = 0.f;
#pragma unroll
  for (int ww = 0; ww < NCW; ++ww) {
    w[ww] = row_m == kNegInf ? 0.f : fast_exp2(w[ww] - row_m);
    row_l += l_s[ww * R + r] * w[ww];
  }
  const float inv = row_l > 0.f ? 1.f / row_l : 0.f;
#pragma unroll
  for (int ww = 0; ww < NCW; ++ww) w[ww] *= inv;
}

// Merge of one segment's per-warp states (o: [NCW][R] rows of kSt floats, unnormalised; m and
// l: [NCW][R]) into the unit's output (complete segment) or its normalised partial (split
// unit: rows of 128
// floats at po, rows of (m, l, 0, 0) at pml; global or shared memory), by NT threads
// t = 0..NT-1. Each thread owns 4 consecutive dims of a row (float4 in, 8 bytes out). One warp
// (NT == 32) forms each row's weights once, in lane r, and shares them by shuffle; a larger
// group has each thread form its own row's weights (the same arithmetic), with no barrier.
template <int NCW, int NT>
__device__ __forceinline__ void merge_segment(const DecodeArgs& a, const float* o_s,
                                              const float* m_s, const float* l_s, int b, int h,
                                              bool complete, float* po, float* pml, int t) {
  const int R = a.R;
  float w_own[NCW], m_own = 0.f, l_own = 0.f;
  if (NT == 32 && t < R) {
    row_weights<NCW>(m_s, l_s, R, t, w_own, m_own, l_own);
    if (!complete) *reinterpret_cast<float4*>(pml + t * 4) = make_float4(m_own, l_own, 0.f, 0.f);
  }
#pragma unroll 1
  for (int gi = t; gi < R * 32; gi += NT) {
    const int r = gi >> 5, c4 = gi & 31;
    float w[NCW];
    if (NT == 32) {
#pragma unroll
      for (int ww = 0; ww < NCW; ++ww) w[ww] = __shfl_sync(0xffffffffu, w_own[ww], r);
    } else {
      float row_m, row_l;
      row_weights<NCW>(m_s, l_s, R, r, w, row_m, row_l);
      if (!complete && c4 == 0)
        *reinterpret_cast<float4*>(pml + r * 4) = make_float4(row_m, row_l, 0.f, 0.f);
    }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int ww = 0; ww < NCW; ++ww) {
      const float4 v = reinterpret_cast<const float4*>(o_s + (ww * R + r) * kSt)[c4];
      const float wt = w[ww];
      acc.x += wt * v.x; acc.y += wt * v.y; acc.z += wt * v.z; acc.w += wt * v.w;
    }
    if (complete)
      store_half4(out_row(a, b, h, r) + c4 * 4, acc);
    else
      reinterpret_cast<float4*>(po + r * kD)[c4] = acc;
  }
}

// The same merge of a segment's per-warp states by NT > 32 threads (the CTA's last segment, at
// the end of the launch): one thread per row forms the row's weights once and leaves them in
// the row's padding (floats kD.. of each state row), then every thread sums its own 4 dims.
template <int NCW, int NT>
__device__ __forceinline__ void merge_segment_wide(const DecodeArgs& a, float* o_s,
                                                   const float* m_s, const float* l_s, int b,
                                                   int h, bool complete, float* po, float* pml,
                                                   int t) {
  const int R = a.R;
  if (t < R) {
    float w[NCW], row_m, row_l;
    row_weights<NCW>(m_s, l_s, R, t, w, row_m, row_l);
#pragma unroll
    for (int ww = 0; ww < NCW; ++ww) o_s[(ww * R + t) * kSt + kD] = w[ww];
    if (!complete) *reinterpret_cast<float4*>(pml + t * 4) = make_float4(row_m, row_l, 0.f, 0.f);
  }
  named_barrier_sync(2, NT);
#pragma unroll 1
  for (int gi = t; gi < R * 32; gi += NT) {
    const int r = gi >> 5, c4 = gi & 31;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int ww = 0; ww < NCW; ++ww) {
      const float* row = o_s + (ww * R + r) * kSt;
      const float4 v = reinterpret_cast<const float4*>(row)[c4];
      const float wt = row[kD];
      acc.x += wt * v.x; acc.y += wt * v.y; acc.z += wt * v.z; acc.w += wt * v.w;
    }
    if (complete)
      store_half4(out_row(a, b, h, r) + c4 * 4, acc);
    else
      reinterpret_cast<float4*>(po + r * kD)[c4] = acc;
  }
}

// Where merge_unit stages partials in the (free) pipeline stage memory.
struct MergeStage {
  float* accv;    // [R][128] running output
  float* rowml;   // [2][R][2] running (max, sum), then [R][2] (scale of the running output,
                  // 1 / sum in the last batch) and [R][2] spare (keeps `so` 16-byte aligned)
  float* so;      // [PB][R][128] partials' o
  float* sml;     // [PB][R][4] partials' (m, l, weight, -)
  int PB;         // partials per batch (>= 2)
  __device__ MergeStage(uint8_t* stage_mem, int stage_bytes, int R) {
    accv = reinterpret_cast<float*>(stage_mem);
    rowml = accv + R * kD;
    PB = (stage_bytes - (R * kD + 8 * R) * 4) / (R * (kD + 4) * 4);
    so = rowml + 8 * R;
    sml = so + PB * R * kD;
  }
};

// Merge of a split unit's partials, run cooperatively by NT threads of the merging CTA (the one
// holding the unit's first chunk, or the last to arrive on the unit's counter), after its whole
// slice is done (so its pipeline stages are free).
// Partial p (in slice order) holds per row its max m_p, sum l_p and normalised output o_p; the
// result is sum_p o_p w_p / sum_p w_p with w_p = l_p 2^(m_p - M), M = max_p m_p, formed in slice
// order. The partials are copied into the stage memory with cp.async (as many per batch as fit,
// usually all: one round trip to L2); then one thread per row forms the row's weights, and every
// thread sums its own 4 output dims over the partials and divides by the row's sum. Each pass
// takes few dependent shared-memory round trips: this runs once per CTA at the end of the
// launch, where its latency is on the critical path.
// own >= 0: the unit's first partial (own == cf, the merging CTA's own) is already in the
// staging area, at index 0 of the first batch; it is not copied from the workspace.
template <int NT, int SEG = kSegCost>
__device__ __forceinline__ void merge_unit(const DecodeArgs& a, int b, int h, int nb,
                                           const int* pre, int per, uint8_t* stage_mem,
                                           int stage_bytes, int t, int own = -1) {
  const int R = a.R;
  const int ua = unit_first<SEG>(pre, a.Hkv, b, h, nb);
  const int cf = ua / per, cl = (ua + nb - 1) / per;
  // the unit is not the first segment of slice cf if that slice reaches back into the unit
  // before it (whose last chunk is the position just before this unit's empty ones)
  const bool first_odd = cf * per < ua - SEG;
  const MergeStage ms(stage_mem, stage_bytes, R);
  float* accv = ms.accv;
  float* rowml = ms.rowml;
  const int PB = ms.PB;
  float* so = ms.so;
  float* sml = ms.sml;   // per partial and row: m, l, then this batch's weight
  const uint32_t so_s = smem_u32(so), sml_s = smem_u32(sml);
  const int o_vec = R * kD / 4;                            // 16-byte pieces of one partial's o
  int batch = 0;
#pragma unroll 1
  for (int base = cf; base <= cl; base += PB, ++batch) {
    const int nbp = min(PB, cl - base + 1);
    const bool last_batch = base + PB > cl;
    merge_sync<NT>();                      // previous batch fully used
#pragma unroll 1
    for (int p = 0; p < nbp; ++p) {
      const int cc = base + p;
      if (cc == own) continue;
      const int64_t sl = 2 * cc + ((cc == cf && first_odd) ? 1 : 0);
      const float* src = a.part_o + sl * R * kD;
      const uint32_t dst = so_s + p * R * kD * 4;
      for (int i = t; i < o_vec; i += NT) cp_async_16(dst + i * 16, src + i * 4);
      if (t < R) cp_async_16(sml_s + (p * R + t) * 16, a.part_ml + (sl * R + t) * 4);
    }
    cp_async_wait_all();
    merge_sync<NT>();
    float* rsc = rowml + 4 * R;
    if (t < R) {
      // The row's (m, l) pairs are read into registers kRegP at a time (one shared-memory round
      // trip per group; a single one in the usual case of at most kRegP partials) before any
      // weight is written back.
      constexpr int kRegP = 8;
      const float* rin = rowml + (batch & 1) * 2 * R;
      float* rout = rowml + ((batch + 1) & 1) * 2 * R;
      const float M0 = batch ? rin[2 * t] : kNegInf;
      const float L0 = batch ? rin[2 * t + 1] : 0.f;
      float2 mlr[kRegP];
      float M = M0;
#pragma unroll 1
      for (int p0 = 0; p0 < nbp; p0 += kRegP) {
#pragma unroll
        for (int i = 0; i < kRegP; ++i) {
          const int p = p0 + i;
          mlr[i] = p < nbp ? *reinterpret_cast<const float2*>(sml + (p * R + t) * 4)
                           : make_float2(kNegInf, 0.f);
          M = fmaxf(M, mlr[i].x);
        }
      }
      const float sc = (M0 == kNegInf || M == kNegInf) ? 0.f : fast_exp2(M0 - M);
      float L = L0 * sc;
#pragma unroll 1
      for (int p0 = 0; p0 < nbp; p0 += kRegP) {
        if (nbp > kRegP) {
#pragma unroll
          for (int i = 0; i < kRegP; ++i) {
            const int p = p0 + i;
            mlr[i] = p < nbp ? *reinterpret_cast<const float2*>(sml + (p * R + t) * 4)
                             : make_float2(kNegInf, 0.f);
          }
        }
#pragma unroll
        for (int i = 0; i < kRegP; ++i) {
          const int p = p0 + i;
          const float wp = mlr[i].x == kNegInf ? 0.f : mlr[i].y * fast_exp2(mlr[i].x - M);
          L += wp;
          if (p < nbp) sml[(p * R + t) * 4 + 2] = wp;
        }
      }
      const float inv = !last_batch ? 1.f : (L > 0.f ? 1.f / L : 0.f);
      *reinterpret_cast<float2*>(rsc + 2 * t) = make_float2(sc, inv);
      rout[2 * t] = M;
      rout[2 * t + 1] = L;
    }
    merge_sync<NT>();
#pragma unroll 1
    for (int gi = t; gi < R * 32; gi += NT) {
      const int r = gi >> 5, c4 = gi & 31;
      const float2 si = *reinterpret_cast<const float2*>(rsc + 2 * r);
      float4 V = make_float4(0.f, 0.f, 0.f, 0.f);
      if (batch) {
        V = reinterpret_cast<const float4*>(accv)[gi];
        V.x *= si.x; V.y *= si.x; V.z *= si.x; V.w *= si.x;
      }
#pragma unroll 4
      for (int p = 0; p < nbp; ++p) {
        const float wp = sml[(p * R + r) * 4 + 2];
        const float4 o4 = reinterpret_cast<const float4*>(so + (p * R + r) * kD)[c4];
        V.x += wp * o4.x; V.y += wp * o4.y; V.z += wp * o4.z; V.w += wp * o4.w;
      }
      if (last_batch) {
        V.x *= si.y; V.y *= si.y; V.z *= si.y; V.w *= si.y;
        store_half4(out_row(a, b, h, r) + c4 * 4, V);
      } else {
        reinterpret_cast<float4*>(accv)[gi] = V;
      }
    }
  }
  if (t == 0) a.counters[b * a.Hkv + h] = 0;
  merge_sync<NT>();                        // stage memory free for the next merge
}

// The CTA's last segment, merged at the end by consumers and epilogue together.
struct LastSeg {
  int k, b, h, nb, slot;   // segment number in the CTA (-1: none), unit, its partial's slot
  bool complete, head;     // the whole unit / its first chunk

  template <int SEG>
  __device__ __forceinline__ static LastSeg of(const CursorT<SEG>& cur, int begin) {
    LastSeg ls{-1, 0, 0, 0, 0, true, false};
    Seg s;
    bool has = cur.first(begin, s);
    int kk = 0;
    while (has) {
      ls.k = kk;
      ls.b = s.b; ls.h = s.h; ls.nb = s.nb;
      ls.complete = (s.c0 == 0 && s.c1 == s.nb);
      ls.head = s.c0 == 0;
      ls.slot = 2 * blockIdx.x + (kk == 0 ? 0 : 1);
      ++kk;
      has = cur.next(s);
    }
    return ls;
  }
};

// End of the slice: the consumers and the epilogue warp (kNE threads, dense index t) merge the
// last segment, then any split unit whose last partial arrived from this CTA (the producer has
// left). smem: the CTA's stage memory, stage_bytes of it; stO, stM, stL: the per-warp states, SB
// buffers of NCW states; npend_s, fast_s: the CTA's pending merges and the outcome of the wait.
// WARPS: consumer warps (more than NCW where several hold different rows of one state).
template <int NCW, int SEG = kSegCost, int WARPS = NCW, int SB = 2>
__device__ __forceinline__ void finish_slice(const DecodeArgs& a, const LastSeg& ls,
                                             const int* pre, int per, uint8_t* smem,
                                             int stage_bytes, float* stO, const float* stM,
                                             const float* stL, int* npend_s,
                                             volatile int* fast_s, int t) {
  constexpr int kNE = (WARPS + 1) * 32;
  const int ua = unit_first<SEG>(pre, a.Hkv, ls.b, ls.h, ls.nb);
  const int parts = (ua + ls.nb - 1) / per - ua / per + 1;
  const MergeStage ms(smem, stage_bytes, a.R);
  named_barrier_sync(2, kNE);                  // last states written, earlier segments merged
  const int sb = ls.k % SB;
  float* so_w = stO + sb * NCW * a.R * kSt;
  const float* sm_w = stM + sb * NCW * a.R;
  const float* sl_w = stL + sb * NCW * a.R;
  int* counter = a.counters + ls.b * a.Hkv + ls.h;
  // A split unit is merged by the CTA that holds its first chunk, the one whose last segment
  // is the unit's head. That CTA keeps its own partial in the staging area (it never goes out
  // to the workspace and back) and waits until the other CTAs have announced theirs; most of
  // them finished that work long before (a unit's other parts are the first segments of
  // later CTAs, or whole slices). The wait is bounded in time: if the other parts are not in
  // (their CTAs may not be resident yet, e.g. when other work holds the GPU), the CTA
  // announces its partial like the others and the last to arrive merges. Either way the
  // partials and their order are the same, so the result does not depend on the path.
  bool merged = false;
  if (!ls.complete && ls.head) {
    merge_segment_wide<NCW, kNE>(a, so_w, sm_w, sl_w, ls.b, ls.h, false, ms.so, ms.sml,
                                 t);
    if (t == 0) {
      const uint64_t t_end = global_time_ns() + kMergeWaitNs;
      int ok = 0;
      do {
        if (ld_acquire_gpu(counter) == parts - 1) { ok = 1; break; }
      } while (global_time_ns() < t_end);
      *fast_s = ok;
    }
    named_barrier_sync(2, kNE);
    merged = *fast_s;
    if (merged) {
      merge_unit<kNE, SEG>(a, ls.b, ls.h, ls.nb, pre, per, smem, stage_bytes, t,
                      blockIdx.x);
    } else {
      // give up waiting: the staged partial goes to the workspace like the others'
      float* po = a.part_o + static_cast<int64_t>(ls.slot) * a.R * kD;
      float* pml = a.part_ml + static_cast<int64_t>(ls.slot) * a.R * 4;
      for (int i = t; i < a.R * 32; i += kNE)
        reinterpret_cast<float4*>(po)[i] = reinterpret_cast<const float4*>(ms.so)[i];
      if (t < a.R) reinterpret_cast<float4*>(pml)[t] = reinterpret_cast<const float4*>(ms.sml)[t];
    }
  } else {
    merge_segment_wide<NCW, kNE>(a, so_w, sm_w, sl_w, ls.b, ls.h, ls.complete,
                                 a.part_o + static_cast<int64_t>(ls.slot) * a.R * kD,
                                 a.part_ml + static_cast<int64_t>(ls.slot) * a.R * 4, t);
  }
  if (!ls.complete && !merged) {
    named_barrier_sync(2, kNE);                // partial written by every thread
    if (t == 0 && atomic_add_acq_rel(counter, 1) == parts - 1) {
      const int n = *npend_s;
      npend_s[1 + 3 * n] = ls.b;
      npend_s[2 + 3 * n] = ls.h;
      npend_s[3 + 3 * n] = ls.nb;
      *npend_s = n + 1;
    }
  }
  named_barrier_sync(2, kNE);
  const int np = *npend_s;
  // every chunk of this CTA's slice has been consumed, so the stage memory is free
#pragma unroll 1
  for (int i = 0; i < np; ++i)
    merge_unit<kNE, SEG>(a, npend_s[1 + 3 * i], npend_s[2 + 3 * i], npend_s[3 + 3 * i], pre, per,
                    smem, stage_bytes, t);
}

// Online softmax: a row's running maximum m is brought up to date (a warp-wide reduction and,
// if it grew, a rescale of l and O) only in a step where one of the row's scores exceeds m by
// more than this many powers of two. Any m with every score <= m + kLazyLog2 gives the same
// softmax: the weights exp2(x - m) stay <= 256, exact to fp16's relative precision, and the
// final 1 / l and the split merges use the same m as l and O.
constexpr float kLazyLog2 = 8.f;

// Word i (0-3) of a 16-byte vector (i a compile-time constant after unrolling).
__device__ __forceinline__ uint32_t u4_word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// Requests segment kk's queries (and, fused append, its new K/V rows) into query buffer kk & 1,
// completing on that buffer's full barrier; waits first until the consumers have released the
// buffer's previous use. One thread.
template <class L, bool APPEND>
__device__ __forceinline__ void issue_queries(const DecodeArgs& a, const CUtensorMap* tmQ,
                                              uint32_t sbase, int B, const Seg& sg, int kk,
                                              volatile int* abort) {
  const uint32_t bar_qfull = sbase + L::kBars + 2 * L::kNST * 8;
  const uint32_t bar_qempty = bar_qfull + 2 * 8;
  const int qs = kk & 1;
  if (kk >= 2 && !mbar_wait(bar_qempty + qs * 8, ((kk >> 1) - 1) & 1, abort))
    flag_timeout(a, abort);
  mbar_arrive_expect_tx(bar_qfull + qs * 8, a.R * 256 + (APPEND ? a.q_len * 512 : 0));
  const uint32_t qdst = sbase + L::kQ + qs * L::kQBuf;
  tma_load_3d(qdst, tmQ, 0, sg.h * a.G, sg.b * a.q_len, bar_qfull + qs * 8);
  tma_load_3d(qdst + L::kQHalf, tmQ, 64, sg.h * a.G, sg.b * a.q_len, bar_qfull + qs * 8);
  if (APPEND) {
    const uint32_t nkv = sbase + L::newkv_off(a.R, B) + qs * a.q_len * 512;
    for (int i = 0; i < a.q_len; ++i) {
      const int64_t row = (static_cast<int64_t>(sg.b) * a.q_len + i) * a.Hkv + sg.h;
      bulk_load(nkv + i * 512, a.k_new + row * kD, 256, bar_qfull + qs * 8);
      bulk_load(nkv + i * 512 + 256, a.v_new + row * kD, 256, bar_qfull + qs * 8);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Host side.

struct Variant {
  const void* fn;
  int mt;
  bool ring;
  int threads;
  size_t (*smem)(int R, int B, int newkv_bytes);
};

// Persistent grid for a variant: SM count x resident CTAs (capped), cached per device/size.
inline int grid_size(const Variant& v, size_t smem, int* status) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, size_t>, int> cache;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) { *status = cuda_status(e); return 0; }
  std::lock_guard<std::mutex> lock(mu);
  auto key = std::make_tuple(dev, v.fn, smem);
  auto it = cache.find(key);
  if (it != cache.end()) return it->second;
  // The attribute is per kernel, not per launch: raise it once to the device's limit, so that
  // a launch with a smaller size never lowers it under a later, larger one (whose grid is
  // already cached).
  int limit = 0;
  e = cudaDeviceGetAttribute(&limit, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess && static_cast<size_t>(limit) < smem) e = cudaErrorInvalidValue;
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(v.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, limit);
  int occ = 0;
  if (e == cudaSuccess)
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, v.fn, v.threads, smem);
  if (e != cudaSuccess) { *status = cuda_status(e); return 0; }
  if (occ < 1) { *status = PKV_EINVAL; return 0; }
  const int grid = sm_count() * std::min(occ, kMaxCtasPerSm);
  cache[key] = grid;
  return grid;
}

struct WsLayout {
  size_t counters, counter_bytes, part_ml, part_o, total;
};

// Counters from the workspace's start, partials up to its end: a workspace of `bytes` that serves
// calls of several sizes keeps the counters, which every call leaves zero, apart from the
// partials, which it does not.
inline WsLayout ws_layout(int num_seqs, int Hkv, int R, size_t bytes) {
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t partials = static_cast<size_t>(2) * sm_count() * kMaxCtasPerSm;
  const size_t ml = up(partials * R * 4 * sizeof(float)), o = up(partials * R * kD * sizeof(float));
  WsLayout w;
  w.counters = 0;
  w.counter_bytes = up(static_cast<size_t>(num_seqs) * Hkv * sizeof(int));
  w.total = w.counter_bytes + ml + o;
  w.part_o = std::max(w.total, bytes & ~static_cast<size_t>(255)) - o;
  w.part_ml = w.part_o - ml;
  return w;
}

inline int encode(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box,
                  CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
  auto fn = tensor_map_encoder();
  if (!fn) return PKV_ECUDA_BASE - static_cast<int>(cudaErrorNotSupported);
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, type, rank, const_cast<void*>(base), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? PKV_OK : PKV_EINVAL;
}

}  // namespace
}  // namespace pkv
