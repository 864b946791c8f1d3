"""The 8-bit cache's oracle (test infrastructure): append, widening, attention and block selection,
in whole numbers and fp64 (numpy).

A block of one kv head holds codes u [bs, 128] of K and of V (uint8), a scale each (a power of two)
and, for K, the least and the greatest code per channel; value = scale * (u - 128).
"""
from __future__ import annotations

import math

import numpy as np

D, LOW, HIGH = 128, -30, 9


def scale_of(x: np.ndarray) -> float:
    """The least power of two s within 2^LOW .. 2^HIGH with |x| <= 127 s; NaN if x has a NaN or an
    infinity."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return math.nan
    top, e = float(np.abs(x).max(initial=0.0)), LOW
    while e < HIGH and top > 127 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def codes_of(x: np.ndarray, s: float) -> np.ndarray:
    """Codes (uint8) at scale s; zeros at a NaN scale."""
    if math.isnan(s):
        return np.full(np.shape(x), 128, np.uint8)
    return (np.clip(np.rint(np.asarray(x, np.float64) / s), -127, 127) + 128).astype(np.uint8)


def moved(u: np.ndarray, old: float, s: float) -> np.ndarray:
    """Codes of scale `old` on the grid of s; zeros where s is NaN."""
    if math.isnan(s):
        return np.full(u.shape, 128, np.uint8)
    return (np.rint((u.astype(np.float64) - 128) * (old / s)) + 128).astype(np.uint8)


def append(k, v, slots, k_pool, v_pool, scales, bounds=None):
    """Rows k, v fp16 [T, Hkv, 128] into the pools [NB, Hkv, bs, 128] in place."""
    nb, hkv, bs, _ = k_pool.shape
    slots = np.asarray(slots)
    good = (slots >= 0) & (slots < nb * bs)
    for blk in np.unique(slots[good] // bs):
        at = np.nonzero(good & (slots // bs == blk))[0]
        off = slots[at] % bs
        fresh = bool((off == 0).any())
        for h in range(hkv):
            for i, (x, pool) in enumerate(((k, k_pool), (v, v_pool))):
                need, old = scale_of(x[at, h]), 0.0 if fresh else float(scales[blk, h, i])
                s = math.nan if math.isnan(need) or math.isnan(old) else max(need, old)
                block = pool[blk, h]
                if fresh:
                    block[:] = 128
                else:
                    block[:] = moved(block, old, s)
                new = codes_of(x[at, h], s)
                block[off] = new
                if i == 0 and bounds is not None:
                    lo, hi = new.min(0), new.max(0)
                    if not fresh:
                        lo = np.minimum(lo, moved(bounds[blk, h, 0], old, s))
                        hi = np.maximum(hi, moved(bounds[blk, h, 1], old, s))
                    bounds[blk, h, 0], bounds[blk, h, 1] = lo, hi
                scales[blk, h, i] = s


def values(pool: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Codes [..., bs, 128] and scales [...] -> float64 values."""
    return (pool.astype(np.float64) - 128) * scales.astype(np.float64)[..., None, None]


def attention(q, k_pool, v_pool, scales, tables, lens, scale):
    """Textbook attention over the values, fp64: (out, tol) float64 [B, q_len, Hq, 128]. tables
    [B, width] or [B, Hkv, width].

    tol is how far a result may be off that takes the codes' products on tensor cores, rounds each
    softmax weight once to fp16, sums in fp32 and rounds the output once to fp16:
      * the output: 2^-11 of it, 2^-25 for subnormals; a weight: 2^-11 of it, and 2^-25 where it is
        subnormal, with the largest weight times value scale taken to 2^11 or more;
      * scores: K codes come as u 2^-24, u = code + 128, their offset's share 128 sum q apart. A sum of 8
        products of 16 terms truncates by 2^-23 of at most 383 sum|q| each time: 2^-11 s_K sum|q|;
        sum q itself is an fp32 sum of 34 terms in a row: 34 2^-24 128 sum|q| < 2^-11 s_K sum|q|;
        and a tensor core cuts products below 2^-25 of the largest, a subnormal's exponent counted
        as -14: 2^-15 of a code step of max|q| each, 128 of them. Then two fp32 roundings of a
        number of at most 256: 2^-15;
      * values: m / 16 fp32 sums, each truncated by 2^-23 of at most sum p|v| (as many partial sums
        merged by at most 8 more), and 16 products cut below 2^-24 of 128 times the largest weight:
        2^-13 sum p s_V.
    A relative error e of the weights moves the output by at most 2 e sum p |v|."""
    q = np.asarray(q, np.float64)
    B, q_len, hq, _ = q.shape
    hkv, bs = k_pool.shape[1], k_pool.shape[2]
    group = hq // hkv
    out, tol = np.zeros(q.shape), np.full(q.shape, 2.0 ** -25)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        for h in range(hkv):
            ids = (tables[b] if tables.ndim == 2 else tables[b, h])[:-(-n // bs)]
            ks, vs = (np.repeat(scales[ids, h, i].astype(np.float64), bs)[:n] for i in (0, 1))
            K = values(k_pool[ids, h], scales[ids, h, 0]).reshape(-1, D)[:n]
            V = values(v_pool[ids, h], scales[ids, h, 1]).reshape(-1, D)[:n]
            for i in range(q_len):
                m = n - q_len + i + 1
                if m <= 0:
                    continue
                at = slice(h * group, (h + 1) * group)
                qq = q[b, i, at]
                x = qq @ K[:m].T * scale
                p = np.exp(x - x.max(-1, keepdims=True))
                L = p.sum(-1, keepdims=True)
                p = p / L
                o = p @ V[:m]
                e = abs(scale) * ks[:m].max() * (
                    2.0 ** -10 * np.abs(qq).sum(-1, keepdims=True) +
                    2.0 ** -8 * np.abs(qq).max(-1, keepdims=True)) + 2.0 ** -15 + m * 2.0 ** -28
                pv = p * vs[:m]
                out[b, i, at] = o
                tol[b, i, at] += (
                    (2.0 ** -11 + 2 * e + (m / 16 + 8) * 2.0 ** -23) * (p @ np.abs(V[:m])) +
                    2.0 ** -11 * np.abs(o) + 2.0 ** -13 * pv.sum(-1, keepdims=True) +
                    m * 2.0 ** -36 * 127 * pv.max(-1, keepdims=True))
    return out, tol


def bound_scores(q_rows, bounds, k_scale):
    """Scores of blocks with bounds [N, 2, 128] and scales [N], the greatest over the query rows
    [R, 128] (a row with a NaN or an infinity does not count); NaN where the scale is, whatever the
    rows hold."""
    lo, hi = (bounds[:, i].astype(np.int64) - 128 for i in (0, 1))
    best = np.full(len(bounds), -np.inf)
    for row in np.asarray(q_rows, np.float64):
        s = scale_of(row)
        if math.isnan(s):
            continue
        p = np.clip(np.rint(row / s), -127, 127).astype(np.int64)
        dot = np.maximum(p * lo, p * hi).sum(-1)
        best = np.maximum(best, dot * s)
    none = np.isneginf(best)      # (the same for all blocks: no row counts)
    return np.where(none & ~np.isnan(k_scale), -np.inf, np.where(none, 1, best) * k_scale)


def select(q, scales, bounds, tables, lens, bs, budget, first, last):
    """(tables [B, Hkv, budget], lens [B]) int32."""
    B, q_len, hq, _ = q.shape
    nb, hkv = bounds.shape[:2]
    group, width = hq // hkv, tables.shape[1]
    out = np.full((B, hkv, budget), -1, np.int32)
    out_lens = np.zeros(B, np.int32)
    for b in range(B):
        n = min(max(int(lens[b]), 0), width * bs)
        count = -(-n // bs)
        ids = tables[b, :count]
        taken = min(count, budget)
        out_lens[b] = n - (count - taken) * bs
        if taken == count:
            out[b, :, :taken] = ids
            continue
        own = count - max(n - q_len, 0) // bs
        there = (ids >= 0) & (ids < nb)
        safe = np.where(there, ids, 0)
        for h in range(hkv):
            rows = [q[b, i, h * group + g] for i in range(q_len) for g in range(group)
                    if n - q_len + i >= 0]
            s = bound_scores(np.array(rows).reshape(-1, D), bounds[safe, h],
                             scales[safe, h, 0].astype(np.float64))
            # kept blocks first, then NaN scales, then the scores, unknown blocks last
            rank = np.where(there, np.where(np.isnan(s), 1, 0), -1)
            s = np.where(there & ~np.isnan(s), s, 0.0)
            rank[:first] = 2
            rank[count - max(last, own):] = 2
            s = np.where(rank == 2, 0.0, s)
            order = np.lexsort((np.arange(count), -s, -rank))
            out[b, h, :taken] = ids[np.sort(order[:taken])]
    return out, out_lens
