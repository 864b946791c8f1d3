"""The 4-bit cache's oracle (test infrastructure): rows, widening and attention in fp64 (numpy).

A row of 128 elements is 80 bytes: 64 bytes of codes (element 2 j in the low half of byte j),
then an fp16 scale s and an fp16 minimum z for each 32 elements; value = s * code + z.
"""
from __future__ import annotations

import numpy as np

D, GROUP, ROW = 128, 32, 80
F16_MAX = np.float32(65504)


def _up(x: np.ndarray) -> np.ndarray:
    """Least fp16 >= x (float32, x >= 0)."""
    with np.errstate(over="ignore"):
        h = x.astype(np.float16)
    return np.where(h.astype(np.float32) < x, np.nextafter(h, np.float16(np.inf)), h)


def _down(x: np.ndarray) -> np.ndarray:
    """Greatest fp16 <= x (float32, x >= 0)."""
    h = x.astype(np.float16)
    return np.where(h.astype(np.float32) > x, np.nextafter(h, np.float16(0)), h)


def quantise(x: np.ndarray) -> np.ndarray:
    """fp16 [..., 128] -> uint8 [..., 80]."""
    x = np.ascontiguousarray(x)
    assert x.dtype == np.float16 and x.shape[-1] == D
    g = x.reshape(x.shape[:-1] + (D // GROUP, GROUP))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], np.float16(0), g)
    lo, hi = g.min(-1), g.max(-1)
    range32 = hi.astype(np.float32) - lo.astype(np.float32)
    up = _up(range32 / np.float32(15))
    s = np.minimum(up, _down((F16_MAX - lo.astype(np.float32)) / np.float32(15)))
    s64, z64 = s.astype(np.float64)[..., None], lo.astype(np.float64)[..., None]
    # x - z is exact in fp64, and so is its comparison with the borders (k + 1/2) s; the quotient
    # is only a first guess
    d = g.astype(np.float64) - z64
    safe = np.where(s64 > 0, s64, 1.0)
    k = np.floor(d / safe)
    k = np.where(d - k * safe < 0, k - 1, k)
    k = np.where(d - (k + 1) * safe >= 0, k + 1, k)
    rem = d - (k + 0.5) * safe
    k = k + ((rem > 0) | ((rem == 0) & (k % 2 == 1)))
    code = np.where(s64 > 0, np.clip(k, 0, 15), 0).astype(np.uint8)
    code = np.where(bad[..., None], np.uint8(0), code).reshape(x.shape)
    out = np.empty(x.shape[:-1] + (ROW,), np.uint8)
    out[..., :64] = code[..., 0::2] | (code[..., 1::2] << 4)
    par = np.stack([np.where(bad, np.float16(np.nan), s), np.where(bad, np.float16(np.nan), lo)], -1)
    bits = par.view(np.uint16)
    bits = np.where(bad[..., None], np.uint16(0x7FFF), bits)
    out[..., 64:] = np.ascontiguousarray(bits).view(np.uint8).reshape(out[..., 64:].shape)
    return out


def parts(rows: np.ndarray):
    """uint8 [..., 80] -> (codes, s, z), each float64 [..., 128]."""
    code = np.empty(rows.shape[:-1] + (D,), np.float64)
    code[..., 0::2], code[..., 1::2] = rows[..., :64] & 15, rows[..., :64] >> 4
    par = np.ascontiguousarray(rows[..., 64:]).view(np.float16).astype(np.float64)
    return code, np.repeat(par[..., 0::2], GROUP, -1), np.repeat(par[..., 1::2], GROUP, -1)


def values(rows: np.ndarray) -> np.ndarray:
    """uint8 [..., 80] -> float64 [..., 128], s * code + z (exact in fp64)."""
    code, s, z = parts(rows)
    return s * code + z


def append(k, v, slots, k_pool, v_pool):
    """Quantises rows k, v [T, Hkv, 128] into pools [NB, Hkv, bs, 80] in place."""
    bs = k_pool.shape[2]
    for x, pool in ((k, k_pool), (v, v_pool)):
        rows = quantise(x)
        for t, slot in enumerate(np.asarray(slots)):
            if 0 <= slot < pool.shape[0] * bs:
                pool[slot // bs, :, slot % bs] = rows[t]


def attention(q, k_pool, v_pool, tables, lens, scale):
    """Textbook attention over the values, fp64: (out, tol) float64 [B, q_len, Hq, 128].

    tol is how far a result may be off that takes the codes' products on tensor cores, rounds each
    softmax weight once to fp16 (half a step, 2^-11 relative; a weight below 2^-14 of a warp's
    largest by 2^-25 of it), sums in fp32, and rounds the output once (2^-11 relative, 2^-25 for
    subnormals). The room for one more rounding of 2^-11 per value is left.
    A tensor core aligns the products of a dot by the sums of their operands' exponents, a
    subnormal's counted as -14, and cuts below 2^-25 of the largest. Codes come as subnormals
    c 2^-22 and c 2^-18, so a code's product with a weight w (scores: query element, scaled by
    16 for the first kind) is cut below 2^(-25 - 14 + 22) = 2^-17 of the largest w, or lost whole.
    Values: w = p s in two fp16 parts, the second under 2^-11 of the first: at most 2^-16 max(p s)
    a key, or 16 p s. Scores: 16 products of a group's 32 with 2^-17 s max|q|, 16 with 2^-21 and
    the sum itself: (2^-13 + 2^-16) s max|q|, the maximum over the group; its query sum times z is
    split in two fp16 numbers, the second down to 2^-24 with the row's largest |q| at 2^-8 or
    more: 2^-17 |z| max|q|, over the row.
    The fp32 sums of p s code and of p z may be kept apart: they nearly cancel where a value is
    near zero, so their errors are relative to S = sum p (15 s + |z|). A sum truncates by less
    than 2^-23 of itself, at most 64 times in a row here: 2^-17 S. Likewise the scores' sums, at
    most 32 times: 2^-18 sum |q| (15 s + |z|).
    A relative error e of the weights moves the output by at most 2 e sum p |v|."""
    q = np.asarray(q, np.float64)
    B, q_len, hq, _ = q.shape
    hkv, bs = k_pool.shape[1], k_pool.shape[2]
    group = hq // hkv
    out = np.zeros(q.shape)
    tol = np.full(q.shape, 2.0 ** -25)
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        ids = tables[b, :(n + bs - 1) // bs]
        for h in range(hkv):
            kc, ks, kz = parts(k_pool[ids, h].reshape(-1, ROW)[:n])
            vc, vs, vz = parts(v_pool[ids, h].reshape(-1, ROW)[:n])
            K, V = ks * kc + kz, vs * vc + vz
            reach_v = 15 * np.abs(vs) + np.abs(vz)
            reach = 15 * np.abs(ks) + np.abs(kz)
            for i in range(q_len):
                m = n - q_len + i + 1
                if m <= 0:
                    continue
                qq = q[b, i, h * group:(h + 1) * group]
                x = qq @ K[:m].T * scale
                p = np.exp(x - x.max(-1, keepdims=True))
                L = p.sum(-1, keepdims=True)
                qmax = np.abs(qq).reshape(group, 4, GROUP).max(-1)             # [group, 4]
                s4, z4 = ks[:m, ::GROUP], np.abs(kz[:m, ::GROUP])              # [m, 4]
                e = (2.0 ** -18 * (np.abs(qq) @ reach[:m].T) +
                     (2.0 ** -13 + 2.0 ** -16) * (qmax @ s4.T) +
                     2.0 ** -17 * qmax.max(-1, keepdims=True) * z4.sum(-1))
                e = abs(scale) * e.max(-1, keepdims=True)
                ps = (p / L)[:, :, None] * vs[:m, ::GROUP]                     # [group, m, 4]
                cut = np.minimum(2.0 ** -16 * ps.max(1, keepdims=True), 16 * ps).sum(1)
                avg = (p / L) @ np.abs(V[:m])
                o = (p / L) @ V[:m]
                out[b, i, h * group:(h + 1) * group] = o
                tol[b, i, h * group:(h + 1) * group] += (
                    (2 * 2.0 ** -11 + 2 * e) * avg + 2.0 ** -11 * np.abs(o) +
                    2.0 ** -17 * ((p / L) @ reach_v[:m]) + np.repeat(cut, GROUP, -1) +
                    m * 2.0 ** -25 / L * np.nanmax(np.abs(V[:m])))
    return out, tol
