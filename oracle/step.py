"""Oracle (test infrastructure) of a serving step's bookkeeping and of the norm with rotation:
plain loops over Python integers, and fp64 (numpy)."""
from __future__ import annotations

import numpy as np


def _blocks(n: int, bs: int) -> int:
    return -(-n // bs)


def extend(tables, lens, new, bs, free, count, max_tokens):
    """-> (tables, lens, count, slots, seqs, positions, cu, refused sequences)."""
    tables, lens, free = tables.copy(), lens.copy(), np.asarray(free)
    num_blocks = len(free)
    slots, seqs, pos = ([-1] * max_tokens for _ in range(3))
    cu, refused = [0], []
    cap = tables.shape[1] * bs
    start, want, taken = 0, 0, 0
    for b, (n, m) in enumerate(zip(lens.tolist(), new.tolist())):
        end = start + max(m, 0)
        fits = 0 <= n <= cap and m >= 0 and n + m <= cap
        need = _blocks(n + m, bs) - _blocks(n, bs) if fits else 0
        want += need
        if not fits or end > max_tokens or (need and want > count):
            refused.append(b)
        else:
            for j in range(need):
                tables[b, _blocks(n, bs) + j] = free[count - 1 - taken]
                taken += 1
            for i in range(m):
                p = n + i
                blk = int(tables[b, p // bs])
                seqs[start + i], pos[start + i] = b, p
                slots[start + i] = blk * bs + p % bs if 0 <= blk < num_blocks else -1
            lens[b] = n + m
        start = end
        cu.append(min(start, max_tokens))
    return (tables, lens, count - taken, np.array(slots, np.int64), np.array(seqs, np.int32),
            np.array(pos, np.int64), np.array(cu, np.int32), refused)


def truncate(tables, lens, keep, bs, free, count):
    """-> (tables, lens, free, count); unchanged if the stack would overflow; a sequence whose
    length its table cannot hold stays as it is."""
    tables, lens, free = tables.copy(), lens.copy(), np.asarray(free).copy()
    gone = [(b, j) for b, (n, m) in enumerate(zip(lens.tolist(), keep.tolist()))
            if 0 <= n <= tables.shape[1] * bs and 0 <= m < n
            for j in range(_blocks(m, bs), _blocks(n, bs))]
    if count + len(gone) > len(free):
        return tables, lens, free, count
    for r, (b, j) in enumerate(gone):
        free[count + len(gone) - 1 - r] = tables[b, j]
        tables[b, j] = -1
    for b, m in enumerate(keep.tolist()):
        if 0 <= m < lens[b] <= tables.shape[1] * bs:
            lens[b] = m
    return tables, lens, free, count + len(gone)


def norm_rope(x, weight, eps, positions, cos_sin):
    """fp64 RMS norm and rotate-half rotation of x [T, H, 128] by rows `positions` of cos_sin
    [n, 64, 2]: (out, tol). tol: the output's rounding to fp16 (2^-11 relative; 2^-25 for
    subnormals) and 2^-20 of the larger terms for the fp32 steps on the way (some ten of
    2^-24 each)."""
    x, w = np.asarray(x, np.float64), np.asarray(weight, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    cs = np.asarray(cos_sin, np.float64)[np.asarray(positions)][:, None]
    c, s = cs[..., 0], cs[..., 1]
    a, b = y[..., :64], y[..., 64:]
    out = np.concatenate([a * c - b * s, b * c + a * s], -1)
    terms = np.concatenate([np.abs(a * c) + np.abs(b * s), np.abs(b * c) + np.abs(a * s)], -1)
    return out, 2.0 ** -11 * np.abs(out) + 2.0 ** -20 * terms + 2.0 ** -25
