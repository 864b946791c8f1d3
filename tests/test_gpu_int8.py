"""GPU parity of the 8-bit cache with a scale per block and head: append, widening, block copies,
decode, block selection and decode over selected blocks.

Codes, scales, bounds and chosen blocks must equal the oracle's; attention must lie within the bound
that the oracle derives for each element."""
import math

import numpy as np
import pytest
import torch

from oracle import int8
from paged_kv_cache_147_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def _rows(rng, shape, outliers=True):
    x = rng.standard_normal(shape + (128,))
    if outliers:
        x[..., rng.choice(128, 5, replace=False)] *= 8
        x += rng.standard_normal(128)
    return x.astype(np.float16)


def _cache(rng, nb, hkv, bs, spread=2):
    """Codes of every value, scales that differ from block to block, bounds that fit the codes."""
    k, v = (rng.integers(1, 256, (nb, hkv, bs, 128)).astype(np.uint8) for _ in range(2))
    scales = 2.0 ** rng.integers(-6 - spread, -6 + spread, (nb, hkv, 2), endpoint=True)
    bounds = np.stack([k.min(2), k.max(2)], 2)
    return k, v, scales.astype(np.float32), bounds


def _tables(rng, lens, bs, extra=3, width=None):
    lens = np.asarray(lens, np.int32)
    nblk = (lens + bs - 1) // bs
    nb = int(nblk.sum()) + extra
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), width or max(int(nblk.max()), 1) + 1), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
    return lens, tables, nb, perm[at:]


def _case(lens, bs=16, hq=12, hkv=2, q_len=1, seed=0, spread=2):
    rng = np.random.default_rng(seed)
    lens, tables, nb, unused = _tables(rng, lens, bs)
    k, v, scales, bounds = _cache(rng, nb, hkv, bs, spread)
    scales[unused] = np.nan
    q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
    return k, v, scales, bounds, tables, lens, q


def _close(out, want, tol, what=""):
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: not finite"
    err = np.abs(got - want)
    worst = np.unravel_index(np.argmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: off {err[worst]:.3g} of {tol[worst]:.3g} at {worst}"


def _decode(k, v, scales, tables, lens, q, scale, ws=None, errors=0):
    qd = _dev(q)
    out = torch.full_like(qd, float("nan"))
    if ws is None:
        ws = pkv.make_workspace(q.shape[0], q.shape[1], q.shape[2], k.shape[1])
    pkv.paged_attn_decode_int8(out, qd, _dev(k), _dev(v), _dev(scales), _dev(tables), _dev(lens),
                               scale, ws)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == errors
    return out


# ----------------------------------------------------------------------------- append
def _append_both(k, v, slots, cache, errors=0, bounds=True):
    """The library and the oracle on the same cache; everything must be equal."""
    dev = [_dev(x) for x in cache]
    pkv.kv_append_int8(_dev(k), _dev(v), _dev(slots), *dev[:3], dev[3] if bounds else None)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == errors
    with np.errstate(invalid="ignore"):
        int8.append(k, v, slots, *cache[:3], cache[3] if bounds else None)
    for got, want, what in zip(dev, cache, ("K", "V", "scales", "bounds")):
        assert np.array_equal(got.cpu().numpy(), want, equal_nan=what == "scales"), what
    return cache


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hkv,T", [(1, 1), (3, 40), (2, 700), (8, 1100)])
def test_append_equals_the_oracle(hkv, T, bs):
    rng = np.random.default_rng(bs * 7 + T)
    nb = T // bs + 6
    cache = _cache(rng, nb, hkv, bs, spread=6)
    k, v = _rows(rng, (T, hkv)), _rows(rng, (T, hkv), outliers=False)
    k[:: max(1, T // 7)] *= np.float16(30)                  # some blocks' scales grow
    start = int(rng.integers(1, bs))                        # the first block holds rows already
    perm = rng.permutation(nb)
    pos = start + np.arange(T)
    slots = (perm[pos // bs] * bs + pos % bs).astype(np.int64)
    if T > 3:
        slots[T // 2] = -1
    _append_both(k, v, slots, cache)


@pytest.mark.parametrize("bs", [16, 64, 256])
def test_append_over_all_magnitudes_token_by_token(bs):
    # any finite bits, the blocks filled by calls of one to five tokens: scales grow all the way
    rng = np.random.default_rng(bs)
    hkv, seqs = 3, 5
    cache = (np.zeros((seqs, hkv, bs, 128), np.uint8), np.zeros((seqs, hkv, bs, 128), np.uint8),
             np.zeros((seqs, hkv, 2), np.float32), np.zeros((seqs, hkv, 2, 128), np.uint8))
    at = np.zeros(seqs, int)
    for step in range(9):
        new = np.minimum(rng.integers(0, 6, seqs), bs - at)
        slots = np.concatenate([b * bs + at[b] + np.arange(new[b]) for b in range(seqs)])
        at += new
        x = rng.integers(0, 1 << 16, (2, len(slots), hkv, 128)).astype(np.uint16).view(np.float16)
        x = np.where(np.isfinite(x), x, np.float16(0.1))
        x = (x.astype(np.float64) * 2.0 ** -(18 - 2 * step)).astype(np.float16)
        if len(slots):
            cache = _append_both(x[0], x[1], slots.astype(np.int64), cache)


def test_append_at_the_edges_of_the_format():
    rng = np.random.default_rng(5)
    hkv, bs = 1, 16
    cache = _cache(rng, 8, hkv, bs)
    k = np.zeros((7, hkv, 128), np.float16)
    k[0, 0, :3] = [65504, -65504, 65024]                    # the largest scale, saturated
    k[1, 0, 5] = 2.0 ** -24                                 # the smallest
    k[2, 0, :6] = [127, 0.5, 1.5, 2.5, -0.5, -1.5]          # ties at scale 1
    k[3, 0, 7] = np.float16(127.0625)                       # just past 127: scale 2
    k[5, 0, 9] = np.nan
    k[6, 0, 9] = -np.inf
    slots = np.array([0, 16, 32, 48, 64, 80, 96], np.int64)
    k_pool, _, scales, bounds = _append_both(k, k[::-1].copy(), slots, cache)
    assert scales[0, 0, 0] == 512 and k_pool[0, 0, 0, 0] == 255 and k_pool[0, 0, 0, 1] == 1
    assert scales[1, 0, 0] == 2.0 ** -30 and scales[2, 0, 0] == 1 and scales[3, 0, 0] == 2
    assert scales[4, 0, 0] == 2.0 ** -30 and np.isnan(scales[5, 0, 0]) and np.isnan(scales[6, 0, 0])
    assert list(k_pool[2, 0, 0, :6]) == [255, 128, 130, 130, 128, 126]
    assert list(bounds[2, 0, :, 0]) == [255, 255]


def test_a_nan_stays_until_the_block_starts_again():
    rng = np.random.default_rng(6)
    cache = _cache(rng, 2, 2, 16)
    k, v = _rows(rng, (3, 2)), _rows(rng, (3, 2))
    k[1, 0, 3] = np.nan
    v[1, 1, 90] = np.inf
    cache = _append_both(k[:2], v[:2], np.array([4, 5], np.int64), cache)
    cache = _append_both(k[2:], v[2:], np.array([6], np.int64), cache)
    assert np.isnan(cache[2][0, 0, 0]) and np.isnan(cache[2][0, 1, 1])
    assert np.isfinite(cache[2][0, 1, 0]) and np.isfinite(cache[2][0, 0, 1])
    cache = _append_both(k[2:], v[2:], np.array([0], np.int64), cache)
    assert np.isfinite(cache[2][0]).all() and (cache[0][0, :, 1:] == 128).all()


@pytest.mark.parametrize("bs", [16, 128])
def test_append_takes_any_order_within_a_block_and_padding_between(bs):
    rng = np.random.default_rng(8 + bs)
    hkv, nb = 2, 5
    for T in (bs - 1, 2100):                 # one team a token, one for sixteen
        cache = _cache(rng, max(nb, 2 * T // bs + 4), hkv, bs, spread=5)
        slots = np.full(T, -1, np.int64)
        blocks = rng.permutation(cache[0].shape[0])
        for i, at in enumerate(range(0, T, bs)):   # every second token of a stretch, shuffled
            here = np.arange(at, min(at + bs, T))[::2]
            slots[here] = blocks[i] * bs + rng.permutation(bs)[:len(here)]
        _append_both(_rows(rng, (T, hkv)), _rows(rng, (T, hkv)), slots, cache)


def test_append_without_bounds_and_with_bad_slots():
    rng = np.random.default_rng(9)
    cache = _cache(rng, 2, 2, 16)
    k = _rows(rng, (4, 2))
    before = cache[3].copy()
    slots = np.array([3, 2 * 16, -7, 1 << 40], np.int64)
    _append_both(k, k.copy(), slots, cache, errors=pkv.DEVERR_SLOT, bounds=False)
    assert np.array_equal(before, cache[3])


def test_append_of_a_large_call_in_mixed_runs():
    # sequences of very different new lengths, many blocks: the form of sixteen tokens a team
    rng = np.random.default_rng(10)
    for bs, hkv in ((16, 3), (256, 2)):
        new = np.concatenate([np.ones(400, int), rng.integers(1, 3 * bs, 30)])
        held = rng.integers(0, 2 * bs, len(new))
        _, tables, nb, _ = _tables(rng, held + new, bs)
        cache = _cache(rng, nb, hkv, bs, spread=4)
        pos = np.concatenate([h + np.arange(n) for h, n in zip(held, new)])
        seq = np.repeat(np.arange(len(new)), new)
        slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
        _append_both(_rows(rng, (len(pos), hkv)), _rows(rng, (len(pos), hkv)), slots, cache)


# ----------------------------------------------------------------------------- widen, copy
@pytest.mark.parametrize("hkv,bs", [(1, 16), (5, 32), (2, 256)])
def test_widen_equals_the_oracle(hkv, bs):
    rng = np.random.default_rng(bs)
    k, v, scales, _ = _cache(rng, 6, hkv, bs, spread=12)
    scales[2, 0, 0] = np.nan
    src, dst = np.array([4, 0, 9, 2, 4], np.int32), np.array([1, 3, 0, 2, 4], np.int32)
    outs = [torch.full((5, hkv, bs, 128), 7.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    pkv.widen_blocks_int8(_dev(k), _dev(v), _dev(scales), _dev(src), _dev(dst), *outs)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_BLOCK_ID
    for i, (out, pool) in enumerate(zip(outs, (k, v))):
        want = np.full(out.shape, 7, np.float16)
        for s, d in zip(src, dst):
            if s < 6:
                want[d] = int8.values(pool[s], scales[s, :, i]).astype(np.float16)
        assert np.array_equal(out.cpu().numpy(), want, equal_nan=True)


@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("bounds", [True, False])
def test_copied_blocks_carry_scales_and_bounds(layers, bounds):
    rng = np.random.default_rng(3)
    parts = [_cache(rng, 7, 3, 32) for _ in range(layers or 1)]
    cache = [np.stack(x) for x in zip(*parts)] if layers else list(parts[0])
    dev = [_dev(x) for x in cache]
    src, dst = np.array([5, 0, 40, 5], np.int32), np.array([2, 6, 1, 3], np.int32)
    pkv.copy_blocks_int8(*dev[:3], dev[3] if bounds else None, _dev(src), _dev(dst))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_BLOCK_ID
    for i, (got, want) in enumerate(zip(dev, cache)):
        want = want if layers else want[None]
        if i < 3 or bounds:
            want[:, [2, 6, 3]] = want[:, [5, 0, 5]]
        assert np.array_equal(got.cpu().numpy(), want if layers else want[0])


# ----------------------------------------------------------------------------- decode
SCALE = 1 / math.sqrt(128)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("hq,hkv,q_len", [(1, 1, 1), (12, 2, 1), (64, 8, 1), (7, 1, 2), (12, 2, 4),
                                          (15, 5, 4), (16, 2, 4)])
def test_decode(bs, hq, hkv, q_len):
    lens = [1, 0, q_len, 15, 16, 17, 100, 33, 700, 257]
    k, v, scales, _, tables, lens, q = _case(lens, bs, hq, hkv, q_len, seed=bs + hq)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    _close(_decode(k, v, scales, tables, lens, q, SCALE), want, tol)


@pytest.mark.parametrize("lens,hq,hkv,q_len,bs", [
    ([5000], 8, 1, 1, 16), ([9001, 3], 12, 2, 1, 64), ([4096] * 3, 32, 4, 2, 16),
    ([20000], 64, 8, 1, 128), ([1] * 300, 4, 2, 1, 16), ([2500, 1, 0, 31] * 8, 24, 2, 2, 32)])
def test_decode_of_long_and_of_many_contexts(lens, hq, hkv, q_len, bs):
    k, v, scales, _, tables, lens, q = _case(lens, bs, hq, hkv, q_len, seed=len(lens))
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    first = _decode(k, v, scales, tables, lens, q, SCALE)
    _close(first, want, tol)
    assert torch.equal(first, _decode(k, v, scales, tables, lens, q, SCALE))


@pytest.mark.parametrize("hq,hkv,q_len", [(8, 1, 1), (8, 1, 2), (8, 1, 3), (8, 1, 4)])
@pytest.mark.parametrize("width", [256, 8])
def test_decode_of_every_row_count_in_wide_and_narrow_tables(hq, hkv, q_len, width):
    # 8, 16, 24 and 32 rows; few long units, whole and split, against many short ones
    for lens in ([4090, 700], [3000], [100] * 160 + [0, 1, 17]):
        rng = np.random.default_rng(hq * q_len + len(lens))
        if max(lens) > 16 * width:
            continue
        lens, tables, nb, _ = _tables(rng, lens, 16, width=width)
        k, v, scales, _ = _cache(rng, nb, hkv, 16)
        q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
        want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
        _close(_decode(k, v, scales, tables, lens, q, SCALE), want, tol)


@pytest.mark.parametrize("rows", [1, 8, 12, 16, 24, 28, 32])
@pytest.mark.parametrize("lens", [[505], [512, 100], [2000], [640, 0, 4095, 1]])
def test_decode_of_few_sequences_in_many_parts(rows, lens):
    # one kv head: units in parts of 1 to 3 rounds, up to 16 partials a unit; tables just below and
    # above the widths at which eight warps take over
    q_len = 1 if rows < 12 else rows // 4
    k, v, scales, _, tables, lens, q = _case(lens, 16, rows // q_len, 1, q_len, seed=rows)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    first = _decode(k, v, scales, tables, lens, q, SCALE)
    _close(first, want, tol)
    assert torch.equal(first, _decode(k, v, scales, tables, lens, q, SCALE))


@pytest.mark.parametrize("q_len", [1, 3, 8, 12, 16, 24, 32])
def test_decode_of_as_many_sequences_as_it_takes(q_len):
    # shared blocks: each sequence reads its own part of a small pool
    rng = np.random.default_rng(q_len)
    B, nb = 4096, 40
    k, v, scales, _ = _cache(rng, nb, 1, 16)
    lens = rng.integers(0, 40, B).astype(np.int32)
    tables = rng.integers(0, nb, (B, 256)).astype(np.int32)
    q = rng.standard_normal((B, q_len, 1, 128)).astype(np.float16)
    out = _decode(k, v, scales, tables, lens, q, SCALE)
    pick = rng.choice(B, 60, replace=False)
    want, tol = int8.attention(q[pick], k, v, scales, tables[pick], lens[pick], SCALE)
    _close(out[torch.as_tensor(pick).to(DEV)], want, tol)


@pytest.mark.parametrize("spread", [0, 9])
@pytest.mark.parametrize("scale", [SCALE, -0.3, 0.0, 2.0])
def test_decode_with_other_scales(scale, spread):
    # blocks whose scales differ by up to 2^18, scores from flat to one-hot
    k, v, scales, _, tables, lens, q = _case([300, 77, 16], 16, 8, 2, 2, seed=5, spread=spread)
    scales[..., 0] = np.minimum(scales[..., 0], 2.0 ** -4)
    want, tol = int8.attention(q, k, v, scales, tables, lens, scale)
    _close(_decode(k, v, scales, tables, lens, q, scale), want, tol)


def test_decode_with_queries_of_all_sizes():
    k, v, scales, _, tables, lens, q = _case([200, 90, 33, 64], 16, 8, 2, 1, seed=12)
    q[0] *= np.float16(2.0 ** -10)
    q[1, 0, 3] = 0
    q[2, 0, :, 5] = 300
    q[3] = np.float16(2.0 ** -24)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    _close(_decode(k, v, scales, tables, lens, q, SCALE), want, tol)


def test_decode_at_the_ends_of_the_scales():
    # zero scales (blocks never written), the least and the greatest ones
    k, v, scales, _, tables, lens, q = _case([64, 64, 64], 16, 4, 2, 1, seed=13)
    scales[tables[0, :2]] = 0
    scales[tables[1, :4]] = 2.0 ** -30
    scales[tables[2, :4], :, 0], scales[tables[2, :4], :, 1] = 2.0 ** -8, 2.0 ** 8
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    _close(_decode(k, v, scales, tables, lens, q, SCALE), want, tol)


def test_a_nan_scale_reaches_the_queries_that_see_its_block():
    # four new tokens, the last two in a block of their own whose V (head 0), K (head 1) is NaN
    k, v, scales, _, tables, lens, q = _case([34, 50], 16, 4, 2, 4, seed=14)
    bad = tables[0, 2]
    scales[bad, 0, 1] = scales[bad, 1, 0] = np.nan
    clean = scales.copy()
    clean[bad] = 1
    want, tol = int8.attention(q, k, v, clean, tables, lens, SCALE)
    out = _decode(k, v, scales, tables, lens, q, SCALE)
    assert out[0, 2:].isnan().all()
    _close(out[0, :2], want[0, :2], tol[0, :2])
    _close(out[1], want[1], tol[1])
    # nothing but NaN to see, in a short and in a split context
    for n, hq in ((5, 4), (6000, 4)):
        k, v, scales, _, tables, lens, q = _case([n], 16, hq, 2, 1, seed=15)
        scales[tables[0, :(n + 15) // 16]] = np.nan
        assert _decode(k, v, scales, tables, lens, q, SCALE).isnan().all()


def test_a_nan_query_stays_in_its_row():
    k, v, scales, _, tables, lens, q = _case([40, 1], 16, 4, 2, 2, seed=16)
    q[0, 1, 2, 77] = np.nan
    q[1, 0] = np.inf                        # before its sequence's first token: sees nothing
    clean = np.where(np.isfinite(q), q, 0)
    want, tol = int8.attention(clean, k, v, scales, tables, lens, SCALE)
    out = _decode(k, v, scales, tables, lens, q, SCALE)
    assert out[0, 1, 2].isnan().all() and (out[1, 0] == 0).all()
    out[0, 1, 2], want[0, 1, 2] = 0, 0
    _close(out, want, tol)


def test_decode_refuses_bad_ids_and_lengths_without_a_fault():
    k, v, scales, _, tables, lens, q = _case([40, 20, 16], 16, 4, 2, 1, seed=17)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    bad = tables.copy()
    bad[0, 1] = k.shape[0]
    out = _decode(k, v, scales, bad, lens, q, SCALE, errors=pkv.DEVERR_BLOCK_ID)
    _close(out[1:], want[1:], tol[1:])
    long = lens.copy()
    long[1] = -5
    out = _decode(k, v, scales, tables, long, q, SCALE, errors=pkv.DEVERR_CONTEXT)
    assert (out[1] == 0).all()
    _close(out[[0, 2]], want[[0, 2]], tol[[0, 2]])


@pytest.mark.parametrize("hq,hkv,q_len", [(12, 2, 1), (8, 1, 2), (12, 2, 4), (8, 2, 8)])
def test_decode_with_a_table_per_head(hq, hkv, q_len):
    rng = np.random.default_rng(hq)
    bs, lens = 16, np.array([100, 16, 0, 900, q_len], np.int32)
    nblk = (lens + bs - 1) // bs
    width = int(nblk.max()) + 2
    nb = int(nblk.sum()) * hkv + 1
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), hkv, width), -1, np.int32)
    at = 0
    for b, n in enumerate(nblk):
        for h in range(hkv):
            tables[b, h, :n] = perm[at:at + n]
            at += n
    k, v, scales, _ = _cache(rng, nb, hkv, bs)
    q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    _close(_decode(k, v, scales, tables, lens, q, SCALE), want, tol)


# ----------------------------------------------------------------------------- selection
def _select_both(q, scales, bounds, tables, lens, bs, budget, first, last, errors=0):
    got = pkv.select_blocks(_dev(q), _dev(scales), _dev(bounds), _dev(tables), _dev(lens), bs, budget,
                            first, last)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == errors
    want = int8.select(q, scales, bounds, tables, lens, bs, budget, first, last)
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("hq,hkv,q_len", [(1, 1, 1), (12, 2, 1), (64, 8, 1), (8, 1, 2), (12, 2, 4),
                                          (15, 5, 4), (16, 2, 4)])
@pytest.mark.parametrize("bs,budget,first,last", [(16, 5, 1, 2), (64, 2, 0, 0), (16, 20, 3, 1),
                                                  (256, 3, 1, 1)])
def test_selection(hq, hkv, q_len, bs, budget, first, last):
    lens = np.array([0, 1, q_len, bs, 5 * bs, 5 * bs + 1, 20 * bs - 3, 63 * bs + 5, 300 * bs // 16 + 9])
    rng = np.random.default_rng(hq + bs)
    lens, tables, nb, unused = _tables(rng, lens, bs)
    _, _, scales, bounds = _cache(rng, nb, hkv, 16)
    # bounds of differing widths, so that scores are not all alike
    mid = rng.integers(60, 196, bounds[:, :, 0].shape)
    half = rng.integers(0, 60, mid.shape)
    bounds[:, :, 0], bounds[:, :, 1] = mid - half, mid + half
    q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
    _select_both(q, scales, bounds, tables, lens, bs, budget, first, last)


@pytest.mark.parametrize("seqs,hkv,blocks,budget", [(1, 1, 2048, 64), (1, 2, 8200, 500), (2, 8, 1024, 128),
                                                    (40, 4, 300, 17), (200, 2, 300, 299)])
def test_selection_across_clusters_of_all_sizes(seqs, hkv, blocks, budget):
    rng = np.random.default_rng(blocks)
    lens = rng.integers(blocks * 8, blocks * 16, seqs, endpoint=True)
    lens[0] = blocks * 16
    lens, tables, nb, _ = _tables(rng, lens, 16, width=blocks)
    bounds = np.sort(rng.integers(1, 256, (nb, hkv, 2, 128)), axis=2).astype(np.uint8)
    scales = (2.0 ** rng.integers(-8, -5, (nb, hkv, 2))).astype(np.float32)
    q = rng.standard_normal((seqs, 1, hkv * 4, 128)).astype(np.float16)
    _select_both(q, scales, bounds, tables, lens, 16, budget, 1, 2)


@pytest.mark.parametrize("blocks,budget,ties", [(20000, 64, False), (20000, 3000, True), (16384, 999, True),
                                                (17000, 16999, True)])
def test_selection_of_more_blocks_than_a_cta_holds(blocks, budget, ties):
    rng = np.random.default_rng(budget)
    nb = 50                                   # blocks that stand in the table many times: many ties
    tables = rng.integers(0, nb, (2, blocks)).astype(np.int32)
    lens = np.array([blocks * 16, blocks * 16 - 5000], np.int32)
    bounds = np.sort(rng.integers(1, 256, (nb, 1, 2, 128)), axis=2).astype(np.uint8)
    if not ties:
        nb = blocks
        tables = np.stack([rng.permutation(nb) for _ in range(2)]).astype(np.int32)
        bounds = np.sort(rng.integers(1, 256, (nb, 1, 2, 128)), axis=2).astype(np.uint8)
    scales = np.full((nb, 1, 2), 2.0 ** -6, np.float32)
    q = rng.standard_normal((2, 2, 3, 128)).astype(np.float16)
    _select_both(q, scales, bounds, tables, lens, 16, budget, 1, 1)


def test_equal_scores_go_to_the_lower_block():
    # all alike, then two levels, then zero queries (all scores 0, with signs of all kinds)
    rng = np.random.default_rng(1)
    lens, tables, nb, _ = _tables(rng, [5000, 3999], 16)
    bounds = np.empty((nb, 2, 2, 128), np.uint8)
    bounds[:, :, 0], bounds[:, :, 1] = 100, 150
    scales = np.full((nb, 2, 2), 0.25, np.float32)
    q = rng.standard_normal((2, 1, 8, 128)).astype(np.float16)
    got, _ = _select_both(q, scales, bounds, tables, lens, 16, 40, 0, 1)
    assert np.array_equal(got[0, 0, :39], tables[0, :39])
    scales[tables[:, ::3].reshape(-1)] = 0.5
    _select_both(q, scales, bounds, tables, lens, 16, 150, 2, 3)
    q[:] = 0
    q[:, :, ::2] = -0.0
    scales[tables[:, 1::4].reshape(-1)] = 0
    _select_both(q, scales, bounds, tables, lens, 16, 150, 2, 3)


def test_selection_with_extreme_queries_scales_and_nan():
    rng = np.random.default_rng(2)
    lens, tables, nb, _ = _tables(rng, [1600, 1600, 1600, 2, 1600], 16, width=100)
    bounds = np.sort(rng.integers(1, 256, (nb, 2, 2, 128)), axis=2).astype(np.uint8)
    scales = (2.0 ** rng.integers(-30, 10, (nb, 2, 2))).astype(np.float32)
    scales[tables[0, 5:60:6]] = np.nan
    q = rng.standard_normal((5, 2, 8, 128)).astype(np.float16)
    q[1] *= np.float16(2.0 ** -14)
    q[2, 0, 3, 5] = np.nan
    q[2, 1, 4, 9] = np.inf
    q[4] = np.nan                                  # nothing counts: the lowest blocks
    q[0, 0, 0] = 65504
    _select_both(q, scales, bounds, tables, lens, 16, 12, 1, 1)
    got, _ = _select_both(q, scales, bounds, tables, lens, 16, 7, 1, 1)
    assert np.array_equal(got[4, 0], np.append(tables[4, :6], tables[4, 99]))


def test_selection_of_bad_ids_and_lengths_without_a_fault():
    rng = np.random.default_rng(3)
    lens, tables, nb, _ = _tables(rng, [800, 640], 16, width=50)
    bounds = np.sort(rng.integers(1, 256, (nb, 2, 2, 128)), axis=2).astype(np.uint8)
    scales = np.full((nb, 2, 2), 0.25, np.float32)
    q = rng.standard_normal((2, 1, 8, 128)).astype(np.float16)
    bad = tables.copy()
    bad[0, [3, 20]] = [nb, -9]
    _select_both(q, scales, bounds, bad, lens, 16, 10, 1, 1, errors=pkv.DEVERR_BLOCK_ID)
    wrong = lens.copy()
    wrong[:] = [-4, 900]
    full = np.where(tables < 0, 0, tables)
    _select_both(q, scales, bounds, full, wrong, 16, 10, 1, 1, errors=pkv.DEVERR_CONTEXT)


# ----------------------------------------------------------------------------- a run of them
@pytest.mark.parametrize("bs,q_len,hq,hkv", [(16, 1, 12, 2), (64, 2, 8, 2), (32, 4, 12, 2)])
def test_a_sparse_step_after_the_other(bs, q_len, hq, hkv):
    """Prompts, then steps: append, select, attend over the selection and over everything."""
    rng = np.random.default_rng(bs)
    budget, first, last = 4, 1, 1
    lens = np.array([9 * bs + 3, 1, 4 * bs, 30 * bs - 2], np.int32)
    steps = 5
    _, tables, nb, _ = _tables(rng, lens + steps * q_len, bs)
    host = [np.zeros((nb, hkv, bs, 128), np.uint8), np.zeros((nb, hkv, bs, 128), np.uint8),
            np.zeros((nb, hkv, 2), np.float32), np.zeros((nb, hkv, 2, 128), np.uint8)]
    dev = list(pkv.make_int8_cache(nb, hkv, bs, device=DEV))
    ws = pkv.make_workspace(len(lens), q_len, hq, hkv)
    for step in range(steps + 1):
        new = lens if step == 0 else np.full(len(lens), q_len)
        old = np.zeros_like(lens) if step == 0 else lens
        pos = np.concatenate([o + np.arange(n) for o, n in zip(old, new)])
        seq = np.repeat(np.arange(len(lens)), new)
        slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
        k, v = (_rows(rng, (len(pos), hkv)) * np.float16(1 + step) for _ in range(2))
        pkv.kv_append_int8(_dev(k), _dev(v), _dev(slots), *dev)
        int8.append(k, v, slots, *host)
        if step == 0:
            continue
        lens = lens + q_len
        q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
        qd, lens_d, tables_d = _dev(q), _dev(lens.astype(np.int32)), _dev(tables)
        chosen, taken = pkv.select_blocks(qd, dev[2], dev[3], tables_d, lens_d, bs, budget, first, last)
        sparse, full = torch.full_like(qd, float("nan")), torch.full_like(qd, float("nan"))
        pkv.paged_attn_decode_int8(sparse, qd, *dev[:3], chosen, taken, SCALE, ws)
        pkv.paged_attn_decode_int8(full, qd, *dev[:3], tables_d, lens_d, SCALE, ws)
        torch.cuda.synchronize()
        assert pkv.device_error(clear=True) == 0
        for got, want in zip(dev, host):
            assert np.array_equal(got.cpu().numpy(), want)
        want_t, want_l = int8.select(q, host[2], host[3], tables, lens, bs, budget, first, last)
        assert np.array_equal(chosen.cpu().numpy(), want_t)
        assert np.array_equal(taken.cpu().numpy(), want_l)
        _close(sparse, *int8.attention(q, *host[:3], want_t, want_l, SCALE), "sparse")
        _close(full, *int8.attention(q, *host[:3], tables, lens, SCALE), "full")
