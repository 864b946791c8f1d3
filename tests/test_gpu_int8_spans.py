"""The 8-bit append where a team of warps takes as many tokens as a block has (large calls): many
blocks' first tokens in one team's span, padding, rows out of order, rows and blocks that straddle
spans, a last span that is not full."""
import numpy as np
import pytest

from test_gpu_int8 import _append_both, _cache, _rows

pytestmark = pytest.mark.gpu


def _span(T, hkv, bs):
    """Tokens a team: about 4096 warps in all, a block's worth at most."""
    return min(max(T * 2 * hkv * (bs // 16) // 4096, 1), bs)


def _slots(rng, runs, bs, shuffled):
    """Slots of runs of tokens, each in blocks of its own (from a random place in the first), with
    padding between some of them; `shuffled`: out of order within each block."""
    need = [-(-(n + bs) // bs) for n in runs]
    perm = rng.permutation(sum(need) + 2)
    out, at = [], 0
    for n, m in zip(runs, need):
        pos = int(rng.integers(0, bs)) + np.arange(n)
        s = perm[at + pos // bs] * bs + pos % bs
        at += m
        if shuffled:
            for b in np.unique(pos // bs):
                here = np.nonzero(pos // bs == b)[0]
                s[here] = rng.permutation(s[here])
        out.append(s)
        if rng.random() < 0.3:
            out.append(np.full(int(rng.integers(1, 4)), -1))
    return np.concatenate(out).astype(np.int64), len(perm)


@pytest.mark.parametrize("bs,hkv,most,shuffled", [
    (16, 8, 1, False),      # a step of thousands of sequences: a block a token, up to 16 in a span
    (16, 8, 70, True), (16, 8, 400, False), (32, 8, 3, True), (32, 8, 90, False), (64, 8, 9, False),
    (64, 16, 300, True), (128, 16, 20, True), (128, 8, 700, False), (256, 32, 40, False),
    (256, 16, 1500, True)])
def test_append_of_as_many_tokens_a_team_as_a_block_has(bs, hkv, most, shuffled):
    rng = np.random.default_rng(bs + most)
    runs, T = [], 0
    while T * hkv < 32768 + 8 * hkv:
        runs.append(int(rng.integers(1, most, endpoint=True)))
        T += runs[-1]
    slots, nb = _slots(rng, runs, bs, shuffled)
    if len(slots) % bs == 0:
        slots = np.append(slots, -1)
    T = len(slots)
    assert _span(T, hkv, bs) == bs and T % bs
    k, v = _rows(rng, (T, hkv)), _rows(rng, (T, hkv), outliers=False)
    k[rng.random(T) < 0.05] *= np.float16(40)                # some scales grow
    v[rng.integers(0, T, 3), 0, 5] = np.nan
    _append_both(k, v, slots, _cache(rng, nb, hkv, bs, spread=5))


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
def test_a_large_call_whose_spans_hold_padding_only(bs):
    # tokens at the ends of spans, nothing in most of them
    rng = np.random.default_rng(bs)
    hkv, T = 8, 4096 + 37
    assert _span(T, hkv, bs) == bs
    slots = np.full(T, -1, np.int64)
    at = np.array([0, bs - 1, bs, 3 * bs - 1, 1000, 1001, 4095, 4096, T - 1])
    at = np.unique(at)
    slots[at] = rng.permutation(len(at)) * bs + rng.integers(0, bs, len(at))
    _append_both(_rows(rng, (T, hkv)), _rows(rng, (T, hkv)), slots, _cache(rng, len(at) + 1, hkv, bs))
