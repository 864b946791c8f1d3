"""The block selection where a cluster of CTAs shares a head: with other work on the GPU, so that its
CTAs run apart, and with guards around the outputs; the largest budget; NaN scales and unknown
blocks where no query counts."""
import numpy as np
import pytest
import torch

from oracle import int8
from paged_kv_cache_147_gb300 import pkv

from test_gpu_int8 import _dev, _tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
GUARD = -77777


def _inputs(rng, seqs, hkv, blocks, q_len=1, group=2):
    lens = rng.integers(blocks * 12, blocks * 16, seqs, endpoint=True)
    lens, tables, nb, _ = _tables(rng, lens, 16, width=blocks)
    bounds = np.sort(rng.integers(1, 256, (nb, hkv, 2, 128)), axis=2).astype(np.uint8)
    scales = (2.0 ** rng.integers(-8, -5, (nb, hkv, 2))).astype(np.float32)
    q = rng.standard_normal((seqs, q_len, hkv * group, 128)).astype(np.float16)
    return q, scales, bounds, tables, lens


@pytest.mark.parametrize("seqs,hkv,blocks,budget,q_len", [
    (1, 8, 2048, 64, 1),        # eight CTAs a head
    (2, 1, 1100, 300, 2), (8, 4, 700, 90, 1), (16, 8, 512, 64, 2), (3, 2, 16384, 1000, 1),
    (1, 1, 16400, 2000, 1)])    # each CTA keeps its own keys
def test_clusters_among_other_work_write_their_own_rows_only(seqs, hkv, blocks, budget, q_len):
    rng = np.random.default_rng(blocks)
    args = _inputs(rng, seqs, hkv, blocks, q_len)
    want = int8.select(*args, 16, budget, 1, 2)
    dev = [_dev(x) for x in args]
    n = seqs * hkv * budget
    load = torch.randn(512, 512, device=DEV)
    busy = torch.empty_like(load)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    for _ in range(40):
        with torch.cuda.stream(side):
            torch.mm(load, load, out=busy)
        room = torch.full((n + 2 * budget,), GUARD, dtype=torch.int32, device=DEV)
        tables = room[budget:budget + n].view(seqs, hkv, budget)
        lens = torch.full((seqs + 2,), GUARD, dtype=torch.int32, device=DEV)
        pkv.select_blocks(*dev, 16, budget, 1, 2, tables, lens[1:-1])
        runs.append((room, lens))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    for room, lens in runs:
        assert (room[:budget] == GUARD).all() and (room[budget + n:] == GUARD).all()
        assert lens[0] == GUARD and lens[-1] == GUARD
        assert np.array_equal(room[budget:budget + n].view(seqs, hkv, budget).cpu().numpy(), want[0])
        assert np.array_equal(lens[1:-1].cpu().numpy(), want[1])


@pytest.mark.parametrize("blocks", [5, 200])      # one CTA, and a cluster
def test_the_largest_budget(blocks):
    # 8.6 GB of places, nearly all of them without a block
    rng = np.random.default_rng(blocks)
    q, scales, bounds, tables, lens = _inputs(rng, 1, 1, blocks)
    budget, pad = 2 ** 31 - 1, 4096
    room = torch.full((pad + budget + pad,), GUARD, dtype=torch.int32, device=DEV)
    out = room[pad:pad + budget].view(1, 1, budget)
    _, taken = pkv.select_blocks(*(_dev(x) for x in (q, scales, bounds, tables, lens)), 16, budget, 1, 1, out)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    n = -(-int(lens[0]) // 16)
    assert int(taken[0]) == lens[0]
    assert np.array_equal(out[0, 0, :n].cpu().numpy(), tables[0, :n])
    assert out[0, 0, n:].amin() == -1 and out[0, 0, n:].amax() == -1
    assert (room[:pad] == GUARD).all() and (room[-pad:] == GUARD).all()


@pytest.mark.parametrize("seqs,hkv,blocks,q_len", [(40, 4, 100, 1), (1, 2, 900, 2), (2, 1, 17000, 1)])
def test_a_nan_scale_comes_first_whatever_the_queries_hold(seqs, hkv, blocks, q_len):
    rng = np.random.default_rng(blocks + 1)
    q, scales, bounds, tables, lens = _inputs(rng, seqs, hkv, blocks, q_len)
    scales[tables[:, 5:blocks // 2:7].reshape(-1), :, 0] = np.nan
    scales[tables[:, 8:blocks // 2:7].reshape(-1), :, 0] = 0
    for x in (np.nan, np.inf, None):
        if x is None:                          # a row that counts beside one that does not
            q[:, 0, 1] = rng.standard_normal(128).astype(np.float16)
        else:
            q[:] = x
        for budget in (9, blocks // 3):        # (fewer places than NaN scales, and more)
            dev = [_dev(t) for t in (q, scales, bounds, tables, lens)]
            got = pkv.select_blocks(*dev, 16, budget, 1, 2)
            want = int8.select(q, scales, bounds, tables, lens, 16, budget, 1, 2)
            torch.cuda.synchronize()
            assert pkv.device_error(clear=True) == 0
            assert np.array_equal(got[0].cpu().numpy(), want[0])
            assert np.array_equal(got[1].cpu().numpy(), want[1])
        assert budget <= 9 or np.isin(tables[0, 5:blocks // 2:7], want[0][0, 0]).all()


@pytest.mark.parametrize("seqs,hkv,blocks", [(40, 4, 100), (1, 2, 900), (2, 1, 17000)])
def test_unknown_blocks_come_last_whatever_the_queries_hold(seqs, hkv, blocks):
    rng = np.random.default_rng(blocks + 2)
    q, scales, bounds, tables, lens = _inputs(rng, seqs, hkv, blocks)
    scales[tables[:, 5:blocks // 2:7].reshape(-1), :, 0] = np.nan
    tables[:, 1:blocks // 2:5], tables[:, 2:blocks // 2:5] = -9, len(bounds)
    for x in (np.nan, 1, 0):
        q[:] = x
        for budget in (9, blocks * 2 // 3, blocks * 4 // 5):   # (the last takes some unknown ones, too)
            dev = [_dev(t) for t in (q, scales, bounds, tables, lens)]
            got = pkv.select_blocks(*dev, 16, budget, 1, 2)
            want = int8.select(q, scales, bounds, tables, lens, 16, budget, 1, 2)
            torch.cuda.synchronize()
            assert pkv.device_error(clear=True) == (pkv.DEVERR_BLOCK_ID if (lens > 16 * budget).any() else 0)
            assert np.array_equal(got[0].cpu().numpy(), want[0])
            assert np.array_equal(got[1].cpu().numpy(), want[1])


@pytest.mark.parametrize("seqs,hkv", [(1, 1), (4, 8), (9, 8), (16, 8)])
def test_tables_around_the_widths_where_clusters_begin(seqs, hkv):
    # 8, 4 and 2 CTAs a head, or one, by the table's columns; contexts of all lengths in them
    rng = np.random.default_rng(seqs)
    q, scales, bounds, tables, lens = _inputs(rng, seqs, hkv, 1024)
    for width in (127, 128, 383, 384, 511, 512, 767, 768, 1023, 1024):
        n = np.minimum(lens, width * 16).astype(np.int32)
        n[::3] = rng.integers(0, width * 16, len(n[::3]))
        args = q, scales, bounds, np.ascontiguousarray(tables[:, :width]), n
        got = pkv.select_blocks(*(_dev(x) for x in args), 16, 50, 2, 1)
        want = int8.select(*args, 16, 50, 2, 1)
        torch.cuda.synchronize()
        # (some of those lengths pass what their table holds: places without a block, which are scored)
        holes = any(c > 800 and (t[:-(-c // 16)] < 0).any() for c, t in zip(n, args[3]))
        assert pkv.device_error(clear=True) == (pkv.DEVERR_BLOCK_ID if holes else 0)
        assert np.array_equal(got[0].cpu().numpy(), want[0])
        assert np.array_equal(got[1].cpu().numpy(), want[1])
