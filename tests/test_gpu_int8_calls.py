"""The 8-bit cache's calls as a server makes them: in a step's order over device tables with drafts
taken back, captured and replayed, on several streams at once, behind copy-on-write and ahead of a
prefill, on pools past 32-bit offsets; and what the binding refuses."""
import math

import numpy as np
import pytest
import torch

from oracle import int8, step
from paged_kv_cache_147_gb300 import pkv

from test_gpu_int8 import _cache, _case, _close, _decode, _dev, _rows, _tables

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALE = 1 / math.sqrt(128)


# ----------------------------------------------------------------------------- a server's steps
@pytest.mark.parametrize("bs,hq,hkv,q_len", [(16, 12, 2, 3), (32, 8, 2, 2)])
def test_prompts_then_drafts_with_rollback_over_device_tables(bs, hq, hkv, q_len):
    rng = np.random.default_rng(bs)
    B, nb, width, budget = 5, 120, 24, 4
    tables, lens = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    free, count = rng.permutation(nb).astype(np.int32), nb
    d = [_dev(x) for x in (tables, lens, free, np.array([count], np.int32))]
    host = [np.zeros((nb, hkv, bs, 128), np.uint8), np.zeros((nb, hkv, bs, 128), np.uint8),
            np.zeros((nb, hkv, 2), np.float32), np.zeros((nb, hkv, 2, 128), np.uint8)]
    cache = pkv.make_int8_cache(nb, hkv, bs)
    ws = pkv.make_workspace(B, q_len, hq, hkv)

    def layer(new, max_tokens, gain):
        """A step's tables and the append of its rows, padded behind the last token."""
        nonlocal tables, lens, count
        slots, *_ = pkv.extend_tables(d[0], d[1], _dev(new), bs, d[2], d[3], max_tokens)
        tables, lens, count, s, *_, refused = step.extend(tables, lens, new, bs, free, count, max_tokens)
        assert not refused
        k, v = (_rows(rng, (max_tokens, hkv)) * np.float16(gain) for _ in range(2))
        pkv.kv_append_int8(_dev(k), _dev(v), slots, *cache)
        int8.append(k, v, s, *host)

    layer(rng.integers(1, 5 * bs, B).astype(np.int32), 5 * 5 * bs, 1)
    for turn in range(4):
        layer(np.full(B, q_len, np.int32), B * q_len + 2, 2 ** turn)
        q = rng.standard_normal((B, q_len, hq, 128)).astype(np.float16)
        qd = _dev(q)
        chosen, taken = pkv.select_blocks(qd, cache[2], cache[3], d[0], d[1], bs, budget, 1, 1)
        out = torch.full_like(qd, float("nan"))
        pkv.paged_attn_decode_int8(out, qd, *cache[:3], chosen, taken, SCALE, ws)
        torch.cuda.synchronize()
        for got, want in zip(cache, host):
            assert np.array_equal(got.cpu().numpy(), want)
        want_t, want_l = int8.select(q, host[2], host[3], tables, lens, bs, budget, 1, 1)
        assert np.array_equal(chosen.cpu().numpy(), want_t)
        assert np.array_equal(taken.cpu().numpy(), want_l)
        _close(out, *int8.attention(q, *host[:3], want_t, want_l, SCALE))
        # some drafts are rejected: a block that becomes free is started afresh by its next owner
        keep = (lens - rng.integers(0, q_len, B)).astype(np.int32)
        pkv.truncate_tables(d[0], d[1], _dev(keep), bs, d[2], d[3])
        tables, lens, free, count = step.truncate(tables, lens, keep, bs, free, count)
    assert pkv.device_error(clear=True) == 0


def test_a_forked_block_is_copied_before_the_child_writes():
    rng = np.random.default_rng(1)
    hkv, bs = 2, 16
    cache = list(_cache(rng, 6, hkv, bs))
    dev = [_dev(x) for x in cache]
    pkv.copy_blocks_int8(*dev, _dev(np.array([2], np.int32)), _dev(np.array([5], np.int32)))
    for x in cache:
        x[5] = x[2]
    k = _rows(rng, (2, hkv)) * np.float16(20)
    slots = np.array([5 * bs + 9, 5 * bs + 10], np.int64)
    pkv.kv_append_int8(_dev(k), _dev(k), _dev(slots), *dev)
    int8.append(k, k, slots, *cache)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    for got, want in zip(dev, cache):
        assert np.array_equal(got.cpu().numpy(), want)


def test_a_chunk_is_read_back_for_the_prefill():
    rng = np.random.default_rng(2)
    hq, hkv, bs, q_len, lens = 8, 2, 16, 24, np.array([100, 40], np.int32)
    lens, tables, nb, _ = _tables(rng, lens, bs)
    cache = pkv.make_int8_cache(nb, hkv, bs, bounds=False)
    pos = np.concatenate([np.arange(n) for n in lens])
    seq = np.repeat(np.arange(2), lens)
    slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
    k, v = (_rows(rng, (len(pos), hkv)) for _ in range(2))
    pkv.kv_append_int8(_dev(k), _dev(v), _dev(slots), *cache)
    wide = [torch.zeros(nb, hkv, bs, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    ids = _dev(np.arange(nb, dtype=np.int32))
    pkv.widen_blocks_int8(*cache[:3], ids, ids, *wide)
    q = rng.standard_normal((2, q_len, hq, 128)).astype(np.float16)
    out = torch.empty(q.shape, dtype=torch.float16, device=DEV)
    pkv.paged_prefill(out, _dev(q), *wide, _dev(tables), _dev(lens), SCALE)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    # The widened values are the cache's own (codes times a power of two are exact in fp16), so the
    # attention over them is the cache's. The bound is that of the decode, whose terms cover the
    # prefill's: one rounding of each weight and of the output to fp16, products of 16 summed in fp32
    # (8 sums of at most sum |q| |k| <= 127 s_K sum |q|, 2^-23 each: 2^-13 s_K sum |q| < 2^-10), but for
    # weights below 2^-14 of the largest, off by 2^-25 each.
    host = [x.cpu().numpy() for x in cache[:3]]
    want, tol = int8.attention(q, *host, tables, lens, SCALE)
    for b, n in enumerate(lens):
        tol[b] += n * 2.0 ** -25 * np.abs(wide[1].cpu().numpy()[tables[b, :-(-n // bs)]]).max()
    _close(out, want, tol)


# ----------------------------------------------------------------------------- graphs and streams
def test_a_captured_step_follows_its_inputs():
    rng = np.random.default_rng(3)
    B, hq, hkv, bs, steps, budget = 3, 8, 2, 16, 20, 3
    lens, tables, nb, _ = _tables(rng, np.array([200, 31, 95]) + steps, bs)
    lens = lens - steps
    host = list(_cache(rng, nb, hkv, bs))
    dev = [_dev(x) for x in host]
    t_d, l_d = _dev(tables), _dev(lens.astype(np.int32))
    k_d, v_d = (torch.zeros(B, hkv, 128, dtype=torch.float16, device=DEV) for _ in range(2))
    s_d = torch.zeros(B, dtype=torch.int64, device=DEV)
    q_d = torch.zeros(B, 1, hq, 128, dtype=torch.float16, device=DEV)
    out, ws = torch.empty_like(q_d), pkv.make_workspace(B, 1, hq, hkv)
    chosen = torch.empty(B, hkv, budget, dtype=torch.int32, device=DEV)
    taken = torch.empty(B, dtype=torch.int32, device=DEV)

    def one():
        pkv.kv_append_int8(k_d, v_d, s_d, *dev)
        pkv.select_blocks(q_d, dev[2], dev[3], t_d, l_d, bs, budget, 1, 1, chosen, taken)
        pkv.paged_attn_decode_int8(out, q_d, *dev[:3], chosen, taken, SCALE, ws)

    s_d.fill_(-1)
    one()                                   # (loads the kernels; nothing is written)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    for _ in range(steps):
        lens = lens + 1
        pos = lens - 1
        slots = tables[np.arange(B), pos // bs].astype(np.int64) * bs + pos % bs
        k, v = (_rows(rng, (B, hkv)) * np.float16(rng.integers(1, 9)) for _ in range(2))
        q = rng.standard_normal((B, 1, hq, 128)).astype(np.float16)
        for t, x in ((k_d, k), (v_d, v), (s_d, slots), (q_d, q), (l_d, lens.astype(np.int32))):
            t.copy_(torch.as_tensor(x))
        graph.replay()
        int8.append(k, v, slots, *host)
        want_t, want_l = int8.select(q, host[2], host[3], tables, lens, bs, budget, 1, 1)
        torch.cuda.synchronize()
        assert np.array_equal(chosen.cpu().numpy(), want_t)
        _close(out, *int8.attention(q, *host[:3], want_t, want_l, SCALE))
    for got, want in zip(dev, host):
        assert np.array_equal(got.cpu().numpy(), want)
    assert pkv.device_error(clear=True) == 0


def test_two_captured_decodes_at_once_with_a_workspace_each():
    cases = [_case(n, 16, 12, 2, 2, seed=i) for i, n in enumerate(([3000, 900], [5500, 17, 1200]))]
    runs, want = [], []
    for k, v, scales, _, tables, lens, q in cases:
        want.append(int8.attention(q, k, v, scales, tables, lens, SCALE))
        a = [_dev(x) for x in (q, k, v, scales, tables, lens)]
        out, ws = torch.empty_like(a[0]), pkv.make_workspace(len(lens), 2, 12, 2)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        pkv.paged_attn_decode_int8(out, *a, SCALE, ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(4):
                pkv.paged_attn_decode_int8(out, *a, SCALE, ws)
        runs.append((graph, stream, out, a, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, out, *_ in runs:
            with torch.cuda.stream(stream):
                out.fill_(float("nan"))
                graph.replay()
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    for (_, _, out, *_), w in zip(runs, want):
        _close(out, *w)


def test_two_selections_at_once():
    rng = np.random.default_rng(4)
    jobs = []
    for i, blocks in enumerate((3000, 700)):
        lens, tables, nb, _ = _tables(rng, [blocks * 16, blocks * 16 - 77], 16)
        bounds = np.sort(rng.integers(1, 256, (nb, 2, 2, 128)), axis=2).astype(np.uint8)
        scales = np.full((nb, 2, 2), 2.0 ** -6, np.float32)
        q = rng.standard_normal((2, 1, 8, 128)).astype(np.float16)
        host = (q, scales, bounds, tables, lens)
        jobs.append((host, [_dev(x) for x in host], torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = []
    for _ in range(3):
        for _, a, stream in jobs:
            with torch.cuda.stream(stream):
                got.append(pkv.select_blocks(*a, 16, 50))
    torch.cuda.synchronize()
    for i, (t, l) in enumerate(got):
        want = int8.select(*jobs[i % 2][0], 16, 50, 1, 1)
        assert np.array_equal(t.cpu().numpy(), want[0]) and np.array_equal(l.cpu().numpy(), want[1])


def test_one_workspace_for_calls_of_different_sizes():
    big = _case([1300] * 40, 16, 8, 8, 1, seed=51)
    one = _case([6000], 16, 12, 2, 4, seed=52)
    few = _case([4100, 700, 5000], 16, 8, 8, 1, seed=53)
    ws = pkv.make_workspace(40, 4, 48, 8)
    runs = []
    for k, v, scales, _, tables, lens, q in (few, big, one, big, few, one, big):
        runs.append(_decode(k, v, scales, tables, lens, q, SCALE, ws))
    assert torch.equal(runs[0], runs[4]) and torch.equal(runs[2], runs[5])
    assert torch.equal(runs[1], runs[3]) and torch.equal(runs[1], runs[6])
    for out, (k, v, scales, _, tables, lens, q) in zip(runs, (few, big, one)):
        want, tol = int8.attention(q[:4], k, v, scales, tables[:4], lens[:4], SCALE)
        _close(out[:4], want, tol)


def test_calls_run_on_the_current_and_on_a_given_stream():
    # the inputs arrive on a side stream behind long work; a launch elsewhere would miss them
    k, v, scales, bounds, tables, lens, q = _case([300, 47], seed=41)
    rng = np.random.default_rng(1)
    x = _rows(rng, (2, 2))
    pos = lens - 1
    slots = tables[np.arange(2), pos // 16].astype(np.int64) * 16 + pos % 16
    src, rows_h = _dev(q), _dev(x)
    big = torch.zeros(1 << 28, dtype=torch.float32, device=DEV)
    host = [k.copy(), v.copy(), scales.copy(), bounds.copy()]
    int8.append(x, x, slots, *host)
    want_t, want_l = int8.select(q, host[2], host[3], tables, lens, 16, 2, 0, 1)
    want = int8.attention(q, *host[:3], want_t, want_l, SCALE)
    side = torch.cuda.Stream()
    for given in (False, True):
        dev = [_dev(t) for t in (k, v, scales, bounds)]
        t_d, l_d, s_d = _dev(tables), _dev(lens), _dev(slots)
        qd, rows = torch.zeros_like(src), torch.zeros_like(rows_h)
        out, ws = torch.empty_like(qd), pkv.make_workspace(2, 1, 12, 2)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(8):
                big.add_(1)
            qd.copy_(src)
            rows.copy_(rows_h)
        at = side if given else None
        with torch.cuda.stream(torch.cuda.current_stream() if given else side):
            pkv.kv_append_int8(rows, rows, s_d, *dev, stream=at)
            chosen, taken = pkv.select_blocks(qd, dev[2], dev[3], t_d, l_d, 16, 2, 0, 1, stream=at)
            pkv.paged_attn_decode_int8(out, qd, *dev[:3], chosen, taken, SCALE, ws, stream=at)
        torch.cuda.synchronize()
        assert np.array_equal(chosen.cpu().numpy(), want_t)
        _close(out, *want)
    assert pkv.device_error(clear=True) == 0


def test_outputs_of_a_selection_on_a_given_stream_belong_to_it():
    side = torch.cuda.Stream()
    cache = pkv.make_int8_cache(4, 2, 16)
    table = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    q = torch.zeros(2, 1, 4, 128, dtype=torch.float16, device=DEV)
    torch.cuda.synchronize()
    for stream in (side, torch.cuda.ExternalStream(side.cuda_stream)):
        for t in pkv.select_blocks(q, cache[2], cache[3], table, table[:, 0].contiguous(), 16, 3,
                                   stream=stream):
            at = [s for s in torch.cuda.memory_snapshot()
                  if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]]
            assert at[0]["stream"] == side.cuda_stream
    torch.cuda.synchronize()


# ----------------------------------------------------------------------------- large, in any place
def test_decode_is_the_same_whatever_blocks_hold_the_data():
    k, v, scales, _, tables, lens, q = _case([2600, 40, 777], 16, 12, 2, 2, seed=21)
    first = _decode(k, v, scales, tables, lens, q, SCALE)
    perm = np.random.default_rng(5).permutation(len(k))
    moved = [np.empty_like(x) for x in (k, v, scales)]
    for m, x in zip(moved, (k, v, scales)):
        m[perm] = x
    t = np.where(tables >= 0, perm[tables.clip(0)], -1).astype(np.int32)
    assert torch.equal(first, _decode(*moved, t, lens, q, SCALE))


def test_pools_past_32_bit_byte_offsets():
    # 4.5 GB a pool, the sequence in its last blocks
    nb, hkv, bs = 34400, 4, 256
    k, v, scales, bounds, tables, lens, q = _case([700, 256], bs, 8, hkv, 1, seed=12)
    dev = list(pkv.make_int8_cache(nb, hkv, bs))
    n = k.shape[0]
    scales = np.nan_to_num(scales, nan=1.0)
    for d, x in zip(dev, (k, v, scales, bounds)):
        d[nb - n:] = _dev(x)
    t = np.where(tables >= 0, tables + nb - n, -1).astype(np.int32)
    want, tol = int8.attention(q, k, v, scales, tables, lens, SCALE)
    qd = _dev(q)
    out = torch.empty_like(qd)
    ws = pkv.make_workspace(2, 1, 8, hkv)
    pkv.paged_attn_decode_int8(out, qd, *dev[:3], _dev(t), _dev(lens), SCALE, ws)
    _close(out, want, tol)
    host = [x.copy() for x in (k, v, scales, bounds)]
    rng = np.random.default_rng(1)
    x = _rows(rng, (4, hkv)) * np.float16(9)
    slots = np.array([3, 4, 5, 0], np.int64) + (n - 1) * bs
    pkv.kv_append_int8(_dev(x), _dev(x), _dev(slots + (nb - n) * bs), *dev)
    int8.append(x, x, slots, *host)
    pkv.copy_blocks_int8(*dev, _dev(np.array([nb - 1], np.int32)), _dev(np.array([7], np.int32)))
    wide = [torch.zeros(1, hkv, bs, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    pkv.widen_blocks_int8(*dev[:3], _dev(np.array([nb - 1], np.int32)), _dev(np.array([0], np.int32)), *wide)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    for d, h in zip(dev, host):
        assert np.array_equal(d[nb - 1].cpu().numpy(), h[-1]) and np.array_equal(d[7].cpu().numpy(), h[-1])
    for i, w in enumerate(wide):
        assert np.array_equal(w[0].cpu().numpy(), int8.values(host[i][-1], host[2][-1, :, i]).astype(np.float16))


def test_bounds_past_32_bit_byte_offsets():
    # 18 M blocks and heads: 4.6 GB of bounds, the blocks at its end
    nb, hkv = 2250000, 8
    bounds = torch.empty(nb, hkv, 2, 128, dtype=torch.uint8, device=DEV)
    scales = torch.empty(nb, hkv, 2, device=DEV)
    rng = np.random.default_rng(6)
    n = 300
    b = np.sort(rng.integers(1, 256, (n, hkv, 2, 128)), axis=2).astype(np.uint8)
    s = (2.0 ** rng.integers(-8, -5, (n, hkv, 2))).astype(np.float32)
    bounds[nb - n:], scales[nb - n:] = _dev(b), _dev(s)
    tables = rng.permutation(n).astype(np.int32)[None]
    q = rng.standard_normal((1, 1, 16, 128)).astype(np.float16)
    lens = np.array([n * 16 - 5], np.int32)
    got, _ = pkv.select_blocks(_dev(q), scales, bounds, _dev(tables + nb - n), _dev(lens), 16, 20)
    want, _ = int8.select(q, s, b, tables, lens, 16, 20, 1, 1)
    assert np.array_equal(got.cpu().numpy(), want + nb - n)


def test_empty_calls():
    cache = pkv.make_int8_cache(4, 2, 16)
    before = [x.clone() for x in cache]
    rows = torch.zeros(0, 2, 128, dtype=torch.float16, device=DEV)
    none = torch.zeros(0, dtype=torch.int32, device=DEV)
    pkv.kv_append_int8(rows, rows, none.long(), *cache)
    pkv.copy_blocks_int8(*cache, none, none)
    q = torch.zeros(0, 1, 4, 128, dtype=torch.float16, device=DEV)
    table = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    t, l = pkv.select_blocks(q, cache[2], cache[3], table, none, 16, 5)
    assert t.shape == (0, 2, 5) and l.shape == (0,)
    ws = pkv.make_workspace(1, 1, 4, 2)
    pkv.paged_attn_decode_int8(q.clone(), q, *cache[:3], t, l, SCALE, ws)
    # sequences without a token, in tables without a column
    q = torch.ones(2, 1, 4, 128, dtype=torch.float16, device=DEV)
    table, lens = torch.zeros(2, 0, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    t, l = pkv.select_blocks(q, cache[2], cache[3], table, lens, 16, 5)
    assert (t == -1).all() and (l == 0).all()
    ws = pkv.make_workspace(2, 1, 4, 2)
    out = pkv.paged_attn_decode_int8(torch.full_like(q, 7), q, *cache[:3], t, l, SCALE, ws)
    assert (out == 0).all()
    for x, y in zip(cache, before):
        assert torch.equal(x, y)
    assert pkv.device_error(clear=True) == 0


# ----------------------------------------------------------------------------- refusals
def test_binding_refuses_what_the_library_cannot_see():
    k, v, s, b = pkv.make_int8_cache(4, 2, 16)
    q = torch.zeros(2, 1, 12, 128, dtype=torch.float16, device=DEV)
    bt = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    ht = torch.zeros(2, 2, 2, dtype=torch.int32, device=DEV)
    cl = torch.ones(2, dtype=torch.int32, device=DEV)
    ws = pkv.make_workspace(2, 1, 12, 2)
    rows = torch.zeros(2, 2, 128, dtype=torch.float16, device=DEV)
    slots = torch.full((2,), -1, dtype=torch.int64, device=DEV)
    wide = torch.zeros(4, 2, 16, 128, dtype=torch.float16, device=DEV)

    def call(fn, base):
        return lambda **kw: (lambda: fn(**{**base, **kw}))

    app = call(pkv.kv_append_int8, dict(k=rows, v=rows, slots=slots, k_cache=k, v_cache=v, kv_scales=s, k_bounds=b))
    wid = call(pkv.widen_blocks_int8, dict(k_cache=k, v_cache=v, kv_scales=s, src=cl, dst=cl, k_out=wide, v_out=wide.clone()))
    cpy = call(pkv.copy_blocks_int8, dict(k_cache=k, v_cache=v, kv_scales=s, k_bounds=b, src=cl, dst=cl * 2))
    dec = call(pkv.paged_attn_decode_int8, dict(out=q.clone(), q=q, k_cache=k, v_cache=v, kv_scales=s, block_tables=bt,
                                                context_lens=cl, scale=0.1, workspace=ws))
    sel = call(pkv.select_blocks, dict(q=q, kv_scales=s, k_bounds=b, block_tables=bt, context_lens=cl, block_size=16, budget=2))
    for ok in (app(), app(k_bounds=None), wid(), cpy(), cpy(k_bounds=None), dec(), dec(block_tables=ht), sel(),
               sel(tables_out=ht.clone(), lens_out=cl.clone())):
        ok()
    strided = torch.zeros(2, 2, 12, 128, dtype=torch.float16, device=DEV)[:, :1]
    bad = [
        app(k=rows.float()), app(v=rows[:1]), app(slots=slots.int()), app(slots=slots[:1]), app(k_cache=k.float()),
        app(v_cache=v[:2]), app(kv_scales=s.half()), app(kv_scales=s[..., 0]), app(k_bounds=b[:2]), app(k_bounds=b.int()),
        app(k_cache=k[..., :64], v_cache=v[..., :64]), app(k=rows.cpu()), app(k_cache=k[:, :, ::2]),
        wid(kv_scales=s[:3]), wid(dst=cl[:1]), wid(k_out=wide[:, :1], v_out=wide[:, :1]), wid(src=cl.long()), wid(v_out=wide[:2]),
        cpy(src=cl[:1]), cpy(kv_scales=s.double()), cpy(k_bounds=b[..., :64]), cpy(k_cache=k[None], v_cache=v[None]),
        dec(q=q.float()), dec(q=strided), dec(out=q[:1]), dec(context_lens=cl.long()), dec(block_tables=bt[:1]),
        dec(block_tables=ht[:, :1]), dec(block_tables=ht[None]), dec(k_cache=k[:2]), dec(kv_scales=s[:2]),
        dec(workspace=ws[:100]), dec(context_lens=cl[:1]), dec(kv_scales=s.cpu()),
        sel(q=q[:1]), sel(kv_scales=s[:3]), sel(k_bounds=b[:, :1]), sel(budget=1, keep_first=1), sel(budget=0),
        sel(block_size=17), sel(keep_last=-1), sel(tables_out=ht[..., :1]), sel(tables_out=ht.long()), sel(lens_out=cl[:1]),
        sel(block_tables=bt.long()), sel(context_lens=cl.cpu()), sel(q=strided[:, :, :11]),
    ]
    for i, refused in enumerate(bad):
        with pytest.raises(pkv.PkvError) as e:
            refused()
        assert e.value.status in (pkv.EINVAL, pkv.ENOSPC), i
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
