"""GPU parity of the block tables kept on the device (extend, truncate) with the step oracle:
every entry of every array, refusals included."""
import numpy as np
import pytest
import torch

from oracle import step
from paged_kv_cache_147_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def _state(rng, lens, bs, width, spare):
    lens = np.asarray(lens, np.int32)
    need = -(-lens // bs)
    nb = int(need.sum()) + spare
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), width), -1, np.int32)
    tables[np.arange(width)[None] < need[:, None]] = perm[:nb - spare]
    free = rng.integers(0, 1000, nb).astype(np.int32)     # entries past the count: anything
    free[:spare] = perm[nb - spare:]
    return tables, lens, free, spare


def _extend(tables, lens, new, bs, free, count, max_tokens, want_error=0):
    d = [_dev(x) for x in (tables, lens, np.asarray(new, np.int32), free,
                           np.array([count], np.int32))]
    slots, seqs, pos, cu = pkv.extend_tables(d[0], d[1], d[2], bs, d[3], d[4], max_tokens)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == want_error
    wt, wl, wc, ws, wq, wp, wcu, _ = step.extend(tables, lens, np.asarray(new), bs, free, count,
                                                 max_tokens)
    for got, want in ((d[0], wt), (d[1], wl), (d[3], free), (d[4], np.array([wc])), (slots, ws),
                      (seqs, wq), (pos, wp), (cu, wcu)):
        assert np.array_equal(got.cpu().numpy(), want)
    return d, wt, wl, wc


@pytest.mark.parametrize("B,bs,hi,new", [
    (1, 16, 0, 1), (1, 16, 40, 1), (3, 16, 40, 17), (64, 16, 2048, 1), (64, 64, 500, 5),
    (700, 32, 100, 40), (4096, 16, 60, 3), (2, 256, 1000, 60000), (300, 16, 64, 1000),
    (100, 16, 3000, 4000),      # more than 16384 blocks: the wide forms of both calls
])
def test_extend_and_back(B, bs, hi, new):
    rng = np.random.default_rng(B + bs)
    lens = rng.integers(0, hi, B, endpoint=True)
    m = rng.integers(0, new, B, endpoint=True)
    width = -(-(hi + new) // bs)
    tables, lens, free, count = _state(rng, lens, bs, width, int((-(-(lens + m) // bs)).sum()) + 3)
    d, wt, wl, wc = _extend(tables, lens, m, bs, free, count, int(m.sum()) + 7)
    keep = lens.copy()
    keep[::3] = -1
    pkv.truncate_tables(d[0], d[1], _dev(keep), bs, d[3], d[4])
    tt, tl, tf, tc = step.truncate(wt, wl, keep, bs, free, wc)
    for got, want in zip((d[0], d[1], d[3], d[4]), (tt, tl, tf, np.array([tc]))):
        assert np.array_equal(got.cpu().numpy(), want)
    assert pkv.device_error(clear=True) == 0


def test_no_sequences_and_no_tokens():
    rng = np.random.default_rng(0)
    tables, lens, free, count = _state(rng, [20, 3], 16, 4, 5)
    _extend(tables, lens, [0, 0], 16, free, count, 0)
    _extend(tables, lens, [0, 0], 16, free, count, 9)
    z = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    e = torch.zeros(0, dtype=torch.int32, device=DEV)
    slots, seqs, pos, cu = pkv.extend_tables(z, e, e, 16, _dev(free),
                                             _dev(np.array([5], np.int32)), 6)
    assert (slots == -1).all() and (seqs == -1).all() and (pos == -1).all() and cu.tolist() == [0]


def test_refusals_leave_a_sequence_as_it_is():
    rng = np.random.default_rng(7)
    bs = 16
    tables, lens, free, count = _state(rng, [20, 16, 40, 5, 0, 31], bs, 6, 9)
    # a negative count, one past the table (6 x 16 = 96), one served
    _extend(tables, lens, [3, -2, 57, 4, 0, 1], bs, free, count, 80,
            want_error=pkv.DEVERR_CONTEXT | pkv.DEVERR_POSITION)
    # the third past the table (40 + 60 of 96), so that the 7 blocks of the others suffice
    _extend(tables, lens, [50, 60, 60, 2, 0, 1], bs, free, count, 200,
            want_error=pkv.DEVERR_POSITION)
    # blocks run out at the third (3 + 4 + 3 of 9); the later ones that need none are served
    _extend(tables, lens, [50, 60, 50, 2, 0, 1], bs, free, count, 200, want_error=pkv.DEVERR_SPACE)
    # the token arrays are too small for the third
    _extend(tables, lens, [10, 10, 10, 2, 0, 1], bs, free, count, 25, want_error=pkv.DEVERR_SPACE)
    # a length outside the table
    bad = lens.copy()
    bad[1], bad[2] = 97, -1
    _extend(tables, bad, [1, 1, 1, 1, 1, 1], bs, free, count, 6, want_error=pkv.DEVERR_CONTEXT)
    # a free id outside the pool: in the table as it is, its tokens' slots -1
    free2 = free.copy()
    free2[count - 1] = len(free) + 4
    _extend(tables, lens, [20, 1, 1, 1, 1, 1], bs, free2, count, 25, want_error=pkv.DEVERR_BLOCK_ID)
    # counts no stack has
    d = [_dev(x) for x in (tables, lens, np.full(6, 40, np.int32), free, np.array([999], np.int32))]
    pkv.extend_tables(d[0], d[1], d[2], bs, d[3], d[4], 300)
    assert pkv.device_error(clear=True) == pkv.DEVERR_SPACE
    assert np.array_equal(d[0].cpu().numpy(), tables) and np.array_equal(d[1].cpu().numpy(), lens)


def test_truncate_refuses_more_blocks_than_the_stack_holds():
    rng = np.random.default_rng(9)
    tables, lens, free, count = _state(rng, [64, 40], 16, 4, 3)
    d = [_dev(x) for x in (tables, lens, np.array([0, 0], np.int32), free[:6],
                           np.array([3], np.int32))]
    pkv.truncate_tables(d[0], d[1], d[2], 16, d[3], d[4])
    assert pkv.device_error(clear=True) == pkv.DEVERR_SPACE
    assert np.array_equal(d[0].cpu().numpy(), tables) and np.array_equal(d[1].cpu().numpy(), lens)
    assert d[4].item() == 3


def test_truncate_leaves_a_length_the_table_cannot_hold():
    rng = np.random.default_rng(7)
    tables, lens, free, count = _state(rng, [50, 90, 33], 16, 6, 4)
    lens = np.array([50, 97, -5], np.int32)            # 96 is the most a table holds
    keep = np.array([20, 40, 0], np.int32)
    d = [_dev(x) for x in (tables, lens, keep, free, np.array([count], np.int32))]
    pkv.truncate_tables(d[0], d[1], d[2], 16, d[3], d[4])
    assert pkv.device_error(clear=True) == pkv.DEVERR_CONTEXT
    want = step.truncate(tables, lens, keep, 16, free, count)
    assert want[1].tolist() == [20, 97, -5]
    for got, w in zip((d[0], d[1], d[3], d[4]), want[:3] + (np.array([want[3]]),)):
        assert np.array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("width", [0, 3])
def test_no_blocks_at_all(width):
    # an empty pool (and empty tables): nothing can be served, nothing is touched
    tables, lens = np.full((2, width), -1, np.int32), np.zeros(2, np.int32)
    free, new = np.zeros(0, np.int32), np.array([0, 5], np.int32)
    d, *_ = _extend(tables, lens, new, 16, free, 0, 8,
                    want_error=pkv.DEVERR_SPACE if width else pkv.DEVERR_POSITION)
    pkv.truncate_tables(d[0], d[1], d[2], 16, d[3], d[4])
    assert pkv.device_error(clear=True) == 0 and d[1].tolist() == [0, 0] and d[4].item() == 0


def test_many_tokens_take_the_wide_path_and_agree_with_the_narrow_one():
    rng = np.random.default_rng(13)
    B, bs = 200, 16
    lens = rng.integers(0, 100, B)
    m = rng.integers(0, 900, B)
    tables, lens, free, count = _state(rng, lens, bs, 64, int((-(-(lens + m) // bs)).sum()))
    assert m.sum() > 65536 > (m // 2).sum()
    _extend(tables, lens, m, bs, free, count, 65536, want_error=pkv.DEVERR_SPACE)
    _extend(tables, lens, m // 2, bs, free, count, 65536)
    _extend(tables, lens, m // 2, bs, free, count, 65537)
    assert (m // 24).sum() < 8192
    _extend(tables, lens, m // 24, bs, free, count, 8192)                           # one launch
    _extend(tables, lens, m // 24, bs, free, count, 8193)                           # two
    _extend(tables, lens, m, bs, free, count, 400001)
    _extend(tables, lens, m, bs, free, count - 900, 400001, want_error=pkv.DEVERR_SPACE)


def test_captured_in_a_graph_and_replayed():
    rng = np.random.default_rng(17)
    bs, B = 16, 12
    tables, lens, free, count = _state(rng, rng.integers(0, 50, B), bs, 9, 60)
    new = np.ones(B, np.int32)
    d = [_dev(x) for x in (tables, lens, new, free, np.array([count], np.int32))]
    out = pkv.extend_tables(d[0].clone(), d[1].clone(), d[2], bs, d[3].clone(), d[4].clone(), B + 2)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pkv.extend_tables(d[0], d[1], d[2], bs, d[3], d[4], B + 2, out=out)
    want = (tables, lens, count)
    for _ in range(20):
        graph.replay()
        t, l, c, slots, seqs, pos, cu, _ = step.extend(want[0], want[1], new, bs, free, want[2], B + 2)
        want = (t, l, c)
        for got, w in zip((d[0], d[1], d[4]) + tuple(out), (t, l, np.array([c]), slots, seqs, pos, cu)):
            assert np.array_equal(got.cpu().numpy(), w)
    assert pkv.device_error(clear=True) == 0


def test_wide_calls_captured_in_a_graph_and_replayed():
    # past one cluster's sizes: two launches a call, the second one's scan beside the first; three
    # calls in a row, lengths and keep_lens written by a kernel right before each
    rng = np.random.default_rng(19)
    bs, B, cap = 16, 300, 90000
    lens = rng.integers(0, 40, B)
    tables, lens, free, count = _state(rng, lens, bs, 60, 26000)
    new = rng.integers(0, 500, B).astype(np.int32)
    assert new.sum() > 32768 and min(B * 60, len(free)) > 16384
    d = [_dev(x) for x in (tables, lens, free, np.array([count], np.int32))]
    news, keep, zero = _dev(new), torch.empty(B, dtype=torch.int32, device=DEV), _dev(0 * new)
    out = pkv.extend_tables(d[0].clone(), d[1].clone(), zero, bs, d[2].clone(), d[3].clone(), cap)

    def steps():
        pkv.extend_tables(d[0], d[1], news + zero, bs, d[2], d[3], cap, out=out)
        torch.div(d[1], 2, rounding_mode="floor", out=keep)
        pkv.truncate_tables(d[0], d[1], keep, bs, d[2], d[3])
        torch.sub(d[1], d[1], out=keep)
        pkv.truncate_tables(d[0], d[1], keep, bs, d[2], d[3])

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        steps()
    for run in (graph.replay, steps, graph.replay):
        run()
        t, l, c, slots, seqs, pos, cu, refused = step.extend(tables, lens, new, bs, free, count, cap)
        assert not refused
        for keep_h in (l // 2, 0 * l):
            t, l, free, c = step.truncate(t, l, keep_h.astype(np.int32), bs, free, c)
        tables, lens, count = t, l, c
        for got, w in zip(d + list(out), (t, l, free, np.array([c]), slots, seqs, pos, cu)):
            assert np.array_equal(got.cpu().numpy(), w)
    assert pkv.device_error(clear=True) == 0


def test_binding_refuses_wrong_types_and_shapes():
    z = torch.zeros(2, 4, dtype=torch.int32, device=DEV)
    n, one = z[0, :2].clone(), z[0, :1].clone()
    bad = [
        lambda: pkv.extend_tables(z.long(), n, n, 16, n, one, 4),
        lambda: pkv.extend_tables(z[:1], n, n, 16, n, one, 4),
        lambda: pkv.extend_tables(z, n, n[:1], 16, n, one, 4),
        lambda: pkv.extend_tables(z, n, n, 12, n, one, 4),
        lambda: pkv.extend_tables(z.t(), z[0].clone(), z[0].clone(), 16, n, one, 4),
        lambda: pkv.truncate_tables(z, n, n.float(), 16, n, one),
        lambda: pkv.truncate_tables(z, n, n, 16, n.cpu(), one),
    ]
    for call in bad:
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status == pkv.EINVAL


@pytest.mark.parametrize("given", [False, True])
def test_neither_sequences_nor_tokens_still_give_a_total(given):
    # an idle step: the total of no tokens is written, whatever the memory held before
    z = torch.zeros(0, 4, dtype=torch.int32, device=DEV)
    e, free = z[:, 0].clone(), torch.arange(5, dtype=torch.int32, device=DEV)
    count = torch.full((1,), 5, dtype=torch.int32, device=DEV)
    wide = torch.zeros(0, dtype=torch.int64, device=DEV)
    cu = torch.full((1,), 77, dtype=torch.int32, device=DEV)
    if given:
        pkv.extend_tables(z, e, e, 16, free, count, 0, out=(wide, e, wide, cu))
    else:
        del cu          # the next allocation of this size takes its place
        cu = pkv.extend_tables(z, e, e, 16, free, count, 0)[3]
    assert cu.tolist() == [0] and count.item() == 5 and free.tolist() == [0, 1, 2, 3, 4]
    # captured as well
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        pkv.extend_tables(z, e, e, 16, free, count, 0, out=(wide, e, wide, cu))
    cu.fill_(77)
    graph.replay()
    assert cu.tolist() == [0] and pkv.device_error(clear=True) == 0


@pytest.mark.parametrize("count", [999, -1])
@pytest.mark.parametrize("max_tokens", [300, 8193])     # one launch, two
def test_a_free_count_no_stack_has_stays_as_it_is(count, max_tokens):
    rng = np.random.default_rng(21)
    tables, lens, free, _ = _state(rng, [20, 16, 40, 5, 0, 31], 16, 6, 9)
    new = np.array([40, 0, 8, 40, 3, 1], np.int32)     # the third and the last need no block
    keep = np.array([19, 16, 0, 0, 0, 31], np.int32)   # the first keeps its blocks
    d = [_dev(x) for x in (tables, lens, new, free, np.array([count], np.int32))]
    pkv.extend_tables(d[0], d[1], d[2], 16, d[3], d[4], max_tokens)
    assert pkv.device_error(clear=True) == pkv.DEVERR_SPACE and d[4].item() == count
    assert np.array_equal(d[0].cpu().numpy(), tables) and np.array_equal(d[3].cpu().numpy(), free)
    assert d[1].tolist() == [20, 16, 48, 5, 0, 32]
    d[1].copy_(_dev(lens))
    pkv.truncate_tables(d[0], d[1], _dev(keep), 16, d[3], d[4])
    assert pkv.device_error(clear=True) == pkv.DEVERR_SPACE and d[4].item() == count
    assert np.array_equal(d[0].cpu().numpy(), tables) and np.array_equal(d[3].cpu().numpy(), free)
    assert np.array_equal(d[1].cpu().numpy(), lens)
