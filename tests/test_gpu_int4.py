"""GPU parity of the 4-bit cache: append, widening, decode and fused append + decode.

Appended bytes must equal the oracle's, every one of the pool; attention must lie within the
bound the oracle derives for each element. Pools are quantised on the host by the oracle, and
every slot that no sequence may read holds NaN scales and minima."""
import math

import numpy as np
import pytest
import torch

from oracle import int4
from paged_kv_cache_147_gb300 import pkv

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a, dtype=None):
    t = torch.as_tensor(np.ascontiguousarray(a))
    return t.to(DEV) if dtype is None else t.to(device=DEV, dtype=dtype)


def _rows(rng, shape, outliers=True):
    x = rng.standard_normal(shape + (128,))
    if outliers:
        x[..., rng.choice(128, 5, replace=False)] *= 8
        x += rng.standard_normal(128)
    return x.astype(np.float16)


def _case(lens, bs=16, hq=12, hkv=2, q_len=1, seed=0, extra=3):
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    nblk = (lens + bs - 1) // bs
    nb = int(nblk.sum()) + extra
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((len(lens), max(int(nblk.max()), 1) + 1), -1, np.int32)
    used = np.zeros((nb, bs), bool)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        at += n
        for j in range(n):
            used[tables[b, j], :max(0, min(bs, int(lens[b]) - j * bs))] = True
    k = int4.quantise(_rows(rng, (nb, hkv, bs)))
    v = int4.quantise(_rows(rng, (nb, hkv, bs), outliers=False))
    for pool in (k, v):   # what no one may read: NaN everywhere
        pool.transpose(0, 2, 1, 3)[~used] = 0xFF
    q = rng.standard_normal((len(lens), q_len, hq, 128)).astype(np.float16)
    return k, v, tables, lens, q


def _close(out, want, tol, what=""):
    err = np.abs(out.float().cpu().numpy().astype(np.float64) - want)
    worst = np.unravel_index(np.nanargmax(err - tol), err.shape)
    assert (err <= tol).all(), f"{what}: off {err[worst]:.3g} of {tol[worst]:.3g} at {worst}"


def _decode(k, v, tables, lens, q, scale, ws=None):
    qd = _dev(q)
    out = torch.full_like(qd, float("nan"))
    if ws is None:
        ws = pkv.make_workspace(q.shape[0], q.shape[1], q.shape[2], k.shape[1])
    pkv.paged_attn_decode_int4(out, qd, _dev(k), _dev(v), _dev(tables), _dev(lens), scale, ws)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    return out


# ----------------------------------------------------------------------------- append, widen
@pytest.mark.parametrize("hkv,T,bs", [(2, 1, 16), (8, 33, 16), (3, 70, 64), (1, 2, 256)])
def test_append_bytes_equal_the_oracle(hkv, T, bs):
    rng = np.random.default_rng(hkv * 100 + T)
    nb = 8
    k, v = _rows(rng, (T, hkv)), _rows(rng, (T, hkv))
    k[0, 0, :4] = [65504, -65504, 0, 2.0 ** -24]           # the largest range
    k[0, 0, 32:64] = 1.25                                   # s = 0
    k[0, 0, 64:96] = (np.arange(32) % 31) * np.float16(2.0 ** -24)   # subnormals
    v[0, 0, 7] = np.nan
    v[0, 0, 40] = np.inf
    # ties: s = 2, z = 0, values on the borders between codes
    v[0, 0, 64:96] = np.arange(32).astype(np.float16)
    v[0, 0, 95] = 30
    slots = rng.choice(nb * bs, size=T, replace=False).astype(np.int64)
    if T > 3:
        slots[2] = -1
    kc = rng.integers(0, 256, (nb, hkv, bs, 80), dtype=np.uint8)
    vc = rng.integers(0, 256, (nb, hkv, bs, 80), dtype=np.uint8)
    kd, vd = _dev(kc), _dev(vc)
    pkv.kv_append_int4(_dev(k), _dev(v), _dev(slots), kd, vd)
    torch.cuda.synchronize()
    int4.append(k, v, slots, kc, vc)
    assert np.array_equal(kd.cpu().numpy(), kc) and np.array_equal(vd.cpu().numpy(), vc)
    assert pkv.device_error(clear=True) == 0


def test_append_bytes_over_all_magnitudes():
    # groups whose values span fp16's whole range of exponents, where x - z rounds
    rng = np.random.default_rng(11)
    T, hkv = 400, 4
    bits = rng.integers(0, 1 << 16, (2, T, hkv, 128)).astype(np.uint16)
    x = bits.view(np.float16)
    x = np.where(np.isfinite(x), x, np.float16(0.1))
    x[:, :200] *= np.float16(2.0 ** -9)
    slots = np.arange(T, dtype=np.int64)
    kc, vc = (np.zeros((T // 16, hkv, 16, 80), np.uint8) for _ in range(2))
    kd, vd = _dev(kc), _dev(vc)
    pkv.kv_append_int4(_dev(x[0]), _dev(x[1]), _dev(slots), kd, vd)
    int4.append(x[0], x[1], slots, kc, vc)
    assert np.array_equal(kd.cpu().numpy(), kc) and np.array_equal(vd.cpu().numpy(), vc)


@pytest.mark.parametrize("hkv,T,bs", [(1, 16389, 16), (8, 2050, 64), (3, 5465, 32)])
def test_large_appends_write_the_same_bytes(hkv, T, bs):
    # 16384 rows and more go a group per thread: any bits (NaN and infinities among them), odd
    # numbers of tokens, skipped and refused slots
    rng = np.random.default_rng(T)
    x = rng.integers(0, 1 << 16, (2, T, hkv, 128)).astype(np.uint16).view(np.float16)
    x[:, ::2] = rng.standard_normal(x[:, ::2].shape).astype(np.float16)
    x[:, 5] = 0.5                                            # s = 0
    x[:, 7, :, :32] = np.arange(32).astype(np.float16)      # ties between codes
    nb = T // bs + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int64)
    slots[[3, 4, T - 1]] = -1
    slots[6] = nb * bs + 5
    pools = [rng.integers(0, 256, (nb, hkv, bs, 80), dtype=np.uint8) for _ in range(2)]
    d = [_dev(p) for p in pools]
    pkv.kv_append_int4(_dev(x[0]), _dev(x[1]), _dev(slots), *d)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_SLOT
    int4.append(x[0], x[1], slots, *pools)
    for got, want in zip(d, pools):
        assert np.array_equal(got.cpu().numpy(), want)


def test_append_skips_a_slot_past_the_pool_and_says_so():
    rng = np.random.default_rng(2)
    k = _rows(rng, (3, 2))
    pools = [torch.zeros(2, 2, 16, 80, dtype=torch.uint8, device=DEV) for _ in range(2)]
    pkv.kv_append_int4(_dev(k), _dev(k), _dev(np.array([5, 32, 1 << 40], np.int64)), *pools)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_SLOT
    want = np.zeros((2, 2, 16, 80), np.uint8)
    int4.append(k[:1], k[:1], [5], want, want.copy())
    assert np.array_equal(pools[0].cpu().numpy(), want)


@pytest.mark.parametrize("hkv,bs", [(2, 16), (5, 64), (1, 256)])
def test_widen_rounds_every_value_once(hkv, bs):
    rng = np.random.default_rng(bs)
    k = int4.quantise(_rows(rng, (6, hkv, bs)) * np.float16(20))
    v = int4.quantise((_rows(rng, (6, hkv, bs)) * np.float16(2.0 ** -12)))
    src, dst = np.array([5, 0, 5, 99, 2], np.int32), np.array([1, 6, 0, 2, -1], np.int32)
    ko, vo = (torch.full((7, hkv, bs, 128), 7.0, dtype=torch.float16, device=DEV) for _ in range(2))
    pkv.widen_blocks_int4(_dev(k), _dev(v), _dev(src), _dev(dst), ko, vo)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_BLOCK_ID
    for pool, out in ((k, ko), (v, vo)):
        want = np.full((7, hkv, bs, 128), 7.0, np.float16)
        want[[1, 6, 0]] = int4.values(pool[[5, 0, 5]]).astype(np.float16)
        assert np.array_equal(out.cpu().numpy(), want)


def test_copy_blocks_moves_4_bit_blocks():
    rng = np.random.default_rng(4)
    k, v = (int4.quantise(_rows(rng, (5, 2, 16))) for _ in range(2))
    kd, vd = _dev(k), _dev(v)
    pkv.copy_blocks(kd.view(torch.float16), vd.view(torch.float16),
                    _dev(np.array([3], np.int32)), _dev(np.array([0], np.int32)))
    k[0], v[0] = k[3], v[3]
    assert np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)


@pytest.mark.parametrize("row", [80, 128])     # 4-bit rows, E4M3 codes
def test_copy_blocks_of_byte_pools_moves_those_blocks_and_no_others(row):
    rng = np.random.default_rng(row)
    pools = [rng.integers(0, 256, (3, 7, 2, 16, row), dtype=np.uint8) for _ in range(2)]
    src, dst = np.array([3, 5], np.int32), np.array([0, 6], np.int32)
    d = [_dev(p) for p in pools]
    pkv.copy_blocks(*d, _dev(src), _dev(dst))                               # every layer
    pkv.copy_blocks(d[0][1], d[1][1], _dev(src[:1]), _dev(dst[:1] + 1))     # one of them
    for p, got in zip(pools, d):
        p[:, dst] = p[:, src]
        p[1, 1] = p[1, 3]
        assert np.array_equal(got.cpu().numpy(), p)
    assert pkv.device_error(clear=True) == 0


# ----------------------------------------------------------------------------- decode
CASES = [
    ([38, 101], 16, 12, 2, 1),                        # the tiny batch
    ([1], 16, 1, 1, 1),                               # one token, one head
    ([1, 2, 15, 16, 17, 31, 32, 33, 47, 49], 16, 12, 2, 1),
    ([300, 47], 16, 64, 8, 1),                        # 8 rows: one full tile
    ([77, 200, 5], 16, 8, 4, 2),
    ([500, 70], 64, 16, 2, 1),
    ([33, 1, 60], 16, 4, 4, 3),                       # drafts, one context shorter than its drafts
    ([20000], 16, 12, 2, 1),                          # one long sequence over many CTAs
    ([5] * 700, 16, 12, 2, 1),                        # many short ones
    ([2, 40, 0, 9], 16, 12, 2, 1),                    # an empty sequence
    ([300, 90, 33], 32, 9, 1, 1),                     # 9 rows: two tiles
    ([257, 64], 128, 32, 2, 1),                       # 16 rows
    ([150, 1, 31, 700], 16, 12, 2, 4),                # 24 rows: four tiles, one of them unused
    ([400, 17, 2], 256, 32, 4, 4),                    # 32 rows
    ([129, 640], 16, 7, 1, 1),                        # 7 rows
    ([1500] * 40, 16, 16, 8, 1),
]


@pytest.mark.parametrize("lens,bs,hq,hkv,q_len", CASES)
def test_decode_matches_oracle(lens, bs, hq, hkv, q_len):
    k, v, tables, lens, q = _case(lens, bs, hq, hkv, q_len, seed=len(lens) + bs)
    scale = 1 / math.sqrt(128)
    out = _decode(k, v, tables, lens, q, scale)
    want, tol = int4.attention(q, k, v, tables, lens, scale)
    _close(out, want, tol, f"bs={bs} G={hq // hkv} q_len={q_len}")


def test_decode_with_scores_that_climb_and_large_scale():
    # keys that grow along the context, so that the running maximum has to follow
    k, v, tables, lens, q = _case([900, 333], 16, 8, 2, 2, seed=9)
    rng = np.random.default_rng(1)
    for b, n in enumerate(lens):
        for t in range(int(n)):
            row = (rng.standard_normal((2, 128)) + q[b, 0, :2] * (t / 150)).astype(np.float16)
            k[tables[b, t // 16], :, t % 16] = int4.quantise(row)
    out = _decode(k, v, tables, lens, q, 0.2)
    want, tol = int4.attention(q, k, v, tables, lens, 0.2)
    _close(out, want, tol)


@pytest.mark.parametrize("gain_q,gain_v", [(1e-3, 1e-4), (200.0, 300.0)])
def test_decode_over_small_and_large_magnitudes(gain_q, gain_v):
    k, v, tables, lens, q = _case([200, 64, 7], 16, 12, 2, 1, seed=6)
    rng = np.random.default_rng(8)
    used = k[..., 64:].view(np.uint16)[..., 0] != 0xFFFF
    x = (rng.standard_normal(used.shape + (128,)) * gain_v).astype(np.float16)
    v[used] = int4.quantise(x)[used]
    q = (q.astype(np.float32) * gain_q).astype(np.float16)
    scale = 0.05 / gain_q
    out = _decode(k, v, tables, lens, q, scale)
    want, tol = int4.attention(q, k, v, tables, lens, scale)
    _close(out, want, tol)


def test_decode_repeats_bit_for_bit_and_whatever_blocks_hold_the_data():
    k, v, tables, lens, q = _case([900, 33, 1500], seed=3)
    ws = pkv.make_workspace(3, 1, 12, 2)
    a = _decode(k, v, tables, lens, q, 0.1, ws)
    assert torch.equal(a, _decode(k, v, tables, lens, q, 0.1, ws))
    perm = np.random.default_rng(0).permutation(k.shape[0]).astype(np.int32)
    k2, v2 = np.empty_like(k), np.empty_like(v)
    k2[perm], v2[perm] = k, v
    t2 = np.where(tables >= 0, perm[tables], -1).astype(np.int32)
    assert torch.equal(a, _decode(k2, v2, t2, lens, q, 0.1, ws))


def test_decode_past_32_bit_byte_offsets():
    # 28 M rows of 80 bytes: 2.2 GB a pool, the sequence in its last blocks
    nb, hkv, bs = 27400, 4, 256
    k, v, tables, lens, q = _case([700], bs, 8, hkv, 1, seed=12, extra=0)
    kd, vd = (torch.zeros(nb, hkv, bs, 80, dtype=torch.uint8, device=DEV) for _ in range(2))
    n = k.shape[0]
    kd[nb - n:], vd[nb - n:] = _dev(k), _dev(v)
    t = np.where(tables >= 0, tables + nb - n, -1).astype(np.int32)
    qd = _dev(q)
    out = torch.empty_like(qd)
    pkv.paged_attn_decode_int4(out, qd, kd, vd, _dev(t), _dev(lens), 0.1,
                               pkv.make_workspace(1, 1, 8, hkv))
    want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    _close(out, want, tol)
    rng = np.random.default_rng(1)
    x = _rows(rng, (2, hkv))
    slots = np.array([nb * bs - 1, 3], np.int64)
    pkv.kv_append_int4(_dev(x), _dev(x), _dev(slots), kd, vd)
    assert np.array_equal(kd[-1, :, -1].cpu().numpy(), int4.quantise(x[0]))
    assert pkv.device_error(clear=True) == 0


def test_decode_bad_block_id_and_length_set_bits_without_fault():
    k, v, tables, lens, q = _case([300, 47, 90], seed=31)
    bad, long = tables.copy(), lens.copy()
    bad[0, 3] = k.shape[0] + 9
    qd = _dev(q)
    ws = pkv.make_workspace(3, 1, 12, 2)
    out = torch.empty_like(qd)
    pkv.paged_attn_decode_int4(out, qd, _dev(k), _dev(v), _dev(bad), _dev(lens), 0.1, ws)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_BLOCK_ID
    want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    _close(out[1:], want[1:], tol[1:])
    long[1] = -4
    pkv.paged_attn_decode_int4(out, qd, _dev(k), _dev(v), _dev(tables), _dev(long), 0.1, ws)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == pkv.DEVERR_CONTEXT
    _close(out[2:], want[2:], tol[2:])
    assert (out[1] == 0).all()


# ----------------------------------------------------------------------------- fused append
def _new_slots(tables, lens, q_len, bs):
    pos = lens[:, None].astype(np.int64) - q_len + np.arange(q_len)
    ids = np.take_along_axis(tables, np.maximum(pos, 0) // bs, 1).astype(np.int64)
    return np.where(pos < 0, -1, ids * bs + pos % bs).reshape(-1)


@pytest.mark.parametrize("lens,bs,hq,hkv,q_len", [
    ([38, 101], 16, 12, 2, 1),
    ([33, 16, 2, 100], 16, 8, 4, 2),                  # new rows across blocks
    ([64, 5, 31, 3, 1], 16, 4, 4, 4),                 # fewer tokens than drafts
    ([500, 70, 1], 64, 16, 2, 1),
    ([18, 50, 97, 16], 16, 8, 4, 4),                  # drafts across both chunks of a stage
    ([40, 300, 5], 32, 12, 2, 4),                     # 24 rows
    ([700, 90, 31], 16, 24, 2, 1),                    # 12 rows
    ([5] * 300, 16, 12, 2, 1),
])
def test_fused_append_decode_matches_oracle(lens, bs, hq, hkv, q_len):
    k, v, tables, lens, q = _case(lens, bs, hq, hkv, q_len, seed=len(lens) * 7 + q_len)
    rng = np.random.default_rng(99)
    kn, vn = (_rows(rng, (len(lens) * q_len, hkv)) for _ in range(2))
    kd, vd, qd = _dev(k), _dev(v), _dev(q)
    out = torch.full_like(qd, float("nan"))
    ws = pkv.make_workspace(len(lens), q_len, hq, hkv)
    pkv.paged_attn_decode_append_int4(out, qd, _dev(kn), _dev(vn), kd, vd, _dev(tables),
                                      _dev(lens), 0.09, ws)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    int4.append(kn, vn, _new_slots(tables, lens, q_len, bs), k, v)
    assert np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)
    want, tol = int4.attention(q, k, v, tables, lens, 0.09)
    _close(out, want, tol)


def test_fused_steps_in_a_row_with_and_without_early_start():
    # three steps with the lengths advanced by a copy in between, captured in a graph as well
    k, v, tables, lens, q = _case([61, 30, 95], 16, 12, 2, 1, seed=21)
    rng = np.random.default_rng(5)
    rows = [(_rows(rng, (3, 2)), _rows(rng, (3, 2))) for _ in range(3)]
    ws = pkv.make_workspace(3, 1, 12, 2)
    qd, td = _dev(q), _dev(tables)
    step_lens = [_dev(lens - 2 + i) for i in range(3)]
    news = [(_dev(a), _dev(b)) for a, b in rows]
    outs = [torch.empty_like(qd) for _ in range(3)]
    kr, vr = k.copy(), v.copy()
    wants = []
    for i in range(3):
        li = (lens - 2 + i).astype(np.int32)
        int4.append(rows[i][0], rows[i][1], _new_slots(tables, li, 1, 16), kr, vr)
        wants.append(int4.attention(q, kr, vr, tables, li, 0.1))
    for early in (True, False):
        before = pkv.set_early_start(early)
        try:
            kd, vd, cl = _dev(k), _dev(v), torch.empty(3, dtype=torch.int32, device=DEV)

            def steps():
                for i in range(3):
                    cl.copy_(step_lens[i])
                    pkv.paged_attn_decode_append_int4(outs[i], qd, *news[i], kd, vd, td, cl, 0.1, ws)

            steps()
            for i in range(3):
                _close(outs[i], *wants[i], f"step {i}")
            assert np.array_equal(kd.cpu().numpy(), kr)
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    steps()
            torch.cuda.synchronize()
            kd.copy_(_dev(k))
            vd.copy_(_dev(v))
            for o in outs:
                o.fill_(float("nan"))
            graph.replay()
            for i in range(3):
                _close(outs[i], *wants[i], f"replayed step {i}")
            assert np.array_equal(vd.cpu().numpy(), vr)
        finally:
            pkv.set_early_start(before)


@pytest.mark.parametrize("lens,width,hq,hkv,q_len", [
    ([33, 1], 300, 3, 3, 2),                          # 12 warps, most of them without a stage
    ([17, 40, 2], 256, 12, 2, 1),
    ([33, 47, 96, 9], 257, 8, 4, 4),
    ([64, 5], 512, 24, 2, 2),                         # 24 rows
])
def test_fused_append_of_short_contexts_in_long_tables(lens, width, hq, hkv, q_len):
    k, v, tables, lens, q = _case(lens, 16, hq, hkv, q_len, seed=width)
    wide = np.full((len(lens), width), -1, np.int32)
    wide[:, :tables.shape[1]] = tables
    rng = np.random.default_rng(98)
    kn, vn = (_rows(rng, (len(lens) * q_len, hkv)) for _ in range(2))
    kd, vd, qd = _dev(k), _dev(v), _dev(q)
    out = torch.full_like(qd, float("nan"))
    pkv.paged_attn_decode_append_int4(out, qd, _dev(kn), _dev(vn), kd, vd, _dev(wide), _dev(lens),
                                      0.09, pkv.make_workspace(len(lens), q_len, hq, hkv))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    int4.append(kn, vn, _new_slots(wide, lens, q_len, 16), k, v)
    assert np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)
    want, tol = int4.attention(q, k, v, wide, lens, 0.09)
    _close(out, want, tol)


@pytest.mark.parametrize("width,q_len", [(7, 1), (7, 3), (260, 1), (260, 3)])
@pytest.mark.parametrize("what", ["block", "last block", "negative", "past the table"])
def test_fused_append_with_a_bad_block_or_length_writes_nothing_else(width, q_len, what):
    # the second of four sequences is bad; the others, and every byte that is not theirs, as ever
    hq, hkv, bs = 8, 2, 16
    k, v, tables, lens, q = _case([100, 97, 18, 60], bs, hq, hkv, q_len, seed=37, extra=300)
    rng = np.random.default_rng(6)
    full = np.full((4, width), -1, np.int32)
    full[:, :7] = tables[:, :7]
    spare = np.setdiff1d(np.arange(k.shape[0]), tables)[:width]
    own = full[1] < 0
    full[1, own] = spare[:own.sum()]              # a table that is full: every entry could be written
    kn, vn = (_rows(rng, (4 * q_len, hkv)) for _ in range(2))
    said, bits = lens.copy(), pkv.DEVERR_CONTEXT
    if what == "block":
        full[1, 2], bits = k.shape[0] + 5, pkv.DEVERR_BLOCK_ID
    elif what == "last block":                    # where new rows would go
        full[1, (lens[1] - 1) // bs], bits = -7, pkv.DEVERR_BLOCK_ID
    else:
        said[1] = -4 if what == "negative" else width * bs + 1
    kd, vd, qd = _dev(k), _dev(v), _dev(q)
    out = torch.full_like(qd, float("nan"))
    pkv.paged_attn_decode_append_int4(out, qd, _dev(kn), _dev(vn), kd, vd, _dev(full), _dev(said),
                                      0.1, pkv.make_workspace(4, q_len, hq, hkv))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == bits
    slots = _new_slots(np.where(full < k.shape[0], full, -1), lens, q_len, bs).reshape(4, q_len)
    if bits == pkv.DEVERR_CONTEXT:
        slots[1] = -1
        assert (out[1] == 0).all()
    int4.append(kn, vn, slots.reshape(-1), k, v)
    assert np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)
    some = [0, 2, 3]
    want, tol = int4.attention(q[some], k, v, full[some], lens[some], 0.1)
    _close(out[some], want, tol)


@pytest.mark.parametrize("lens,bs,hq,hkv,q_len", [
    ([1, 18, 33, 0, 250], 16, 9, 1, 1),               # 9 rows
    ([40, 3, 200], 16, 12, 4, 5),                     # 15
    ([40, 16, 200], 32, 17, 1, 1),                    # 17
    ([64, 9, 30], 16, 5, 1, 5),                       # 25
    ([64, 31, 700], 16, 32, 1, 1),                    # 32 heads
    ([64, 31, 33, 100], 16, 2, 2, 32),                # 32 new tokens
])
def test_fused_append_of_9_to_32_rows(lens, bs, hq, hkv, q_len):
    test_fused_append_decode_matches_oracle(lens, bs, hq, hkv, q_len)


@pytest.mark.parametrize("lens,bs,hq,hkv,q_len", [
    ([5000, 30], 16, 12, 2, 1),                       # few units, long tables: 12 warps share each
    ([4300, 0, 77, 4096], 64, 8, 4, 4),
    ([9000], 256, 8, 1, 1),
    ([33, 1], 4096 // 16, 3, 3, 2),                   # two blocks of 256: short contexts in there
])
def test_fused_append_of_few_sequences_with_long_tables(lens, bs, hq, hkv, q_len):
    if max(lens) < 4096:   # widen the tables without lengthening the contexts
        k, v, tables, lens, q = _case(lens, bs, hq, hkv, q_len, seed=77)
        wide = np.full((len(lens), 20), -1, np.int32)
        wide[:, :tables.shape[1]] = tables
        out = _decode(k, v, wide, lens, q, 0.09)
        want, tol = int4.attention(q, k, v, wide, lens, 0.09)
        _close(out, want, tol)
    else:
        test_fused_append_decode_matches_oracle(lens, bs, hq, hkv, q_len)


@pytest.mark.parametrize("hq,hkv,q_len", [(24, 1, 1), (1, 1, 24), (4, 1, 8), (1, 1, 32)])
def test_fused_append_of_as_many_sequences_as_a_call_takes(hq, hkv, q_len):
    # 4096 sequences: two of three empty (padding), the others short
    lens = np.zeros(4096, np.int32)
    lens[::3] = np.random.default_rng(2).integers(1, 50, len(lens[::3]))
    test_fused_append_decode_matches_oracle(lens, 16, hq, hkv, q_len)


@pytest.mark.parametrize("scale", [-0.1, 0.0, -3.0])
def test_decode_with_a_scale_that_is_not_positive(scale):
    k, v, tables, lens, q = _case([900, 33, 2, 70], 16, 12, 2, 2, seed=17)
    out = _decode(k, v, tables, lens, q, scale)
    want, tol = int4.attention(q, k, v, tables, lens, scale)
    _close(out, want, tol)


@pytest.mark.parametrize("hq,q_len", [(32, 1), (48, 4)])
def test_decode_of_long_slices(hq, q_len):
    # 20 sequences of up to 6000 tokens, 8 kv heads: more stages a warp than it sums in one go. Keys
    # grow along the context (the reference moves from one sum to the next), and values past
    # two thirds of it pass the scale that moves the reference by kShift.
    hkv, bs, B = 8, 16, 20
    rng = np.random.default_rng(3)
    lens = rng.integers(5000, 6000, B).astype(np.int32)
    nblk = (lens + bs - 1) // bs
    nb = int(nblk.sum())
    tables = np.full((B, int(nblk.max())), -1, np.int32)
    perm = rng.permutation(nb).astype(np.int32)
    pos = np.full((nb, bs), 0.0)
    at = 0
    for b, n in enumerate(nblk):
        tables[b, :n] = perm[at:at + n]
        pos[tables[b, :n]] = (np.arange(n * bs) / lens[b]).reshape(n, bs)
        at += n
    q = rng.standard_normal((B, q_len, hq, 128)).astype(np.float16)
    kd, vd = (torch.zeros(nb, hkv, bs, 80, dtype=torch.uint8, device=DEV) for _ in range(2))
    gen = torch.Generator(DEV).manual_seed(5)
    share = _dev(pos.reshape(-1), torch.float32)[:, None, None]
    slots = torch.arange(nb * bs, device=DEV)
    kx = torch.randn(nb * bs, hkv, 128, device=DEV, generator=gen) * (0.2 + share)
    vx = torch.randn(nb * bs, hkv, 128, device=DEV, generator=gen) * torch.where(share > 0.66, 20., 1.)
    pkv.kv_append_int4(kx.half(), vx.half(), slots, kd, vd)
    qd = _dev(q)
    out = torch.full_like(qd, float("nan"))
    pkv.paged_attn_decode_int4(out, qd, kd, vd, _dev(tables), _dev(lens), 0.2,
                               pkv.make_workspace(B, q_len, hq, hkv))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    k, v = kd.cpu().numpy(), vd.cpu().numpy()
    assert (int4.parts(v)[1] >= 2).any() and (int4.parts(v)[1] < 2).any()
    pick = [0, 7, 19]
    want, tol = int4.attention(q[pick], k, v, tables[pick], lens[pick], 0.2)
    _close(out[pick], want, tol)
    assert torch.isfinite(out).all()


def _same_nan_and_close(out, want, tol):
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= tol[ok]).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_decode_keeps_a_bad_query_to_its_row(what):
    k, v, tables, lens, q = _case([130, 40], 16, 12, 2, 2, seed=23)
    q[0, 1, 7, 100] = what
    out = _decode(k, v, tables, lens, q, 0.1)
    with np.errstate(invalid="ignore"):
        want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    assert np.isnan(want[0, 1, 7]).all() and np.isnan(want).sum() == 128
    _same_nan_and_close(out, want, tol)


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("hq,hkv,q_len", [(2, 1, 4), (4, 1, 4), (12, 2, 4), (1, 1, 32)])
@pytest.mark.parametrize("fused", [False, True])
def test_a_bad_query_that_sees_no_token_gets_zeros(what, hq, hkv, q_len, fused):
    # contexts shorter than their drafts: the first queries see nothing and are padding
    k, v, tables, lens, q = _case([2, 40, 1], 16, hq, hkv, q_len, seed=24)
    blind = [(b, i) for b in (0, 1, 2) for i in range(q_len) if lens[b] - q_len + i < 0]
    for b, i in blind:
        q[b, i] = what
    if fused:
        rng = np.random.default_rng(7)
        kn, vn = (_rows(rng, (3 * q_len, hkv)) for _ in range(2))
        qd = _dev(q)
        out = torch.full_like(qd, float("nan"))
        pkv.paged_attn_decode_append_int4(out, qd, _dev(kn), _dev(vn), _dev(k), _dev(v), _dev(tables),
                                          _dev(lens), 0.1, pkv.make_workspace(3, q_len, hq, hkv))
        assert pkv.device_error(clear=True) == 0
        int4.append(kn, vn, _new_slots(tables, lens, q_len, 16), k, v)
    else:
        out = _decode(k, v, tables, lens, q, 0.1)
    want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    _close(out, want, tol)
    assert len(blind) >= 5 and all((out[b, i] == 0).all() for b, i in blind)


@pytest.mark.parametrize("q_len,hq,hkv", [(1, 12, 2), (4, 12, 2), (3, 6, 2)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("back", [0, 1, 2])
def test_decode_keeps_a_bad_row_to_the_queries_that_see_it(q_len, hq, hkv, which, back):
    # one group of a row, `back` tokens from the end, is NaN (what the append makes of a NaN)
    lens = [70, 33, 17, 48]
    k, v, tables, lens, q = _case(lens, 16, hq, hkv, q_len, seed=29)
    pool = k if which == "k" else v
    for b in (0, 1, 3):
        t = int(lens[b]) - 1 - back
        row = pool[tables[b, t // 16], 1, t % 16]
        row[32:48] = 0
        row[72:76] = (0xFF, 0x7F, 0xFF, 0x7F)
    out = _decode(k, v, tables, lens, q, 0.1)
    with np.errstate(invalid="ignore"):
        want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    sees = min(q_len, back + 1)
    assert np.isnan(want).sum() == 3 * sees * (hq // hkv) * (128 if which == "k" else 32)
    _same_nan_and_close(out, want, tol)


def test_fused_append_of_a_nan_row():
    # the last of three new tokens is NaN in one group: earlier drafts and other heads do not see it
    k, v, tables, lens, q = _case([70, 35, 18], 16, 8, 2, 3, seed=33)
    rng = np.random.default_rng(4)
    kn, vn = (_rows(rng, (9, 2)) for _ in range(2))
    vn[2, 0, 40] = np.nan
    vn[5, 1, 127] = np.inf
    kd, vd, qd = _dev(k), _dev(v), _dev(q)
    out = torch.empty_like(qd)
    pkv.paged_attn_decode_append_int4(out, qd, _dev(kn), _dev(vn), kd, vd, _dev(tables), _dev(lens),
                                      0.1, pkv.make_workspace(3, 3, 8, 2))
    assert pkv.device_error(clear=True) == 0
    int4.append(kn, vn, _new_slots(tables, lens, 3, 16), k, v)
    assert np.array_equal(kd.cpu().numpy(), k) and np.array_equal(vd.cpu().numpy(), v)
    with np.errstate(invalid="ignore"):
        want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    assert np.isnan(want).sum() == 2 * 4 * 32
    _same_nan_and_close(out, want, tol)


def test_two_captured_decodes_at_once_with_a_workspace_each():
    cases = [_case(n, 16, 12, 2, 1, seed=i) for i, n in enumerate(([3000, 900], [2500, 17, 1200]))]
    want = [int4.attention(c[4], *c[:4], 0.1) for c in cases]
    runs = []
    for k, v, tables, lens, q in cases:
        a = [_dev(x) for x in (q, k, v, tables, lens)]
        out, ws = torch.empty_like(a[0]), pkv.make_workspace(len(lens), 1, 12, 2)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(4):
                pkv.paged_attn_decode_int4(out, *a, 0.1, ws)
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


def test_one_workspace_for_calls_of_different_sizes():
    # counters of a large batch lie where a smaller call's partials must not: many split units,
    # then one sequence with 24 rows, and again
    big = _case([1300] * 40, 16, 8, 8, 1, seed=51)
    one = _case([6000], 16, 12, 2, 4, seed=52)
    few = _case([4100, 700, 5000], 16, 8, 8, 1, seed=53)
    ws = pkv.make_workspace(40, 4, 48, 8)
    runs = []
    for k, v, tables, lens, q in (few, big, one, big, few, one, big):
        a = [_dev(x) for x in (q, k, v, tables, lens)]
        out = torch.full_like(a[0], float("nan"))
        pkv.paged_attn_decode_int4(out, *a, 0.1, ws)
        runs.append((out, q, k, v, tables, lens))
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    assert torch.equal(runs[0][0], runs[4][0]) and torch.equal(runs[2][0], runs[5][0])
    assert torch.equal(runs[1][0], runs[3][0]) and torch.equal(runs[1][0], runs[6][0])
    for out, q, k, v, tables, lens in runs[:3]:
        pick = slice(0, 4)
        want, tol = int4.attention(q[pick], k, v, tables[pick], lens[pick], 0.1)
        _close(out[pick], want, tol)


def test_a_call_runs_on_the_current_stream():
    # the query arrives on a side stream behind a long copy; a launch elsewhere would miss it
    k, v, tables, lens, q = _case([300, 47], seed=41)
    rng = np.random.default_rng(1)
    x = _rows(rng, (2, 2))
    a = [_dev(t) for t in (k, v, tables, lens, x, _new_slots(tables, lens, 1, 16))]
    src, qd = _dev(q), torch.zeros(q.shape, dtype=torch.float16, device=DEV)
    big = torch.zeros(1 << 28, dtype=torch.float32, device=DEV)
    out, ws = torch.empty_like(qd), pkv.make_workspace(2, 1, 12, 2)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(8):
            big.add_(1)
        qd.copy_(src)
        rows = a[4] + 0
        pkv.kv_append_int4(rows, rows, a[5], a[0], a[1])
        pkv.paged_attn_decode_int4(out, qd, *a[:4], 0.1, ws)
    torch.cuda.synchronize()
    int4.append(x, x, _new_slots(tables, lens, 1, 16), k, v)
    want, tol = int4.attention(q, k, v, tables, lens, 0.1)
    _close(out, want, tol)


# ----------------------------------------------------------------------------- refusals
def test_binding_refuses_what_the_library_cannot_see():
    k = torch.zeros(4, 2, 16, 80, dtype=torch.uint8, device=DEV)
    q = torch.zeros(2, 1, 12, 128, dtype=torch.float16, device=DEV)
    bt = torch.zeros(2, 2, dtype=torch.int32, device=DEV)
    cl = torch.ones(2, dtype=torch.int32, device=DEV)
    ws = pkv.make_workspace(2, 1, 12, 2)
    rows = torch.zeros(2, 2, 128, dtype=torch.float16, device=DEV)
    slots = torch.zeros(2, dtype=torch.int64, device=DEV)

    def dec(**kw):
        a = dict(out=q.clone(), q=q, k_cache=k, v_cache=k, block_tables=bt, context_lens=cl,
                 scale=0.1, workspace=ws)
        a.update(kw)
        return lambda: pkv.paged_attn_decode_int4(**a)

    wide = torch.zeros(2, 2, 12, 128, dtype=torch.float16, device=DEV)[:, :1]
    bad = [
        dec(q=q.float()), dec(q=q.cpu()), dec(q=wide), dec(out=q[:1]), dec(context_lens=cl.long()),
        dec(block_tables=bt[:1]), dec(k_cache=k[..., :64]), dec(v_cache=k[:2]),
        dec(workspace=ws[:100]), dec(context_lens=cl[:1]),
        lambda: pkv.kv_append_int4(rows, rows, slots[:1], k, k),
        lambda: pkv.kv_append_int4(rows.float(), rows, slots, k, k),
        lambda: pkv.kv_append_int4(rows, rows, slots.int(), k, k),
        lambda: pkv.kv_append_int4(rows, rows, slots, k.float(), k),
        lambda: pkv.widen_blocks_int4(k, k, cl, cl[:1], rows, rows),
        lambda: pkv.paged_attn_decode_append_int4(q.clone(), q, rows[:1], rows[:1], k, k, bt, cl,
                                                  0.1, ws),
    ]
    for call in bad:
        with pytest.raises(pkv.PkvError) as e:
            call()
        assert e.value.status in (pkv.EINVAL, pkv.ENOSPC)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
