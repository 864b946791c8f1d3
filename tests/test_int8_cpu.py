"""CPU pins of the 8-bit cache's oracle, and the host refusals of its entry points (their argument
checks run before any CUDA call)."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import int8
from paged_kv_cache_147_gb300 import build, pkv


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load()


# ------------------------------------------------------------------------------- the format
@pytest.mark.parametrize("top,want", [(0, 2.0 ** -30), (2.0 ** -24, 2.0 ** -30), (127, 1), (127.0625, 2),
                                      (128, 2), (254, 2), (0.9921875, 2.0 ** -7), (1, 2.0 ** -6),
                                      (65024, 512), (65504, 512)])
def test_scale_of_a_largest_element(top, want):
    assert int8.scale_of(np.array([top, -top / 2])) == want
    assert want == 512 or top <= 127 * want
    assert want == 2.0 ** -30 or top > 127 * want / 2


def test_values_are_off_by_half_a_step_and_repeated_moves_by_less_than_one():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((16, 1, 128)) * 2.0 ** np.arange(-4, 12)[:, None, None]).astype(np.float16)
    pools = [np.zeros((1, 1, 16, 128), np.uint8) for _ in range(2)]
    scales = np.zeros((1, 1, 2), np.float32)
    for t in range(16):        # every token doubles the largest element
        int8.append(x[t:t + 1], x[t:t + 1], [t], *pools, scales)
    got = int8.values(pools[0], scales[..., 0])[0, 0]
    assert (np.abs(got - x[:, 0].astype(np.float64)) < scales[0, 0, 0]).all()
    int8.append(x, x, np.arange(16), *pools, scales)
    got = int8.values(pools[0], scales[..., 0])[0, 0]
    assert (np.abs(got - x[:, 0].astype(np.float64)) <= scales[0, 0, 0] / 2).all()


def test_bounds_hold_every_key_of_a_block_and_bound_its_scores():
    rng = np.random.default_rng(1)
    hkv, bs, T = 2, 16, 75
    pools = [np.zeros((6, hkv, bs, 128), np.uint8) for _ in range(2)]
    scales, bounds = np.zeros((6, hkv, 2), np.float32), np.zeros((6, hkv, 2, 128), np.uint8)
    at = 0
    while at < T:
        n = min(int(rng.integers(1, 20)), T - at)
        k = (rng.standard_normal((n, hkv, 128)) * (1 + at)).astype(np.float16)
        int8.append(k, k, at + np.arange(n), *pools, scales, bounds)
        at += n
    q = rng.standard_normal((3, 128))
    for h in range(hkv):
        score = int8.bound_scores(q, bounds[:5, h], scales[:5, h, 0].astype(np.float64))
        for j in range(5):
            rows = pools[0][j, h, :min(bs, T - j * bs)]
            assert (rows >= bounds[j, h, 0]).all() and (rows <= bounds[j, h, 1]).all()
            p = np.stack([np.rint(r / int8.scale_of(r)) * int8.scale_of(r) for r in q])
            assert (p @ int8.values(rows, scales[j, h, 0]).T).max() <= score[j]


def test_oracle_attention_over_all_blocks_is_plain_softmax():
    rng = np.random.default_rng(2)
    k, v = (rng.integers(1, 256, (3, 1, 16, 128)).astype(np.uint8) for _ in range(2))
    scales = np.full((3, 1, 2), 2.0 ** -6, np.float32)
    q = rng.standard_normal((1, 2, 2, 128)).astype(np.float16)
    tables, lens = np.array([[2, 0, 1]], np.int32), [37]
    out, tol = int8.attention(q, k, v, scales, tables, lens, 0.1)
    K, V = ((x[[2, 0, 1]].reshape(-1, 128).astype(float) - 128) / 64 for x in (k, v))
    for i in range(2):
        x = torch.as_tensor(q[0, i].astype(np.float64) @ K[:36 + i].T * 0.1)
        assert np.allclose(out[0, i], torch.softmax(x, -1).numpy() @ V[:36 + i])
    assert (tol > 0).all()
    per_head = int8.attention(q, k, v, scales, tables[:, None], lens, 0.1)[0]
    assert np.array_equal(per_head, out)


def test_oracle_selection_keeps_the_ends_and_the_best():
    bounds = np.full((10, 1, 2, 128), 128, np.uint8)
    bounds[[4, 7], 0, 1, 0] = [200, 190]                # keys that reach far in channel 0
    bounds[5, 0, 0, 1] = 60                             # and one in the negative of channel 1
    q = np.zeros((1, 1, 1, 128), np.float16)
    q[0, 0, 0, :2] = [1, -1]
    scales = np.ones((1, 10, 1, 2), np.float32)[0]
    tables = np.arange(10, dtype=np.int32)[None, ::-1].copy()
    got, lens = int8.select(q, scales, bounds, tables, [155], 16, 4, 1, 1)
    assert list(got[0, 0]) == [9, 5, 4, 0] and lens[0] == 155 - 6 * 16
    scales[2, 0, 0] = math.nan
    got, _ = int8.select(q, scales, bounds, tables, [155], 16, 4, 1, 1)
    assert list(got[0, 0]) == [9, 4, 2, 0]


# ------------------------------------------------------------------------------- refusals
P = ctypes.c_void_p(256)    # a well-aligned address that no refused call may touch
ODD = ctypes.c_void_p(264)


def test_append_widen_and_copy_refuse_bad_arguments(lib):
    def app(k=P, v=P, s=P, T=4, kc=P, vc=P, sc=P, kb=P, nb=8, h=2, d=128, bs=16):
        return lib.pkv_kv_append_int8(k, v, s, T, kc, vc, sc, kb, nb, h, d, bs, None)

    assert app(T=0, k=None, s=None, kc=None, sc=None, kb=None) == pkv.OK
    for bad in (dict(T=-1), dict(h=0), dict(d=64), dict(bs=24), dict(nb=-1), dict(k=None), dict(v=ODD),
                dict(s=None), dict(kc=ODD), dict(vc=None), dict(sc=None), dict(sc=ctypes.c_void_p(4)),
                dict(kb=ODD), dict(T=0x7fffffff, h=1 << 20)):
        assert app(**bad) == pkv.EINVAL, bad

    def wid(k=P, v=P, sc=P, s=P, t=P, n=3, nb=8, ko=P, vo=P, nbo=8, h=2, d=128, bs=16):
        return lib.pkv_widen_blocks_int8(k, v, sc, s, t, n, nb, ko, vo, nbo, h, d, bs, None)

    assert wid(n=0, k=None, ko=None) == pkv.OK
    for bad in (dict(n=-1), dict(nb=-1), dict(nbo=-1), dict(h=0), dict(d=80), dict(bs=48), dict(sc=None),
                dict(ko=ODD), dict(vo=None), dict(s=None), dict(n=0x7fffffff, h=128, bs=256)):
        assert wid(**bad) == pkv.EINVAL, bad

    def cpy(k=P, v=P, sc=P, kb=P, s=P, t=P, n=3, L=2, nb=8, h=2, d=128, bs=16):
        return lib.pkv_copy_blocks_int8(k, v, sc, kb, s, t, n, L, nb, h, d, bs, None)

    assert cpy(n=0, k=None) == pkv.OK and cpy(L=0, k=None) == pkv.OK
    for bad in (dict(n=-1), dict(L=-1), dict(nb=-1), dict(h=0), dict(d=64), dict(bs=8), dict(k=None),
                dict(sc=None), dict(kb=ODD), dict(t=None), dict(n=1 << 20, L=1 << 20)):
        assert cpy(**bad) == pkv.EINVAL, bad


@pytest.mark.parametrize("name", ["pkv_paged_attn_decode_int8", "pkv_selected_attn_decode_int8"])
def test_decode_refuses_bad_arguments(lib, name):
    def dec(out=P, q=P, k=P, v=P, sc=P, nb=8, bt=P, mb=4, cl=P, B=2, q_len=1, hq=12, hkv=2, d=128,
            bs=16, ws=P, n=1 << 30):
        return getattr(lib, name)(out, q, k, v, sc, nb, bt, mb, cl, B, q_len, hq, hkv, d, bs, 0.1,
                                  ws, n, None)

    assert dec(B=0) == pkv.OK
    for bad in (dict(d=64), dict(bs=20), dict(hq=13), dict(q_len=0), dict(hkv=0, hq=0), dict(q_len=6),
                dict(hq=66), dict(B=-1), dict(B=5000), dict(nb=0), dict(out=None), dict(sc=None),
                dict(sc=ctypes.c_void_p(4)), dict(q=ctypes.c_void_p(8)), dict(cl=None), dict(ws=None),
                dict(ws=ctypes.c_void_p(128)), dict(mb=1 << 28), dict(nb=1 << 28),
                dict(hq=(1 << 20) + 1, hkv=(1 << 20) + 1, nb=1, mb=1, B=1)):
        assert dec(**bad) == pkv.EINVAL, bad
    assert dec(B=0, hq=33, hkv=1) == pkv.EINVAL


def test_selection_refuses_bad_arguments(lib):
    def sel(t=P, l=P, q=P, sc=P, kb=P, nb=8, bt=P, mb=64, cl=P, B=2, q_len=1, hq=12, hkv=2, d=128, bs=16,
            budget=8, first=1, last=1):
        return lib.pkv_select_blocks(t, l, q, sc, kb, nb, bt, mb, cl, B, q_len, hq, hkv, d, bs, budget,
                                     first, last, None)

    assert sel(B=0, t=None, q=None) == pkv.OK
    for bad in (dict(t=None), dict(l=None), dict(q=None), dict(q=ODD), dict(sc=None), dict(kb=ODD),
                dict(kb=None), dict(bt=None), dict(cl=None), dict(B=-1), dict(q_len=0), dict(q_len=6),
                dict(hq=13), dict(hq=0), dict(hkv=0), dict(d=64), dict(bs=100), dict(nb=0),
                dict(mb=-1), dict(mb=262145), dict(budget=0), dict(first=-1), dict(last=-1),
                dict(first=7, last=2), dict(budget=1),
                dict(first=7, q_len=2), dict(B=1 << 28)):
        assert sel(**bad) == pkv.EINVAL, bad


# ------------------------------------------------------------------------- launches that wait
@pytest.mark.parametrize("source", ["pkv_cache_int8.cu", "pkv_decode_int8.cu", "pkv_select.cu"])
def test_kernels_that_start_early_read_through_plain_loads(source):
    # their CTAs are resident while the kernel before them still writes what they will read
    with open(os.path.join(build.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert "griddep_wait()" in code
    assert not re.findall(r"__ldg\b|__restrict__|__restrict\b|ld\.global\.nc", code)


# ----------------------------------------------------------------------------- the binding
def test_compiled_binding_refuses_what_is_not_on_a_gpu():
    ops = pkv._torch_ops()
    with pytest.raises(TypeError):
        ops.select_blocks(1, 2)
    cache = pkv.make_int8_cache(4, 2, 16, device="cpu")
    assert cache[0].shape == (4, 2, 16, 128) and cache[2].shape == (4, 2, 2)
    assert pkv.make_int8_cache(4, 2, 16, layers=3, bounds=False, device="cpu")[3] is None
    rows, slots = torch.zeros(2, 2, 128, dtype=torch.float16), torch.zeros(2, dtype=torch.int64)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(RuntimeError):      # PkvError, or no CUDA device
        pkv.kv_append_int8(rows, rows, slots, *cache)
    with pytest.raises(RuntimeError):
        pkv.copy_blocks_int8(*cache, table[0], table[0])
    with pytest.raises(RuntimeError):
        pkv.select_blocks(rows[:, None], cache[2], cache[3], table, table[:, 0], 16, 2)
    with pytest.raises(RuntimeError):
        pkv.paged_attn_decode_int8(rows, rows, *cache[:3], table, table[:, 0], 1.0, slots)
