"""CPU pins of the 4-bit oracle and the step oracle, and the host refusals of the entry points
around the 4-bit cache (their argument checks run before any CUDA call)."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from oracle import int4, step
from paged_kv_cache_147_gb300 import build, pkv


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pkv.load()


# ------------------------------------------------------------------------------- the 4-bit row
def test_rows_of_exact_values_come_back_exactly():
    # 16 equally spaced values per group, spacing a power of two: s, z and every code are exact
    x = (np.arange(128) % 16).astype(np.float16) * np.float16(0.25) - np.float16(2)
    rows = int4.quantise(x[None])
    assert rows.shape == (1, 80)
    assert np.array_equal(int4.values(rows)[0], x.astype(np.float64))
    assert rows[0, 0] == 0x10 and rows[0, 7] == 0xFE           # element 2 j is the low half
    assert np.array_equal(rows[0, 64:68].view(np.float16), np.float16([0.25, -2]))


@pytest.mark.parametrize("gain", [2.0 ** -20, 1e-3, 1.0, 300.0])
def test_rows_are_off_by_half_a_step_at_most(gain):
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((50, 128)) * gain).astype(np.float16)
    rows = int4.quantise(x)
    _, s, _ = int4.parts(rows)
    assert (np.abs(int4.values(rows) - x.astype(np.float64)) <= s / 2).all()


def test_rows_at_the_edges_of_fp16():
    x = np.zeros((6, 128), np.float16)
    x[0, :2] = [65504, -65504]             # the largest range: 15 s + z must stay finite
    x[1, 5] = 2.0 ** -24                   # one smallest subnormal
    x[2, 40] = np.inf
    x[3, 40] = np.nan
    x[4, :] = 3.5                          # constant: s = 0
    x[5, 40:44] = [-np.inf, 1, 2, 3]
    rows = int4.quantise(x)
    val = int4.values(rows)
    assert (np.abs(val[0]) <= 65504).all()
    code, s, z = int4.parts(rows)
    assert abs(val[0, 0] - 65504) <= s[0, 0] / 50 and val[0, 1] == -65504
    assert (val[4] == 3.5).all() and (s[4] == 0).all() and (code[4] == 0).all()
    for r in (2, 3, 5):                    # the group of 32 with the bad element, no other
        assert np.isnan(val[r, 32:64]).all() and np.isfinite(val[r, :32]).all()
        assert np.isfinite(val[r, 64:]).all()
    assert np.abs(val[1] - x[1].astype(np.float64)).max() <= 2.0 ** -25


def test_oracle_attention_is_textbook_attention_on_contiguous_values():
    rng = np.random.default_rng(5)
    n, bs = 21, 16
    k = int4.quantise(rng.standard_normal((3, 2, bs, 128)).astype(np.float16))
    v = int4.quantise(rng.standard_normal((3, 2, bs, 128)).astype(np.float16))
    q = rng.standard_normal((1, 1, 4, 128)).astype(np.float16)
    out, tol = int4.attention(q, k, v, np.array([[2, 0]]), [n], 0.1)
    for h in range(4):
        K = np.concatenate([int4.values(k[2, h // 2]), int4.values(k[0, h // 2])])[:n]
        V = np.concatenate([int4.values(v[2, h // 2]), int4.values(v[0, h // 2])])[:n]
        w = np.exp(K @ q[0, 0, h].astype(np.float64) * 0.1)
        assert np.allclose(out[0, 0, h], (w / w.sum()) @ V, atol=1e-12)
    assert (tol > 0).all() and tol.max() < 0.02


# ------------------------------------------------------------------------------- the tables
def test_oracle_extend_then_truncate_restores_everything():
    rng = np.random.default_rng(1)
    bs, B = 16, 9
    lens = rng.integers(0, 60, B).astype(np.int32)
    perm = rng.permutation(80).astype(np.int32)
    tables = np.full((B, 10), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-int(n) // bs)
        tables[b, :k] = perm[at:at + k]
        at += k
    free = np.zeros(80, np.int32)
    free[:80 - at] = perm[at:]
    new = rng.integers(0, 50, B).astype(np.int32)
    t2, l2, c2, slots, seqs, pos, cu, refused = step.extend(tables, lens, new, bs, free, 80 - at,
                                                           int(new.sum()) + 3)
    assert not refused and (slots[:cu[-1]] >= 0).all() and (slots[cu[-1]:] == -1).all()
    assert len(set(slots[:cu[-1]])) == cu[-1]
    t3, l3, f3, c3 = step.truncate(t2, l2, lens, bs, free, c2)
    assert np.array_equal(t3, tables) and np.array_equal(l3, lens) and c3 == 80 - at
    assert np.array_equal(f3, free)


# ------------------------------------------------------------------------------- refusals
P = ctypes.c_void_p(256)    # a well-aligned address that no refused call may touch


def test_append_and_widen_refuse_bad_arguments(lib):
    app = lib.pkv_kv_append_int4
    assert app(None, None, None, 0, None, None, 8, 2, 128, 16, None) == pkv.OK
    assert app(None, None, None, 4, None, None, 8, 2, 128, 16, None) == pkv.EINVAL
    assert app(P, P, P, 4, P, P, 8, 2, 64, 16, None) == pkv.EINVAL          # head size
    assert app(P, P, P, 4, P, P, 8, 2, 128, 24, None) == pkv.EINVAL         # block size
    assert app(P, P, P, -1, P, P, 8, 2, 128, 16, None) == pkv.EINVAL
    assert app(P, P, P, 4, P, P, 8, 0, 128, 16, None) == pkv.EINVAL
    assert app(ctypes.c_void_p(264), P, P, 4, P, P, 8, 2, 128, 16, None) == pkv.EINVAL
    wid = lib.pkv_widen_blocks_int4
    assert wid(None, None, None, None, 0, 8, None, None, 8, 2, 128, 16, None) == pkv.OK
    assert wid(P, P, P, P, 3, 8, P, None, 8, 2, 128, 16, None) == pkv.EINVAL
    assert wid(P, P, P, P, -3, 8, P, P, 8, 2, 128, 16, None) == pkv.EINVAL
    assert wid(P, P, P, P, 3, 8, ctypes.c_void_p(8), P, 8, 2, 128, 16, None) == pkv.EINVAL
    assert wid(P, P, P, P, 3, 8, P, P, 8, 2, 128, 48, None) == pkv.EINVAL
    # more CTAs than a grid holds
    assert wid(P, P, P, P, 0x7fffffff, 8, P, P, 8, 128, 128, 256, None) == pkv.EINVAL


def test_decode_refuses_bad_arguments(lib):
    def dec(out=P, q=P, k=P, v=P, nb=8, bt=P, mb=4, cl=P, B=2, q_len=1, hq=12, hkv=2, d=128, bs=16,
            ws=P, n=1 << 30):
        return lib.pkv_paged_attn_decode_int4(out, q, k, v, nb, bt, mb, cl, B, q_len, hq, hkv, d,
                                              bs, 0.1, ws, n, None)

    assert dec(B=0) == pkv.OK
    for bad in (dict(d=64), dict(bs=20), dict(hq=13), dict(q_len=0), dict(hkv=0, hq=0),
                dict(q_len=6), dict(hq=66), dict(B=-1), dict(B=5000), dict(nb=0), dict(out=None),
                dict(q=ctypes.c_void_p(8)), dict(cl=None), dict(ws=None),
                dict(ws=ctypes.c_void_p(128)), dict(mb=1 << 28), dict(nb=1 << 28)):
        assert dec(**bad) == pkv.EINVAL, bad
    # R = 33 is refused for an empty batch too
    assert dec(B=0, hq=33, hkv=1) == pkv.EINVAL
    app = lib.pkv_paged_attn_decode_append_int4
    assert app(P, P, None, P, P, P, 8, P, 4, P, 2, 1, 12, 2, 128, 16, 0.1, P, 1 << 30,
               None) == pkv.EINVAL
    assert app(P, P, P, ctypes.c_void_p(8), P, P, 8, P, 4, P, 2, 1, 12, 2, 128, 16, 0.1, P, 1 << 30,
               None) == pkv.EINVAL


def test_decode_refuses_more_heads_than_it_can_count(lib):
    # a call within every other limit: one block, one sequence
    for hkv in ((1 << 20) + 1, 1 << 23, 1 << 26):
        for fn, new in ((lib.pkv_paged_attn_decode_int4, ()), (lib.pkv_paged_attn_decode_append_int4, (P, P))):
            assert fn(P, P, *new, P, P, 1, P, 1, P, 1, 1, hkv, hkv, 128, 16, 0.1, P, 1 << 40,
                      None) == pkv.EINVAL


def test_norm_rope_refuses_bad_arguments(lib):
    def norm(qo=P, ko=P, q=P, k=P, qs=1536, ks=256, eps=1e-6, n=16, T=3, hq=12, hkv=2, d=128, pos=P):
        return lib.pkv_qk_norm_rope(qo, ko, q, k, qs, ks, P, P, eps, pos, P, n, T, hq, hkv, d, None)

    assert norm(T=0) == pkv.OK
    for bad in (dict(d=64), dict(qs=1535), dict(qs=1538), dict(ks=128), dict(eps=-1.0),
                dict(eps=float("nan")), dict(n=0), dict(T=-1), dict(hq=0), dict(hkv=0),
                dict(q=None), dict(pos=None), dict(k=ctypes.c_void_p(4))):
        assert norm(**bad) == pkv.EINVAL, bad


def test_tables_refuse_bad_arguments(lib):
    def ext(t=P, l=P, m=P, B=4, mb=8, bs=16, f=P, c=P, nb=64, s=P, q=P, p=P, cu=P, T=10):
        return lib.pkv_extend_tables(t, l, m, B, mb, bs, f, c, nb, s, q, p, cu, T, None)

    assert ext(B=0, T=0) == pkv.OK
    for bad in (dict(B=-1), dict(B=4097), dict(bs=17), dict(mb=-1), dict(nb=-1), dict(T=-1),
                dict(t=None), dict(f=None), dict(c=None), dict(s=None), dict(cu=None),
                dict(mb=1 << 28, bs=16)):
        assert ext(**bad) == pkv.EINVAL, bad
    cut = lib.pkv_truncate_tables
    assert cut(P, P, P, 0, 8, 16, P, P, 64, None) == pkv.OK
    assert cut(P, P, None, 3, 8, 16, P, P, 64, None) == pkv.EINVAL
    assert cut(P, P, P, 4097, 8, 16, P, P, 64, None) == pkv.EINVAL
    assert cut(P, P, P, 3, 8, 15, P, P, 64, None) == pkv.EINVAL


# ------------------------------------------------------------------------- launches that wait
@pytest.mark.parametrize("source", ["pkv_cache_int4.cu", "pkv_decode_int4.cu", "pkv_norm_rope.cu",
                                    "pkv_tables.cu"])
def test_kernels_that_start_early_read_through_plain_loads(source):
    # their CTAs are resident while the kernel before them still writes what they will read:
    # no load there may be declared read-only (__ldg, const __restrict__)
    with open(os.path.join(build.CSRC, source)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    assert "griddep_wait()" in code
    assert not re.findall(r"__ldg\b|__restrict__|__restrict\b|ld\.global\.nc", code)


# ----------------------------------------------------------------------------- the binding
def test_compiled_binding_loads_and_refuses_what_is_not_on_a_gpu():
    ops = pkv._torch_ops()
    with pytest.raises(TypeError):
        ops.kv_append_int4(1, 2)
    rows, slots = torch.zeros(2, 2, 128, dtype=torch.float16), torch.zeros(2, dtype=torch.int64)
    pool = torch.zeros(2, 2, 16, 80, dtype=torch.uint8)
    with pytest.raises(RuntimeError):      # PkvError, or no CUDA device
        pkv.kv_append_int4(rows, rows, slots, pool, pool)
    with pytest.raises(RuntimeError):
        pkv.truncate_tables(None, None, None, 16, None, None)
    table = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(RuntimeError):
        pkv.extend_tables(table, table[0], table[0], 16, table[0], table[0, :1], 4)
