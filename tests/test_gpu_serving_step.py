"""The operators of a serving step over a 4-bit cache, as they are used together: prompts are
admitted (tables on the device, norm + rotation, append, prefill over widened blocks), then
decode steps with drafts, some of which are taken back."""
import numpy as np
import pytest
import torch

import oracle
from oracle import int4, step
from paged_kv_cache_147_gb300 import pkv

from _util import f16_host

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def test_prompts_then_drafts_with_rollback():
    rng = np.random.default_rng(42)
    B, hq, hkv, bs, nb, width, q_len = 5, 12, 2, 16, 90, 16, 3
    scale, eps = 128 ** -0.5, 1e-6
    table = pkv.rope_table(512)
    table_h, table_d = table.numpy(), table.to(DEV)
    w = (1 + 0.2 * rng.standard_normal((2, 128))).astype(np.float16)
    wd = [_dev(x) for x in w]
    tables, lens = np.full((B, width), -1, np.int32), np.zeros(B, np.int32)
    free, count = rng.permutation(nb).astype(np.int32), nb
    d = [_dev(x) for x in (tables, lens, free, np.array([count], np.int32))]
    kd, vd = (torch.full((nb, hkv, bs, 80), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    kp, vp = kd.cpu().numpy().copy(), vd.cpu().numpy().copy()

    def layer(new, max_tokens):
        """One step's tables, projections, norm and rotation on the GPU; tables by the oracle."""
        nonlocal tables, lens, count
        slots, seqs, pos, cu = pkv.extend_tables(d[0], d[1], _dev(new), bs, d[2], d[3], max_tokens)
        tables, lens, count, s, q_, p, c, refused = step.extend(tables, lens, new, bs, free, count,
                                                                max_tokens)
        assert not refused and np.array_equal(slots.cpu().numpy(), s)
        x = rng.standard_normal((max_tokens, (hq + 2 * hkv) * 128)).astype(np.float16)
        xd = _dev(x)
        q, k = pkv.qk_norm_rope(xd[:, :hq * 128].view(-1, hq, 128),
                                xd[:, hq * 128:-hkv * 128].view(-1, hkv, 128), *wd, eps, pos, table_d)
        v = xd[:, -hkv * 128:].view(-1, hkv, 128).contiguous()
        real = p >= 0
        for got, lo, hi, ww in ((q, 0, hq, w[0]), (k, hq, hq + hkv, w[1])):
            want, tol = step.norm_rope(x[real, lo * 128:hi * 128].reshape(-1, hi - lo, 128), ww, eps,
                                       p[real], table_h)
            assert (np.abs(got.cpu().numpy()[real].astype(np.float64) - want) <= tol).all()
        return q, k, v, slots, s

    # ---- prompts of the same chunk length (the prefill's), padded token arrays ----
    chunk = 37
    q, k, v, slots, s = layer(np.full(B, chunk, np.int32), B * chunk + 4)
    pkv.kv_append_int4(k, v, slots, kd, vd)
    int4.append(f16_host(k), f16_host(v), s, kp, vp)
    assert np.array_equal(kd.cpu().numpy(), kp) and np.array_equal(vd.cpu().numpy(), vp)
    used = tables[tables >= 0]
    wide = [torch.zeros(nb, hkv, bs, 128, dtype=torch.float16, device=DEV) for _ in range(2)]
    pkv.widen_blocks_int4(kd, vd, _dev(used), _dev(used), *wide)
    qp = q[:B * chunk].view(B, chunk, hq, 128)
    out = torch.empty_like(qp)
    pkv.paged_prefill(out, qp, *wide, d[0], d[1], scale)
    ref = oracle.paged_attention(f16_host(qp), f16_host(wide[0]), f16_host(wide[1]), tables, lens,
                                 bs, scale)
    assert np.abs(out.float().cpu().numpy() - ref).max() <= 2e-3     # the prefill's own bar

    # ---- decode steps: three drafts each, some rejected ----
    ws = pkv.make_workspace(B, q_len, hq, hkv)
    for i in range(8):
        q, k, v, slots, s = layer(np.full(B, q_len, np.int32), B * q_len)
        out = torch.empty(B, q_len, hq, 128, dtype=torch.float16, device=DEV)
        qd = q.view(B, q_len, hq, 128)
        if i % 2:
            pkv.kv_append_int4(k, v, slots, kd, vd)
            pkv.paged_attn_decode_int4(out, qd, kd, vd, d[0], d[1], scale, ws)
        else:
            pkv.paged_attn_decode_append_int4(out, qd, k, v, kd, vd, d[0], d[1], scale, ws)
        int4.append(f16_host(k), f16_host(v), s, kp, vp)
        assert np.array_equal(kd.cpu().numpy(), kp) and np.array_equal(vd.cpu().numpy(), vp)
        want, tol = int4.attention(f16_host(qd), kp, vp, tables, lens, scale)
        assert (np.abs(out.float().cpu().numpy() - want) <= tol).all()
        keep = (lens - rng.integers(0, q_len, B)).astype(np.int32)
        pkv.truncate_tables(d[0], d[1], _dev(keep), bs, d[2], d[3])
        tables, lens, free, count = step.truncate(tables, lens, keep, bs, free, count)
        for got, want in zip(d, (tables, lens, free, np.array([count]))):
            assert np.array_equal(got.cpu().numpy(), want)

    # ---- one sequence ends; its blocks serve the others ----
    keep = np.full(B, -1, np.int32)
    keep[2] = 0
    pkv.truncate_tables(d[0], d[1], _dev(keep), bs, d[2], d[3])
    tables, lens, free, count = step.truncate(tables, lens, keep, bs, free, count)
    assert d[3].item() == count and d[1][2].item() == 0
    assert pkv.device_error(clear=True) == 0


@pytest.mark.parametrize("B,fused", [(3, False), (40, False), (40, True)])
def test_steps_in_a_row_without_a_pause(B, fused):
    # every call reads what the one before it wrote, with no synchronisation and no other kernel in
    # between (their launches overlap); issued one by one and as a captured graph
    rng = np.random.default_rng(B)
    hq, hkv, bs, width, q_len, steps = 12, 2, 16, 30, 3, 5
    scale, eps = 128 ** -0.5, 1e-6
    lens = rng.integers(0, 300, B).astype(np.int32)
    need = -(-lens // bs)
    nb = int(need.sum()) + 3 * B
    perm = rng.permutation(nb).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    tables[np.arange(width)[None] < need[:, None]] = perm[:need.sum()]
    free = np.concatenate([perm[need.sum():], perm[:need.sum()]])
    count = nb - int(need.sum())
    k0, v0 = (int4.quantise(rng.standard_normal((nb, hkv, bs, 128)).astype(np.float16)) for _ in range(2))
    table = pkv.rope_table(1024).to(DEV)
    w = [_dev((1 + 0.2 * rng.standard_normal(128)).astype(np.float16)) for _ in range(2)]
    qs, ks, vs = (_dev(rng.standard_normal((steps, B * q_len, h, 128)).astype(np.float16))
                  for h in (hq, hkv, hkv))
    new = np.full(B, q_len, np.int32)
    newd, keeps = _dev(new), []
    t, l, f, c, sim = tables, lens, free, count, []
    for i in range(steps):          # what the tables must be, and how much each step takes back
        t, l, c, s, _, _, _, refused = step.extend(t, l, new, bs, f, c, B * q_len)
        assert not refused
        sim.append((t, l, s))
        keeps.append((l - rng.integers(0, q_len, B)).astype(np.int32))
        t, l, f, c = step.truncate(t, l, keeps[-1], bs, f, c)
    keepd = [_dev(x) for x in keeps]
    start = [_dev(x) for x in (tables, lens, free, np.array([count], np.int32), k0, v0)]
    d = [x.clone() for x in start]
    ws = pkv.make_workspace(B, q_len, hq, hkv)
    outs = [torch.empty(B, q_len, hq, 128, dtype=torch.float16, device=DEV) for _ in range(steps)]
    q_out, k_out = torch.empty_like(qs), torch.empty_like(ks)
    maps = pkv.extend_tables(d[0].clone(), d[1].clone(), 0 * newd, bs, d[2].clone(), d[3].clone(),
                             B * q_len)

    def run():
        for i in range(steps):
            pkv.extend_tables(d[0], d[1], newd, bs, d[2], d[3], B * q_len, out=maps)
            pkv.qk_norm_rope(qs[i], ks[i], *w, eps, maps[2], table, q_out[i], k_out[i])
            args = (d[4], d[5], d[0], d[1], scale, ws)
            q = q_out[i].view(B, q_len, hq, 128)
            if fused:
                pkv.paged_attn_decode_append_int4(outs[i], q, k_out[i], vs[i], *args)
            else:
                pkv.kv_append_int4(k_out[i], vs[i], maps[0], d[4], d[5])
                pkv.paged_attn_decode_int4(outs[i], q, *args)
            pkv.truncate_tables(d[0], d[1], keepd[i], bs, d[2], d[3])

    run()
    torch.cuda.synchronize()
    kp, vp = k0.copy(), v0.copy()
    for i, (t_i, l_i, s_i) in enumerate(sim):
        int4.append(f16_host(k_out[i]), f16_host(vs[i]), s_i, kp, vp)
        want, tol = int4.attention(f16_host(q_out[i].view(B, q_len, hq, 128)), kp, vp, t_i, l_i, scale)
        assert (np.abs(outs[i].float().cpu().numpy() - want) <= tol).all(), i
    first = [o.clone() for o in outs] + [x.clone() for x in d]
    for got, want in zip(d, (t, l, f, np.array([c]), kp, vp)):
        assert np.array_equal(got.cpu().numpy(), want)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        run()
    for again in (run, graph.replay, run, graph.replay):
        for x, y in zip(d, start):
            x.copy_(y)
        for o in outs:
            o.fill_(float("nan"))
        again()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs + d, first))
    assert pkv.device_error(clear=True) == 0


@pytest.mark.parametrize("fused", [True, False])
def test_refused_and_idle_sequences_keep_their_cached_rows(fused):
    # five sequences, no free block: the second needs one and is refused, the fourth is idle. Their
    # cached rows stay whichever way the step takes, though the norm left their keys as they were
    rng = np.random.default_rng(8)
    B, q_len, hq, hkv, bs, width = 5, 2, 12, 2, 16, 6
    scale, eps = 128 ** -0.5, 1e-6
    lens = np.array([20, 31, 46, 9, 33], np.int32)
    new = np.array([2, 2, 2, 0, 2], np.int32)
    need = -(-lens // bs)
    nb = int(need.sum())
    tables = np.full((B, width), -1, np.int32)
    tables[np.arange(width)[None] < need[:, None]] = rng.permutation(nb)
    free = np.zeros(nb, np.int32)
    k0, v0 = (int4.quantise(rng.standard_normal((nb, hkv, bs, 128)).astype(np.float16)) for _ in range(2))
    td, ld, kd, vd, news = (_dev(x) for x in (tables, lens, k0, v0, new))
    T = B * q_len
    slots, seqs, pos, cu = pkv.extend_tables(td, ld, news, bs, _dev(free), _dev(np.zeros(1, np.int32)), T)
    assert pkv.device_error(clear=True) == pkv.DEVERR_SPACE
    wt, wl, _, ws, _, _, _, refused = step.extend(tables, lens, new, bs, free, 0, T)
    assert refused == [1] and np.array_equal(slots.cpu().numpy(), ws)
    x = [_dev(rng.standard_normal((T, h, 128)).astype(np.float16)) for h in (hq, hkv, hkv)]
    w = [_dev((1 + 0.2 * rng.standard_normal(128)).astype(np.float16)) for _ in range(2)]
    q, k = (torch.full_like(t, float("nan")) for t in x[:2])
    pkv.qk_norm_rope(*x[:2], *w, eps, pos, pkv.rope_table(64).to(DEV), q, k)
    # the packed tokens of each sequence (those of one without new tokens are somebody else's)
    rows = (cu[:-1, None] + torch.arange(q_len, device=DEV)).clamp(max=T - 1)
    qb = q[rows]
    out = torch.full_like(qb, float("nan"))
    space = pkv.make_workspace(B, q_len, hq, hkv)
    if fused:
        served = (seqs[rows[:, 0]] == torch.arange(B, device=DEV)) & (news == q_len)
        step_lens = torch.where(served, ld, 0)
        kb, vb = (t[rows].view(T, hkv, 128) for t in (k, x[2]))
        pkv.paged_attn_decode_append_int4(out, qb, kb, vb, kd, vd, td, step_lens, scale, space)
    else:
        pkv.kv_append_int4(k, x[2], slots, kd, vd)
        pkv.paged_attn_decode_int4(out, qb, kd, vd, td, ld, scale, space)
    torch.cuda.synchronize()
    assert pkv.device_error(clear=True) == 0
    int4.append(f16_host(k), f16_host(x[2]), ws, k0, v0)
    assert np.array_equal(kd.cpu().numpy(), k0) and np.array_equal(vd.cpu().numpy(), v0)
    some = [0, 2, 4]
    want, tol = int4.attention(f16_host(qb)[some], k0, v0, wt[some], wl[some], scale)
    assert (np.abs(out[some].float().cpu().numpy() - want) <= tol).all()
    if fused:
        assert (out[[1, 3]] == 0).all()
