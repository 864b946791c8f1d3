"""Cases for a decode step over an 8-bit paged KV cache with a scale per block and head, dense and
over selected blocks: the operators' plain forms in elementary torch operations, and the library's
calls for the same work.

Operators (what each call computes, on the GPU):

* append   rows of K and V are quantised to 8 bits and scattered to their slots; a block's scale
           grows with its rows, and what it already held is brought to the new scale, or, where
           its first row is written, set to zero (``kv_append_int8``); then the blocks are read
           back as fp16 blocks, as a chunked prefill over the cache needs them
           (``widen_blocks_int8``);
* decode   a few query tokens per sequence attend over the 8-bit cache
           (``paged_attn_decode_int8``);
* select   for each sequence and kv head the blocks that may hold the largest scores
           (``select_blocks``);
* sparse   a step's run of them: the new tokens' rows are appended, blocks are selected, and the
           queries attend over the selected blocks only.

The format: a block of `bs` tokens of one kv head holds uint8 codes u [bs, 128] of K and of V; an
element's value is s * (u - 128), with s the block's and head's scale, kv_scales[block, head, 0]
for K and [.., 1] for V, a power of two. k_bounds[block, head] holds the smallest and the greatest
key code of each channel among the rows written into the block.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head size
DEV = "cuda"
LOWEST, HIGHEST = -30, 9      # exponents of a scale
MOST = 127                    # largest code (without the offset)


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt chunk of 512 tokens for each of 16 sequences of the 70B shape goes into the
        # cache and comes back as fp16 blocks for the chunk's attention
        dict(name="append_70b_chunk", kind="append", seqs=16, lo=512, hi=512, hkv=8, bs=16),
        # one decode step's rows of the 1.1B edge shape, into partly filled blocks
        dict(name="append_edge_step", kind="append", seqs=64, lo=1, hi=1, hkv=2, bs=16),
        # the smallest call: one sequence early in its answer, where latency counts
        dict(name="decode_one", kind="decode", seqs=1, lo=101, hi=101, hq=12, hkv=2, q_len=1, bs=16),
        # one layer of the 70B shape, batch 16 at 4096 tokens
        dict(name="decode_70b_b16", kind="decode", seqs=16, lo=4096, hi=4096, hq=64, hkv=8, q_len=1,
             bs=16),
        # one layer of the 70B shape's mixed batch
        dict(name="decode_70b_mixed", kind="decode", seqs=32, lo=50, hi=8000, hq=64, hkv=8, q_len=1,
             bs=16),
        # long documents: 32 sequences at 16384 tokens in 64-token blocks
        dict(name="decode_70b_long", kind="decode", seqs=32, lo=16384, hi=16384, hq=64, hkv=8,
             q_len=1, bs=64),
        # four drafts per sequence of the edge shape, ragged lengths
        dict(name="decode_edge_drafts", kind="decode", seqs=64, lo=16, hi=2048, hq=12, hkv=2,
             q_len=4, bs=16),
        # the edge shape's ragged lengths, at most 16 blocks of 16 tokens each
        dict(name="select_edge", kind="select", seqs=64, lo=16, hi=2048, hq=12, hkv=2, q_len=1,
             bs=16, budget=16, first=1, last=1),
        # 128 of 1024 blocks of long documents of the 70B shape
        dict(name="select_70b_long", kind="select", seqs=32, lo=16384, hi=16384, hq=64, hkv=8,
             q_len=1, bs=16, budget=128, first=1, last=2),
        # one step over one very long document: 64 of 2048 blocks
        dict(name="sparse_one", kind="sparse", seqs=1, lo=131072, hi=131072, hq=64, hkv=8, q_len=1,
             bs=64, budget=64, first=1, last=2),
        # one step over long documents of mixed lengths, two drafts each: 64 blocks of 64 tokens
        dict(name="sparse_70b_long", kind="sparse", seqs=16, lo=32768, hi=65536, hq=64, hkv=8,
             q_len=2, bs=64, budget=64, first=1, last=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "select", "sparse", "sparse"])
    hkv, group = rng.choice([(1, 1), (1, 7), (2, 6), (4, 2), (8, 8), (8, 4), (32, 1), (5, 3)])
    bs = rng.choice([16, 32, 64, 128, 256])
    if kind == "append":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(2, 65536 // (seqs * hkv)))
        return dict(kind=kind, seqs=seqs, lo=rng.randint(0, hi), hi=hi, hkv=hkv, bs=bs)
    seqs, q_len = _log_int(rng, 1, 64), rng.randint(1, 4)
    case = dict(kind=kind, seqs=seqs, hq=hkv * group, hkv=hkv, q_len=q_len, bs=bs)
    if kind == "decode":
        most = 4000000 // (seqs * hkv * max(1, q_len * group // 8))
        hi = _log_int(rng, 4, min(65536, max(5, most)))
        return dict(case, lo=rng.randint(min(4, hi), hi), hi=hi)
    first, last = rng.randint(0, 3), rng.randint(0, 3)
    ends = first + max(last, 1 + -(-(q_len - 1) // bs))
    budget = ends + _log_int(rng, 1, max(2, 4096 // bs))
    hi = _log_int(rng, 16, min(131072, max(17, 8000000 // (seqs * hkv))))
    return dict(case, lo=rng.randint(min(4, hi), hi), hi=hi, budget=budget, first=first, last=last)


def _lens(case, rng):
    return rng.integers(case["lo"], case["hi"], size=case["seqs"], endpoint=True).astype(np.int64)


def _rng(case, seed):
    return np.random.default_rng([seed, case["seqs"], case["hi"], case["bs"]])


def _blocks(lens, bs):
    return (lens + bs - 1) // bs


def _make_tables(rng, lens, bs, most=None):
    """Blocks of one shuffled pool for each sequence: (num_blocks, tables). `most`: the pool's size
    where it is not to depend on the lengths."""
    need = _blocks(lens, bs)
    total = int(need.sum())
    num_blocks = total + 2 if most is None else most
    perm = rng.permutation(num_blocks).astype(np.int32)
    tables = np.full((len(lens), max(1, int(need.max()))), -1, np.int32)
    tables[np.arange(tables.shape[1])[None, :] < need[:, None]] = perm[:total]
    return num_blocks, tables


def _gpu(a):
    return torch.as_tensor(np.ascontiguousarray(a)).to(DEV)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _keys(g, rows, hkv):
    """fp16 keys as a model leaves them: a few channels of each head much larger than the rest."""
    x = torch.randn(rows, hkv, D, generator=g, device=DEV)
    gain = torch.where(torch.rand(hkv, D, generator=g, device=DEV) < 0.04, 4.0, 1.0)
    return (x * gain).half()


def _values(g, rows, hkv):
    return torch.randn(rows, hkv, D, generator=g, device=DEV).half()


def _filled_cache(g, nb, hkv, bs):
    """A cache whose every block holds quantised rows, of a size that differs from block to block:
    K and V codes, scales, bounds."""
    scales = torch.empty(nb, hkv, 2, device=DEV)
    bounds = torch.empty(nb, hkv, 2, D, dtype=torch.uint8, device=DEV)
    pools = []
    for i, make in enumerate((_keys, _values)):
        pool = torch.empty(nb, hkv, bs, D, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 18) // (hkv * bs))
        for at in range(0, nb, step):
            n = min(step, nb - at)
            gain = torch.exp2(0.7 * torch.randn(n, 1, hkv, 1, generator=g, device=DEV))
            rows = (make(g, n * bs, hkv).view(n, bs, hkv, D) * gain).half().transpose(1, 2)
            s = _scale_of(rows.abs().amax((2, 3)))
            pool[at:at + n] = _codes(rows, s[..., None, None])
            scales[at:at + n, :, i] = s
        pools.append(pool)
        if i == 0:
            bounds[:, :, 0], bounds[:, :, 1] = pool.amin(2), pool.amax(2)
    return pools[0], pools[1], scales, bounds


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    kind = case["kind"]
    rng, g = _rng(case, seed), _gen(seed)
    lens, bs, hkv = _lens(case, rng), case["bs"], case["hkv"]
    if kind == "append":
        return _prepare_append(rng, g, lens, case)
    q_len = case["q_len"]
    nb, tables = _make_tables(rng, lens, bs)
    k_pool, v_pool, scales, bounds = _filled_cache(g, nb, hkv, bs)
    s = dict(kind=kind, bs=bs, k_pool=k_pool, v_pool=v_pool, scales=scales, bounds=bounds,
             tables=_gpu(tables), lens=_gpu(lens.astype(np.int32)), scale=1.0 / math.sqrt(D),
             q=(1.5 * torch.randn(len(lens), q_len, case["hq"], D, generator=g, device=DEV)).half(),
             out=torch.empty(len(lens), q_len, case["hq"], D, dtype=torch.float16, device=DEV))
    if kind in ("select", "sparse"):
        s.update(budget=case["budget"], first=case["first"], last=case["last"])
    if kind == "sparse":
        pos = lens[:, None] - q_len + np.arange(q_len)
        row = np.take_along_axis(tables.astype(np.int64), np.maximum(pos, 0) // bs, 1)
        s.update(k=_keys(g, len(lens) * q_len, hkv), v=_values(g, len(lens) * q_len, hkv),
                 slots=_gpu((row * bs + pos % bs).reshape(-1)))
    if own and kind in ("decode", "sparse"):
        from paged_kv_cache_147_gb300 import pkv
        s["workspace"] = pkv.make_workspace(len(lens), q_len, case["hq"], hkv, DEV)
    return s


def _prepare_append(rng, g, new, case):
    """New rows for sequences that hold up to two blocks of tokens already."""
    bs, hkv = case["bs"], case["hkv"]
    new = np.maximum(new, (np.arange(len(new)) == 0).astype(np.int64))
    held = rng.integers(0, 2 * bs, size=len(new))
    most = len(new) * -(-(case["hi"] + 2 * bs - 1) // bs) + 2
    nb, tables = _make_tables(rng, held + new, bs, most)
    k_pool, v_pool, scales, bounds = _filled_cache(g, nb, hkv, bs)
    pos = np.concatenate([h + np.arange(n) for h, n in zip(held, new)])
    seq = np.repeat(np.arange(len(new)), new)
    # the blocks that the new rows go to
    src = np.unique(tables[seq, pos // bs])
    s = dict(kind="append", bs=bs, k_pool=k_pool, v_pool=v_pool, scales=scales, bounds=bounds,
             k=_keys(g, len(pos), hkv), v=_values(g, len(pos), hkv),
             slots=_gpu(tables[seq, pos // bs].astype(np.int64) * bs + pos % bs),
             src=_gpu(src.astype(np.int32)), dst=_gpu(np.arange(len(src), dtype=np.int32)))
    for x in ("k_wide", "v_wide"):
        s[x] = torch.zeros(nb, hkv, bs, D, dtype=torch.float16, device=DEV)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _scale_of(top):
    """The least power of two s, of those allowed, with top <= 127 s."""
    m, e = torch.frexp(top.float())
    e = e - 7 + (m > MOST / 128).int()
    e = torch.where(top == 0, torch.full_like(e, LOWEST), e).clamp(LOWEST, HIGHEST)
    return torch.ldexp(torch.ones_like(m), e)


def _codes(x, s):
    return (torch.round(x.float() / s).clamp(-MOST, MOST) + 128).to(torch.uint8)


def _rescaled(u, factor):
    return (torch.round((u.float() - 128) * factor) + 128).to(torch.uint8)


def _plain_write(s):
    """The append: every block that rows go to is written anew, one whose first row is among them
    with zeros behind them, any other with what it held on the grid of its new scale."""
    bs, slots = s["bs"], s["slots"]
    touched, at = torch.unique(slots // bs, return_inverse=True)
    off = slots % bs
    t, n, hkv = len(touched), len(slots), s["k"].shape[1]
    fresh = torch.zeros(t, dtype=torch.bool, device=DEV)
    fresh[at[off == 0]] = True
    for i, x in enumerate(("k", "v")):
        rows, pool = s[x], s[x + "_pool"]
        top = torch.zeros(t, hkv, device=DEV).scatter_reduce(
            0, at[:, None].expand(n, hkv), rows.abs().amax(-1).float(), "amax")
        old = s["scales"][touched, :, i]
        new = torch.where(fresh[:, None], _scale_of(top), torch.maximum(_scale_of(top), old))
        factor = old / new
        block = _rescaled(pool[touched], factor[..., None, None])
        block = torch.where(fresh[:, None, None, None], torch.full_like(block, 128), block)
        codes = _codes(rows, new[at][..., None])
        block[at, :, off] = codes
        if i == 0:
            lo, hi = (_rescaled(s["bounds"][touched, :, j], factor[..., None]) for j in (0, 1))
            lo = torch.where(fresh[:, None, None], torch.full_like(lo, 255), lo)
            hi = torch.where(fresh[:, None, None], torch.zeros_like(hi), hi)
            to = at[:, None, None].expand(n, hkv, D)
            s["bounds"][touched, :, 0] = lo.scatter_reduce(0, to, codes, "amin")
            s["bounds"][touched, :, 1] = hi.scatter_reduce(0, to, codes, "amax")
        pool[touched] = block
        s["scales"][touched, :, i] = new


def _plain_append(s):
    _plain_write(s)
    src, dst = s["src"].long(), s["dst"].long()
    for i, x in enumerate(("k", "v")):
        value = (s[x + "_pool"][src].float() - 128) * s["scales"][src, :, i][..., None, None]
        s[x + "_wide"][dst] = value.half()
    return [s["k_wide"], s["v_wide"], s["scales"]]


def _plain_select(s):
    tables, lens, q, bs = s["tables"].long(), s["lens"].long(), s["q"], s["bs"]
    b, q_len, hq, _ = q.shape
    hkv, width = s["bounds"].shape[1], tables.shape[1]
    group, ids = hq // hkv, tables.clamp(min=0)
    qg = q.view(b, q_len, hkv, group, D).transpose(1, 2)
    e = _scale_of(qg.abs().amax(-1))                                   # [b, hkv, q_len, group]
    p = (_codes(qg, e[..., None]).float() - 128).flatten(2, 3)
    bound = (s["bounds"][ids].float() - 128).permute(3, 0, 2, 4, 1)    # [2, b, hkv, 128, width]
    # whole numbers below 2^24 times powers of two: exact in fp32 in any order
    dot = torch.matmul(p.clamp(max=0), bound[0]) + torch.matmul(p.clamp(min=0), bound[1])
    score = dot * e.flatten(2, 3)[..., None] * s["scales"][ids, :, 0].transpose(1, 2)[:, :, None]
    sees = lens[:, None] - q_len + torch.arange(q_len, device=DEV) >= 0
    sees = sees[:, None, :, None].expand(b, 1, q_len, group).flatten(2, 3)[..., None]
    score = torch.where(sees, score, torch.full_like(score, -math.inf)).amax(2)   # [b, hkv, width]
    col = torch.arange(width, device=DEV)
    count = _blocks(lens, bs)[:, None]
    tail = torch.maximum(torch.full_like(count, s["last"]),
                         count - ((lens - q_len).clamp(min=0) // bs)[:, None])
    kept = (col < s["first"]) | (col >= count - tail)
    score = torch.where(kept[:, None], torch.full_like(score, math.inf), score)
    score = torch.where((col < count)[:, None], score, torch.full_like(score, -math.inf))
    # the best first, equal ones by their place; blocks that are not there last
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :s["budget"]]
    taken = torch.minimum(count, torch.full_like(count, s["budget"]))             # [b, 1]
    slot = torch.arange(order.shape[-1], device=DEV)
    order = torch.where((slot < taken)[:, None], order, torch.full_like(order, width))
    order = torch.sort(order, dim=-1).values
    found = torch.gather(tables[:, None].expand(b, hkv, width), 2, order.clamp(max=width - 1))
    found = torch.where((slot < taken)[:, None], found, torch.full_like(found, -1))
    out = torch.full((b, hkv, s["budget"]), -1, dtype=torch.int32, device=DEV)
    out[..., :order.shape[-1]] = found.int()
    return out, (lens - (count - taken)[:, 0] * bs).int()


def _plain_attention(s, tables, lens):
    """tables [b, heads, width], a table per kv head or (heads = 1) one for all."""
    q, bs, hkv = s["q"], s["bs"], s["k_pool"].shape[1]
    b, q_len, hq, _ = q.shape
    length = tables.shape[2] * bs
    ids = tables.long().clamp(min=0).expand(b, hkv, tables.shape[2])
    head = torch.arange(hkv, device=DEV)[:, None]

    def gathered(i, pool):   # [b, hkv, length, 128]
        value = pool[ids, head].float() - 128
        return (value * s["scales"][ids, head, i][..., None, None]).flatten(2, 3)

    limit = lens.long()[:, None] - q_len + torch.arange(q_len, device=DEV) + 1
    seen = torch.arange(length, device=DEV) < limit[:, :, None]        # [b, q_len, length]
    seen = seen[:, None, :, None, :]
    qg = q.float().view(b, q_len, hkv, hq // hkv, D).transpose(1, 2)   # [b, hkv, q_len, group, 128]
    score = torch.matmul(qg.flatten(2, 3), gathered(0, s["k_pool"]).transpose(-1, -2))
    score = score.view(b, hkv, q_len, hq // hkv, length) * s["scale"]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    values = gathered(1, s["v_pool"])
    out = torch.matmul(p.flatten(2, 3), values).view(b, hkv, q_len, hq // hkv, D)
    s["out"].copy_(out.transpose(1, 2).reshape(b, q_len, hq, D))
    return s["out"]


def _plain_sparse(s):
    _plain_write(s)
    tables, lens = _plain_select(s)
    return [_plain_attention(s, tables, lens), tables, lens]


# ------------------------------------------------------------------------------------ one pass
def run(s):
    kind = s["kind"]
    if not own:
        return dict(append=_plain_append, sparse=_plain_sparse,
                    decode=lambda s: _plain_attention(s, s["tables"][:, None], s["lens"]),
                    select=lambda s: list(_plain_select(s)))[kind](s)
    from paged_kv_cache_147_gb300 import pkv
    if kind == "append":
        pkv.kv_append_int8(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["scales"],
                           s["bounds"])
        pkv.widen_blocks_int8(s["k_pool"], s["v_pool"], s["scales"], s["src"], s["dst"],
                              s["k_wide"], s["v_wide"])
        return [s["k_wide"], s["v_wide"], s["scales"]]
    if kind == "decode":
        return pkv.paged_attn_decode_int8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["scales"],
                                          s["tables"], s["lens"], s["scale"], s["workspace"])
    if kind == "sparse":
        pkv.kv_append_int8(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"], s["scales"],
                           s["bounds"])
    tables, lens = pkv.select_blocks(s["q"], s["scales"], s["bounds"], s["tables"], s["lens"],
                                     s["bs"], s["budget"], s["first"], s["last"])
    if kind == "select":
        return [tables, lens]
    out = pkv.paged_attn_decode_int8(s["out"], s["q"], s["k_pool"], s["v_pool"], s["scales"],
                                     tables, lens, s["scale"], s["workspace"])
    return [out, tables, lens]


def work(case):
    """Bytes that have to move once, and the products' operations; ragged lengths by their mean."""
    kind, n, bs, hkv = case["kind"], case["seqs"], case["bs"], case["hkv"]
    mean = (case["lo"] + case["hi"]) / 2
    if kind == "append":
        blocks = math.ceil(n * mean / bs)
        moved = n * mean * (hkv * 2 * (2 * D + D) + 8)         # fp16 rows in, codes out, slots
        moved += blocks * hkv * (8 + 2 * D)                    # scales and bounds
        return dict(bytes=moved + blocks * hkv * bs * 2 * (D + 2 * D), flops=0)   # and widened
    q_rows = n * case["q_len"] * case["hq"]
    queries = q_rows * D * 2
    if kind == "decode":
        blocks = n * math.ceil(mean / bs)
        return dict(bytes=n * mean * hkv * 2 * D + blocks * (4 + 8 * hkv) + 2 * queries,
                    flops=4 * D * q_rows * mean)
    # bounds and the keys' scale of every block; the tables that come out
    blocks = math.ceil(mean / bs)
    taken = min(blocks, case["budget"])
    moved = n * blocks * (4 + hkv * (2 * D + 4)) + n * hkv * case["budget"] * 4 + queries
    flops = 4 * D * q_rows * blocks
    if kind == "sparse":
        seen = min(mean, taken * bs)
        moved += n * hkv * (seen * 2 * D + taken * 8) + queries
        moved += n * case["q_len"] * hkv * 2 * 3 * D
        flops += 4 * D * q_rows * seen
    return dict(bytes=moved, flops=flops)


# ------------------------------------------------------------------------------------ 64 bits
def _exact_scale(top):
    """Least power of two s with top <= 127 s (numpy)."""
    s = 2.0 ** LOWEST
    s = np.full(top.shape, s)
    for _ in range(HIGHEST - LOWEST):
        s = np.where(top > MOST * s, 2 * s, s)
    return s


def _exact_append(s):
    """What the cache holds after the append, for the blocks that rows went to: {block: (K values,
    V values [hkv, bs, 128], their scales [hkv])}, in 64 bits."""
    bs, slots = s["bs"], s["slots"].cpu().numpy()
    scales = s["scales"].cpu().numpy().astype(np.float64)
    got = {}
    rows = [s[x].cpu().numpy().astype(np.float64) for x in ("k", "v")]
    pools = [s[x + "_pool"] for x in ("k", "v")]
    order = np.argsort(slots, kind="stable")
    cuts = np.nonzero(np.diff(slots[order] // bs))[0] + 1
    groups = np.split(order, cuts)
    held = torch.as_tensor([int(slots[at[0]] // bs) for at in groups], device=DEV)
    held = [p[held].cpu().numpy().astype(np.float64) - 128 for p in pools]
    for j, at in enumerate(groups):
        block, off = int(slots[at[0]] // bs), slots[at] % bs
        entry = []
        for i in (0, 1):
            new = np.swapaxes(rows[i][at], 0, 1)                        # [hkv, rows, 128]
            want = _exact_scale(np.abs(new).max((1, 2)))
            if off.min() > 0:
                want = np.maximum(want, scales[block, :, i])
            w = want[:, None, None]
            # as they stand before the call, and then on the new grid
            codes = np.rint(held[i][j] * scales[block, :, i][:, None, None] / w) * (off.min() > 0)
            codes[:, off] = np.clip(np.rint(new / w), -MOST, MOST)
            entry += [codes * w, want]
        got[block] = (entry[0], entry[2], entry[1], entry[3])
    return got


def exact(case, seed):
    kind = case["kind"]
    if kind == "select":       # whole numbers only
        return None
    s = prepare(case, seed)
    if kind == "append":
        got = _exact_append(s)
        wide = [np.zeros(tuple(s["k_wide"].shape)) for _ in range(2)]
        scales = s["scales"].cpu().numpy().astype(np.float64)
        for i, block in enumerate(s["src"].cpu().tolist()):
            for j in (0, 1):
                wide[j][i] = got[block][j]
                scales[block, :, j] = got[block][2 + j]
        return [torch.as_tensor(x) for x in (*wide, scales)]
    if kind == "decode":
        return _exact_attention(s, case, {}, None)
    got = _exact_append(s)
    return [_exact_attention(s, case, got, case["budget"]), None, None]


def _exact_choice(s, case, b, n, blocks, k_of, budget):
    """Logical blocks that each kv head of sequence b attends to, [hkv, taken], by the definition:
    the bound of a block is the greatest product any of its codes' extremes allow."""
    bs, q_len, hkv = case["bs"], case["q_len"], case["hkv"]
    count = len(blocks)
    taken = min(count, budget)
    if taken == count:
        return np.tile(np.arange(count), (hkv, 1))
    lo, hi, scale = k_of                                               # [count, hkv, 128], [count, hkv]
    rows = s["q"][b].double().cpu().numpy()                            # [q_len, hq, 128]
    tail = max(case["last"], count - max(n - q_len, 0) // bs)
    out = []
    for h in range(hkv):
        group = case["hq"] // hkv
        best = np.full(count, -np.inf)
        for i in range(q_len):
            if n - q_len + i < 0:
                continue
            for r in range(h * group, (h + 1) * group):
                step = _exact_scale(np.abs(rows[i, r]).max())
                p = np.clip(np.rint(rows[i, r] / step), -MOST, MOST)
                bound = np.maximum(p * lo[:, h], p * hi[:, h]).sum(-1) * scale[:, h] * step
                best = np.maximum(best, bound)
        best[:case["first"]] = np.inf
        best[count - tail:] = np.inf
        out.append(np.sort(np.lexsort((np.arange(count), -best))[:taken]))
    return np.stack(out)


def _exact_attention(s, case, got, budget):
    """Textbook attention, one sequence after the other, in 64 bits; `got`: blocks as an append
    left them."""
    bs, q_len, hkv = case["bs"], case["q_len"], case["hkv"]
    q, lens = s["q"].double(), s["lens"].cpu().tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    group = case["hq"] // hkv
    for b, n in enumerate(lens):
        blocks = s["tables"][b, :-(-n // bs)].long()
        where = blocks.cpu().tolist()
        if budget is None:
            pick = np.tile(np.arange(len(where)), (hkv, 1))
        else:
            k_of = [x.cpu().numpy().astype(np.float64)
                    for x in (s["bounds"][blocks, :, 0], s["bounds"][blocks, :, 1],
                              s["scales"][blocks, :, 0])]
            for j, block in enumerate(where):
                if block in got:
                    _exact_bounds(s, got[block], block, j, k_of)
            k_of[0] -= 128
            k_of[1] -= 128
            pick = _exact_choice(s, case, b, n, where, k_of, budget)
        m = n - (len(where) - pick.shape[1]) * bs                      # tokens attended over
        for h in range(hkv):
            ids = blocks[torch.as_tensor(pick[h], device=q.device)]
            kv = []
            for i, x in enumerate(("k", "v")):
                value = (s[x + "_pool"][ids, h].double() - 128) * s["scales"][ids, h, i].double()[:, None, None]
                for j, block in enumerate(ids.cpu().tolist()):
                    if block in got:
                        value[j] = torch.as_tensor(got[block][i][h]).to(q.device)
                kv.append(value.flatten(0, 1)[:m])
            at = slice(h * group, (h + 1) * group)
            for i in range(q_len):
                e = m - q_len + i + 1
                if e > 0:
                    w = torch.softmax(kv[0][:e] @ q[b, i, at].T * s["scale"], 0)
                    out[b, i, at] = w.T @ kv[1][:e]
    return out


def _exact_bounds(s, entry, block, j, k_of):
    """Bounds of a block that rows were appended to: those it had, on its new grid, and the rows'."""
    bs = s["bs"]
    slots = s["slots"].cpu().numpy()
    at = np.nonzero(slots // bs == block)[0]
    off = slots[at] % bs
    codes = np.rint(entry[0][:, off] / entry[2][:, None, None]) + 128   # [hkv, rows, 128]
    lo, hi = codes.min(1), codes.max(1)
    if off.min() > 0:
        factor = (k_of[2][j] / entry[2])[:, None]
        lo = np.minimum(lo, np.rint((k_of[0][j] - 128) * factor) + 128)
        hi = np.maximum(hi, np.rint((k_of[1][j] - 128) * factor) + 128)
    k_of[0][j], k_of[1][j], k_of[2][j] = lo, hi, entry[2]
