"""Cases for the operators of a serving step over a 4-bit paged KV cache: their plain forms in
elementary torch operations, and the library's calls for the same work.

Operators (what each call computes, on the GPU):

* append   rows of K and V are quantised to 4 bits and scattered to their slots
           (``kv_append_int4``), then the blocks they went to are widened to fp16 blocks, as a
           chunked prefill over the cache needs them (``widen_blocks_int4``);
* decode   a few query tokens per sequence attend over the 4-bit cache
           (``paged_attn_decode_int4``);
* fused    the same with this step's rows appended in the same call
           (``paged_attn_decode_append_int4``), and the blocks it wrote widened;
* tables   rejected tokens are cut off each sequence's block table (``truncate_tables``), then
           the tables grow for the step's new tokens and the slots, sequences and positions of
           those tokens are written (``extend_tables``);
* norm     per-head RMS norm of queries and keys and the rotation by position
           (``qk_norm_rope``).

The 4-bit format: a row (one token, one kv head, K or V) of 128 elements is 80 bytes. Bytes
0-63 hold the codes, element 2j in the low half of byte j and 2j + 1 in the high half; bytes
64 + 4g .. 67 + 4g hold the scale s and the minimum z of elements 32g .. 32g + 31, two fp16.
An element's value is s * code + z.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head size
GROUP = 32       # elements that share a scale and a minimum
ROW = 80         # bytes of a 4-bit row
DEV = "cuda"
F16_MAX = 65504.0


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt chunk of 512 tokens for each of 16 sequences of the 70B shape goes into the
        # cache and comes back as fp16 blocks for the chunk's attention
        dict(name="append_70b_chunk", kind="append", seqs=16, lo=512, hi=512, hkv=8, bs=16),
        # one decode step's rows of the 1.1B edge shape
        dict(name="append_edge_step", kind="append", seqs=64, lo=1, hi=1, hkv=2, bs=16),
        # the smallest call: one sequence early in its answer, where latency counts
        dict(name="decode_one", kind="decode", seqs=1, lo=101, hi=101, hq=12, hkv=2, q_len=1, bs=16),
        # one layer of the 70B shape, batch 16 at 4096 tokens
        dict(name="decode_70b_b16", kind="decode", seqs=16, lo=4096, hi=4096, hq=64, hkv=8, q_len=1,
             bs=16),
        # long documents: 32 sequences at 16384 tokens in 64-token blocks
        dict(name="decode_70b_long", kind="decode", seqs=32, lo=16384, hi=16384, hq=64, hkv=8,
             q_len=1, bs=64),
        # four drafts per sequence of the edge shape, ragged lengths
        dict(name="decode_edge_drafts", kind="decode", seqs=64, lo=16, hi=2048, hq=12, hkv=2,
             q_len=4, bs=16),
        # one layer of the edge model's decode step, append included, ragged lengths
        dict(name="fused_edge", kind="fused", seqs=64, lo=16, hi=2048, hq=12, hkv=2, q_len=1, bs=16),
        # one layer of the 70B shape's mixed batch, append included
        dict(name="fused_70b_mixed", kind="fused", seqs=32, lo=50, hi=8000, hq=64, hkv=8, q_len=1,
             bs=16),
        # a speculative step's bookkeeping: two of four drafts cut off, four more to come
        dict(name="tables_drafts", kind="tables", seqs=64, lo=16, hi=2048, new=4, cut=2, bs=16),
        # prompts of up to 4096 tokens admitted for 256 sequences
        dict(name="tables_prompts", kind="tables", seqs=256, lo=0, hi=63, new=4096, cut=0, bs=16),
        # one decode step of the edge shape
        dict(name="norm_edge_step", kind="norm", tokens=64, hq=12, hkv=2, pad=0),
        # a prompt chunk of the 70B shape, read from packed projections
        dict(name="norm_70b_chunk", kind="norm", tokens=8192, hq=64, hkv=8, pad=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "decode", "decode", "fused", "tables", "norm"])
    hkv, group = rng.choice([(1, 1), (1, 7), (2, 6), (4, 2), (8, 8), (8, 4), (32, 1), (5, 3)])
    bs = rng.choice([16, 32, 64, 128, 256])
    if kind == "append":
        seqs = _log_int(rng, 1, 64)
        hi = _log_int(rng, 1, max(2, 65536 // (seqs * hkv)))
        return dict(kind=kind, seqs=seqs, lo=rng.randint(0, hi), hi=hi, hkv=hkv, bs=bs)
    if kind in ("decode", "fused"):
        seqs, q_len = _log_int(rng, 1, 64), rng.randint(1, 4)
        most = 4000000 // (seqs * hkv * max(1, q_len * group // 8))
        hi = _log_int(rng, 4, min(65536, max(5, most)))
        return dict(kind=kind, seqs=seqs, lo=rng.randint(min(4, hi), hi), hi=hi, hq=hkv * group,
                    hkv=hkv, q_len=q_len, bs=bs)
    if kind == "tables":
        seqs = _log_int(rng, 1, 512)
        hi = _log_int(rng, 1, 8192)
        return dict(kind=kind, seqs=seqs, lo=rng.randint(0, hi), hi=hi,
                    new=_log_int(rng, 1, min(4096, 600000 // seqs)), cut=rng.randint(0, 40), bs=bs)
    return dict(kind=kind, tokens=_log_int(rng, 1, 65536 // max(8, hkv * group)), hq=hkv * group,
                hkv=hkv, pad=rng.randint(0, 1))


def _lens(case, rng):
    return rng.integers(case["lo"], case["hi"], size=case["seqs"], endpoint=True).astype(np.int64)


def _rng(case, seed):
    return np.random.default_rng([seed, case["seqs"], case["hi"], case["bs"]])


def _blocks(lens, bs):
    return (lens + bs - 1) // bs


def _make_tables(rng, lens, bs, spare=2):
    """Blocks of one shuffled pool for each sequence: (num_blocks, tables, unused blocks)."""
    need = _blocks(lens, bs)
    total = int(need.sum())
    perm = rng.permutation(total + spare).astype(np.int32)
    width = max(1, int(need.max()))
    tables = np.full((len(lens), width), -1, np.int32)
    tables[np.arange(width)[None, :] < need[:, None]] = perm[:total]
    return total + spare, tables, perm[total:]


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


def _filled_pools(g, nb, hkv, bs):
    """4-bit pools whose every row holds quantised data."""
    pools = []
    for make in (_keys, _values):
        pool = torch.empty(nb, hkv, bs, ROW, dtype=torch.uint8, device=DEV)
        step = max(1, (1 << 17) // (hkv * bs))
        for i in range(0, nb, step):
            n = min(step, nb - i)
            rows = make(g, n * bs, hkv).view(n, bs, hkv, D).transpose(1, 2)
            pool[i:i + n] = _quantise(rows)
        pools.append(pool)
    return pools


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    kind = case["kind"]
    if kind == "norm":
        return _prepare_norm(case, seed)
    if kind == "tables":
        return _prepare_tables(case, seed)
    rng, g = _rng(case, seed), _gen(seed)
    lens, bs, hkv = _lens(case, rng), case["bs"], case["hkv"]
    s = dict(kind=kind, bs=bs)
    if kind == "append":
        lens = np.maximum(lens, (np.arange(len(lens)) == 0).astype(np.int64))
        nb, tables, _ = _make_tables(rng, lens, bs)
        pos = np.concatenate([np.arange(n) for n in lens])
        seq = np.repeat(np.arange(len(lens)), lens)
        used = tables[tables >= 0]
        s.update(k=_keys(g, len(pos), hkv), v=_values(g, len(pos), hkv),
                 slots=_gpu(tables[seq, pos // bs].astype(np.int64) * bs + pos % bs),
                 src=_gpu(used), dst=_gpu(np.arange(len(used), dtype=np.int32)))
        for x in ("k", "v"):
            s[x + "_pool"] = torch.zeros(nb, hkv, bs, ROW, dtype=torch.uint8, device=DEV)
            s[x + "_wide"] = torch.zeros(len(lens) * -(-case["hi"] // bs), hkv, bs, D,
                                         dtype=torch.float16, device=DEV)
        return s
    q_len = case["q_len"]
    nb, tables, _ = _make_tables(rng, lens, bs)
    s["k_pool"], s["v_pool"] = _filled_pools(g, nb, hkv, bs)
    s.update(q=torch.randn(len(lens), q_len, case["hq"], D, generator=g, device=DEV).half(),
             tables=_gpu(tables), lens=_gpu(lens.astype(np.int32)), scale=1.0 / math.sqrt(D),
             out=torch.empty(len(lens), q_len, case["hq"], D, dtype=torch.float16, device=DEV))
    if kind == "fused":
        s.update(k=_keys(g, len(lens) * q_len, hkv), v=_values(g, len(lens) * q_len, hkv))
        # the blocks that hold the first and the last new row of each sequence
        at = np.stack([np.maximum(lens - q_len, 0), lens - 1], 1)
        src = tables[np.arange(len(lens))[:, None], at // bs].reshape(-1)
        s.update(src=_gpu(src), dst=_gpu(np.arange(len(src), dtype=np.int32)))
        for x in ("k", "v"):
            s[x + "_wide"] = torch.zeros(len(src), hkv, bs, D, dtype=torch.float16, device=DEV)
    if own:
        from paged_kv_cache_147_gb300 import pkv
        s["workspace"] = pkv.make_workspace(len(lens), q_len, case["hq"], hkv, DEV)
    return s


def _prepare_tables(case, seed):
    """Tables that hold the drafts of the step before (up to `cut` of them to be taken back), a
    stack of free blocks, and the numbers of new tokens. A pass ends with the new tokens in the
    tables; the next one cuts those off again, which restores the stack, so that every pass
    after it finds the same blocks."""
    rng = _rng(case, seed)
    bs, n = case["bs"], case["seqs"]
    lens = _lens(case, rng)
    keep = np.maximum(lens - rng.integers(0, case["cut"], size=n, endpoint=True), 0)
    new = rng.integers(1, case["new"], size=n, endpoint=True)
    new[n - n // 2:] = case["new"] + 1 - new[:n // 2]      # as many in all whatever the seed
    new[n // 2:n - n // 2] = (case["new"] + 1) // 2
    held = _blocks(lens, bs)
    width = -(-(case["hi"] + case["new"]) // bs)
    total = n * width + 8
    perm = rng.permutation(total).astype(np.int32)
    tables = np.full((n, width), -1, np.int32)
    tables[np.arange(width)[None, :] < held[:, None]] = perm[:held.sum()]
    free = np.zeros(total, np.int32)
    free[:total - held.sum()] = perm[held.sum():]
    return dict(kind="tables", bs=bs, tables=_gpu(tables), lens=_gpu(lens.astype(np.int32)),
                keep=_gpu(keep.astype(np.int32)), new=_gpu(new.astype(np.int32)), free=_gpu(free),
                count=_gpu(np.array([total - held.sum()], np.int32)), tokens=int(new.sum()) + 5)


def _prepare_norm(case, seed):
    g = _gen(seed)
    t, hq, hkv = case["tokens"], case["hq"], case["hkv"]
    # queries, keys and values of a token side by side, as one projection leaves them
    width = (hq + 2 * hkv) * D if case["pad"] else (hq + hkv) * D
    x = (torch.randn(t, width, generator=g, device=DEV) * 3.0).half()
    q, k = x[:, :hq * D], x[:, hq * D:(hq + hkv) * D]
    if not case["pad"]:
        q, k = q.contiguous(), k.contiguous()
    index = 8192
    inv = 10000.0 ** (-2.0 * np.arange(D // 2) / D)
    ang = np.arange(index)[:, None] * inv
    table = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    return dict(kind="norm", q=q.view(t, hq, D), k=k.view(t, hkv, D), eps=1e-6,
                q_weight=(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).half(),
                k_weight=(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).half(),
                positions=torch.randint(0, index, (t,), generator=g, device=DEV),
                table=_gpu(table))


# ------------------------------------------------------------------------------------ plain forms
def _quantise(x):
    """fp16 rows [..., 128] -> 4-bit rows [..., 80] bytes. For each 32 elements z = min and
    s = (max - min) / 15 rounded up to fp16 (down where 15 s + z would pass the largest fp16);
    code = round((x - z) / s), ties to even, kept within 0 .. 15. In 64 bits: the codes of
    values on a border go by the last bit."""
    g = x.double().unflatten(-1, (D // GROUP, GROUP))
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = torch.minimum(_half_up((hi - lo) / torch.full_like(lo, 15)), _half_down((F16_MAX - lo) / torch.full_like(lo, 15)))
    code = torch.where(s > 0, torch.round((g - lo) / s), torch.zeros_like(g))
    code = code.clamp(0, 15).to(torch.uint8).flatten(-2)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    par = torch.cat([s, lo], -1).half().contiguous().view(torch.uint8).flatten(-2)
    return torch.cat([packed, par], -1)


def _half_up(x):
    """The least fp16 value >= x (x >= 0), as fp64."""
    h = x.half()
    return torch.where(h.double() < x, (h.view(torch.int16) + 1).view(torch.float16), h).double()


def _half_down(x):
    """The greatest fp16 value <= x (x >= 0), as fp64."""
    h = x.half()
    return torch.where(h.double() > x, (h.view(torch.int16) - 1).view(torch.float16), h).double()


def _widen(rows):
    """4-bit rows [..., 80] bytes -> fp32 values [..., 128]."""
    b = rows[..., :D // 2]
    code = torch.stack([b & 15, b >> 4], -1).flatten(-2).float()
    par = rows[..., D // 2:].contiguous().view(torch.float16).float().unflatten(-1, (D // GROUP, 2))
    return (code.unflatten(-1, (D // GROUP, GROUP)) * par[..., :1] + par[..., 1:]).flatten(-2)


def _write(pool, slots, rows):
    bs = pool.shape[2]
    pool[slots // bs, :, slots % bs] = rows


def _plain_append(s):
    for x in ("k", "v"):
        _write(s[x + "_pool"], s["slots"], _quantise(s[x]))
        s[x + "_wide"][s["dst"].long()] = _widen(s[x + "_pool"][s["src"].long()]).half()
    return [s["k_wide"], s["v_wide"]]


def _plain_decode(s):
    tables, lens, q, bs = s["tables"].long(), s["lens"].long(), s["q"], s["bs"]
    b, q_len, hq, _ = q.shape
    hkv = s["k_pool"].shape[1]
    length = tables.shape[1] * bs
    ids = tables.clamp(min=0)

    def gathered(pool):   # [b, hkv, length, 128]
        return _widen(pool[ids].transpose(1, 2).reshape(b, hkv, length, ROW))

    pos = torch.arange(length, device=DEV)
    limit = lens[:, None] - q_len + torch.arange(q_len, device=DEV) + 1
    seen = pos < limit[:, :, None]                                     # [b, q_len, length]
    seen = seen[:, None, :, None, :]
    qg = q.float().view(b, q_len, hkv, hq // hkv, D).transpose(1, 2)   # [b, hkv, q_len, group, 128]
    score = torch.matmul(qg.flatten(2, 3), gathered(s["k_pool"]).transpose(-1, -2))
    score = score.view(b, hkv, q_len, hq // hkv, length) * s["scale"]
    score = torch.where(seen, score, torch.full_like(score, -math.inf))
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    values = gathered(s["v_pool"])
    out = torch.matmul(p.flatten(2, 3), values).view(b, hkv, q_len, hq // hkv, D)
    s["out"].copy_(out.transpose(1, 2).reshape(b, q_len, hq, D))
    return s["out"]


def _plain_fused(s):
    b, q_len = s["q"].shape[:2]
    pos = s["lens"].long()[:, None] - q_len + torch.arange(q_len, device=DEV)
    row = torch.gather(s["tables"].long(), 1, pos.clamp(min=0) // s["bs"])
    slots = (row * s["bs"] + pos % s["bs"]).flatten()
    for x in ("k", "v"):
        _write(s[x + "_pool"], slots, _quantise(s[x]))
    out = _plain_decode(s)
    for x in ("k", "v"):
        s[x + "_wide"][s["dst"].long()] = _widen(s[x + "_pool"][s["src"].long()]).half()
    return [out, s["k_wide"], s["v_wide"]]


def _plain_tables(s):
    bs, tables, free = s["bs"], s["tables"], s["free"]
    n, width = tables.shape
    col = torch.arange(width, device=DEV)
    last = free.numel()

    # cut off what lies past `keep`: those blocks go back on the stack
    lens = s["lens"].long()
    kept = torch.minimum(lens, s["keep"].long())
    gone = (col >= _blocks(kept, bs)[:, None]) & (col < _blocks(lens, bs)[:, None])
    rank = torch.cumsum(gone.flatten(), 0).view(n, width) - 1
    count = s["count"].long()
    total = gone.sum()
    at = torch.where(gone, count + total - 1 - rank, torch.full_like(rank, last))
    spare = torch.cat([free, free[:1]])
    spare[at.flatten()] = tables.flatten()
    tables = torch.where(gone, torch.full_like(tables, -1), tables)
    count = count + total

    # grow for the new tokens: blocks from the top of the stack, sequence after sequence
    new = s["new"].long()
    grown = kept + new
    fresh = (col >= _blocks(kept, bs)[:, None]) & (col < _blocks(grown, bs)[:, None])
    rank = torch.cumsum(fresh.flatten(), 0).view(n, width) - 1
    tables = torch.where(fresh, spare[(count - 1 - rank).clamp(min=0)], tables)
    count = count - fresh.sum()
    ends = torch.cumsum(new, 0)
    token = torch.arange(s["tokens"], device=DEV)
    live = token < ends[-1]
    seq = torch.searchsorted(ends, token, right=True).clamp(max=n - 1)
    pos = kept[seq] + token - (ends - new)[seq]
    slot = tables[seq, (pos // bs).clamp(max=width - 1)].long() * bs + pos % bs
    none = torch.full_like(token, -1)
    s["tables"].copy_(tables)
    s["free"].copy_(spare[:last])
    s["count"].copy_(count)
    s["lens"].copy_(grown)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends]).int()
    return [s["tables"], s["lens"], s["free"], s["count"], torch.where(live, slot, none),
            torch.where(live, seq, none).int(), torch.where(live, pos, none), cu]


def _plain_norm(s):
    c, d = s["table"][s["positions"]][:, None].unbind(-1)              # [t, 1, 64] each

    def one(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * c - b * d, b * c + a * d], -1).half()

    return [one(s["q"], s["q_weight"]), one(s["k"], s["k_weight"])]


# ------------------------------------------------------------------------------------ one pass
def run(s):
    kind = s["kind"]
    if not own:
        return dict(append=_plain_append, decode=_plain_decode, fused=_plain_fused,
                    tables=_plain_tables, norm=_plain_norm)[kind](s)
    from paged_kv_cache_147_gb300 import pkv
    if kind == "append":
        pkv.kv_append_int4(s["k"], s["v"], s["slots"], s["k_pool"], s["v_pool"])
        pkv.widen_blocks_int4(s["k_pool"], s["v_pool"], s["src"], s["dst"], s["k_wide"], s["v_wide"])
        return [s["k_wide"], s["v_wide"]]
    if kind == "decode":
        return pkv.paged_attn_decode_int4(s["out"], s["q"], s["k_pool"], s["v_pool"], s["tables"],
                                          s["lens"], s["scale"], s["workspace"])
    if kind == "fused":
        pkv.paged_attn_decode_append_int4(s["out"], s["q"], s["k"], s["v"], s["k_pool"], s["v_pool"],
                                          s["tables"], s["lens"], s["scale"], s["workspace"])
        pkv.widen_blocks_int4(s["k_pool"], s["v_pool"], s["src"], s["dst"], s["k_wide"], s["v_wide"])
        return [s["out"], s["k_wide"], s["v_wide"]]
    if kind == "tables":
        pkv.truncate_tables(s["tables"], s["lens"], s["keep"], s["bs"], s["free"], s["count"])
        slots, seq, pos, cu = pkv.extend_tables(s["tables"], s["lens"], s["new"], s["bs"],
                                                s["free"], s["count"], s["tokens"])
        return [s["tables"], s["lens"], s["free"], s["count"], slots, seq, pos, cu]
    return list(pkv.qk_norm_rope(s["q"], s["k"], s["q_weight"], s["k_weight"], s["eps"],
                                 s["positions"], s["table"]))


def work(case):
    """Bytes that have to move once, and the products' operations; ragged lengths by their mean."""
    kind = case["kind"]
    if kind == "norm":
        t, heads = case["tokens"], case["hq"] + case["hkv"]
        return dict(bytes=t * heads * D * 4 + t * 8 + min(t, 8192) * D * 4, flops=t * heads * D * 8)
    n, bs = case["seqs"], case["bs"]
    mean = (case["lo"] + case["hi"]) / 2
    if kind == "tables":
        new = n * (1 + case["new"]) // 2
        moved = (n * case["cut"] / 2 + new) / bs
        return dict(bytes=n * 20 + new * 20 + moved * 8, flops=0)
    hkv = case["hkv"]
    wide = hkv * bs * 2 * (ROW + 2 * D)                  # one block's K and V widened
    if kind == "append":
        rows = n * mean * hkv
        return dict(bytes=rows * 2 * (2 * D + ROW) + n * mean * 8 + math.ceil(n * mean / bs) * wide,
                    flops=0)
    q_rows = n * case["q_len"] * case["hq"]
    moved = n * mean * hkv * 2 * ROW + n * math.ceil(mean / bs) * 4 + q_rows * D * 4
    if kind == "fused":
        moved += n * case["q_len"] * hkv * 2 * (2 * D + ROW) + 2 * n * wide
    return dict(bytes=moved, flops=4 * D * q_rows * mean)


# ------------------------------------------------------------------------------------ 64 bits
def _exact_rows(x):
    """What 4-bit rows of x (fp16, [..., 128]) stand for, in 64 bits (numpy)."""
    x = x.cpu().numpy().astype(np.float64)
    g = x.reshape(x.shape[:-1] + (D // GROUP, GROUP))
    z, top = g.min(-1), g.max(-1)
    want, most = (top - z) / 15, (F16_MAX - z) / 15
    s, m = want.astype(np.float16), most.astype(np.float16)
    s = np.where(s.astype(np.float64) < want, np.nextafter(s, np.float16(np.inf)), s)
    m = np.where(m.astype(np.float64) > most, np.nextafter(m, np.float16(0)), m)
    s = np.minimum(s.astype(np.float64), m.astype(np.float64))[..., None]
    z = z[..., None]
    code = np.clip(np.rint((g - z) / np.where(s > 0, s, 1)), 0, 15) * (s > 0)
    return (s * code + z).reshape(x.shape)


def _exact_codes(rows):
    """What stored 4-bit rows (uint8, [..., 80]) stand for, in 64 bits (numpy)."""
    rows = rows.cpu().numpy()
    out = np.empty(rows.shape[:-1] + (D,))
    out[..., 0::2], out[..., 1::2] = rows[..., :64] % 16, rows[..., :64] // 16
    par = np.ascontiguousarray(rows[..., 64:]).view(np.float16).astype(np.float64)
    return out * np.repeat(par[..., 0::2], GROUP, -1) + np.repeat(par[..., 1::2], GROUP, -1)


def _exact_norm(s):
    at = s["table"].double()[s["positions"]]
    turn = torch.complex(at[..., 0], at[..., 1])[:, None]
    out = []
    for x, w in ((s["q"].double(), s["q_weight"].double()), (s["k"].double(), s["k_weight"].double())):
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + s["eps"]) * w
        y = torch.complex(x[..., :64], x[..., 64:]) * turn
        out.append(torch.cat([y.real, y.imag], -1))
    return out


def exact(case, seed):
    kind = case["kind"]
    if kind == "tables":       # whole numbers only
        return None
    s = prepare(case, seed)
    if kind == "norm":
        return _exact_norm(s)
    bs = case["bs"]
    wide = {}
    slots = s.get("slots")
    if kind == "fused":
        q_len = case["q_len"]
        tab, lens = s["tables"].cpu().numpy(), s["lens"].cpu().numpy()
        pos = (lens[:, None] - q_len + np.arange(q_len)).astype(np.int64)
        slots = tab[np.arange(len(lens))[:, None], pos // bs].astype(np.int64) * bs + pos % bs
        slots = torch.as_tensor(slots.reshape(-1))
    if kind != "decode":
        at = slots.cpu().numpy()
        src = s["src"].cpu().numpy()
        for x in ("k", "v"):
            held = _exact_codes(s[x + "_pool"][s["src"].long()])
            new = _exact_rows(s[x])
            for i, blk in enumerate(src):
                for t in np.nonzero(at // bs == blk)[0]:
                    held[i, :, at[t] % bs] = new[t]
            wide[x] = np.zeros(tuple(s[x + "_wide"].shape))     # blocks that no row went to
            wide[x][:len(held)] = held
    if kind == "append":
        return [torch.as_tensor(wide["k"]), torch.as_tensor(wide["v"])]
    out = _exact_attention(s, wide, slots, case)
    return out if kind == "decode" else [out, torch.as_tensor(wide["k"]), torch.as_tensor(wide["v"])]


def _exact_attention(s, wide, slots, case):
    """Textbook attention, one sequence after the other, in 64 bits."""
    bs, q_len = case["bs"], case["q_len"]
    q, lens = s["q"].double(), s["lens"].cpu().tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    group = case["hq"] // case["hkv"]
    new = {x: torch.as_tensor(_exact_rows(s[x])).to(q.device) for x in ("k", "v")} if wide else {}
    for b, n in enumerate(lens):
        blocks = s["tables"][b, :-(-n // bs)].long()

        def rows(x):                                        # [n, hkv, 128]
            raw = s[x + "_pool"][blocks].transpose(1, 2).flatten(0, 1)[:n]
            code = torch.empty(raw.shape[:-1] + (D,), dtype=torch.float64, device=q.device)
            code[..., 0::2], code[..., 1::2] = raw[..., :64] % 16, raw[..., :64] // 16
            par = raw[..., 64:].contiguous().view(torch.float16).double()
            val = code * par[..., 0::2].repeat_interleave(GROUP, -1)
            val += par[..., 1::2].repeat_interleave(GROUP, -1)
            if new:
                val[n - q_len:] = new[x][b * q_len:(b + 1) * q_len]
            return val

        k, v = rows("k"), rows("v")
        for i in range(q_len):
            m = n - q_len + i + 1
            if m <= 0:
                continue
            kh = k[:m].repeat_interleave(group, 1)
            w = torch.softmax((kh * q[b, i]).sum(-1) * s["scale"], 0)
            out[b, i] = (w[..., None] * v[:m].repeat_interleave(group, 1)).sum(0)
    return out
