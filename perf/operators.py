"""The attention operators over the paged key/value cache, as they are measured.

Four operators, reached as a decoder layer reaches them:

  append    tq.qk_norm_rope: RMS norm of every query and key head, rotation by
            position, keys and values written into their cache slots
  tree      tq.tree_attention: a tree of drafted tokens (or one token) per
            sequence attends to the cache and to its own ancestors
  window    tq.window_attention: causal attention of new tokens over the cache,
            with a sliding window and first tokens that stay visible
  fork, accept, turnover
            tq.cache_fork, tq.cache_accept, tq.cache_free + tq.cache_reserve:
            the cache's pages shared, copied, compacted, freed and reserved

``own`` selects between the plain forms (elementary torch operations in 32
bits) and the library's calls.

Cache layout (one layer): keys [pages, kv_heads, D/8, P, 8], values
[pages, kv_heads, P/8, D, 8]; P tokens a page.
"""
import random

import torch

own = False
DEV = "cuda"
EPS = 1e-6
THETA = 1e7


# ---- the cases ----------------------------------------------------------

def listed():
    return [
        # the four rows of one decode call: q of 24 heads x 256 is the 6144-wide projection
        dict(name="append_4_d256", op="append", tokens=4, seqs=1, hq=24, hkv=4, d=256, rot=64, page=16,
             interleaved=False, fp16=False, far=200000),
        # prompts of five requests in one call, every dimension rotated, adjacent pairs
        dict(name="append_8191_d128", op="append", tokens=8191, seqs=5, hq=32, hkv=8, d=128, rot=128, page=64,
             interleaved=True, fp16=True, far=1000),
        # four drafted rows over a short context: the smallest attention call of a decode step
        dict(name="tree_4_ctx1000", op="tree", seqs=1, nodes=4, ctx=1000, hq=24, hkv=4, d=256, page=16, fp16=False),
        # one token each of 64 requests of unlike lengths: plain batched decoding
        dict(name="tree_1x64_ctx8191", op="tree", seqs=64, nodes=1, ctx=8191, hq=32, hkv=8, d=128, page=32,
             fp16=False),
        # drafted trees of 13 tokens for nine requests, no sharing of key heads
        dict(name="tree_13x9_ctx5000", op="tree", seqs=9, nodes=13, ctx=5000, hq=16, hkv=16, d=64, page=16,
             fp16=True),
        # wide trees over long documents
        dict(name="tree_64x2_ctx131000", op="tree", seqs=2, nodes=64, ctx=131000, hq=24, hkv=4, d=256, page=64,
             fp16=False),
        # one token each over long windowed contexts: only the sinks and the window are read
        dict(name="window_1x32_w1024", op="window", seqs=32, new=1, ctx=32767, window=1024, sinks=4, hq=32, hkv=8,
             d=128, page=16, fp16=False),
        # a first prompt chunk, full causal
        dict(name="window_2048_full", op="window", seqs=1, new=2048, ctx=0, window=0, sinks=0, hq=24, hkv=4, d=256,
             page=16, fp16=False),
        # later prompt chunks of three requests behind a window
        dict(name="window_2047x3_w2500", op="window", seqs=3, new=2047, ctx=6000, window=2500, sinks=5, hq=32, hkv=8,
             d=128, page=32, fp16=True),
        # 24 continuations of six requests: shared pages, the last partial page copied in every layer
        dict(name="fork_24_layers16", op="fork", seqs=6, children=24, ctx=1000, layers=16, hkv=4, d=256, page=16,
             spare=400, fp16=False),
        # the accepted paths of 8 drafted trees move up behind their contexts, in every layer
        dict(name="accept_8x16_layers32", op="accept", seqs=8, nodes=16, keep=5, ctx=777, layers=32, hkv=4, d=256,
             page=16, fp16=False),
        # 16 finished requests leave, 16 new prompts get their pages
        dict(name="turnover_16_of_48", op="turnover", seqs=48, gone=16, ctx=2000, new=1500, page=16, spare=20000),
    ]


HEADS = [(24, 4, 256), (32, 8, 128), (16, 16, 64), (8, 1, 128), (16, 4, 64), (16, 2, 256)]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "append", "tree", "tree", "tree", "window", "window", "window", "fork", "accept",
                     "turnover"])
    hq, hkv, d = rng.choice(HEADS)
    page = rng.choice([16, 32, 64, 128])
    fp16 = rng.random() < 0.4
    if op == "append":
        tokens = _log(rng, 1, 8000)
        return dict(op=op, tokens=tokens, seqs=min(tokens, rng.randint(1, 9)), hq=hq, hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2, d // 4]), page=page, interleaved=rng.random() < 0.5, fp16=fp16,
                    far=_log(rng, 1, 1000000))
    if op == "tree":
        seqs, nodes = _log(rng, 1, 48), _log(rng, 1, 64)
        ctx = _log(rng, 1, min(100000, 200000 // seqs))
        return dict(op=op, seqs=seqs, nodes=nodes, ctx=ctx, hq=hq, hkv=hkv, d=d, page=page, fp16=fp16)
    if op == "window":
        if rng.random() < 0.4:
            seqs, new = _log(rng, 1, 40), _log(rng, 1, 8)
            ctx = _log(rng, 1, min(60000, 400000 // seqs))
        else:
            seqs, new = rng.randint(1, 3), _log(rng, 9, 2000)
            ctx = _log(rng, 1, 6000)
        window = rng.choice([0, _log(rng, 1, 4096), _log(rng, 100, 4096)])
        return dict(op=op, seqs=seqs, new=new, ctx=ctx, window=window, sinks=rng.choice([0, 1, 4, 60]) if window else 0,
                    hq=hq, hkv=hkv, d=d, page=page, fp16=fp16)
    if op == "fork":
        return dict(op=op, seqs=rng.randint(1, 8), children=rng.randint(1, 24), ctx=_log(rng, 20, 1500),
                    layers=rng.randint(1, 16), hkv=min(hkv, 8), d=d, page=min(page, 64), spare=_log(rng, 50, 300),
                    fp16=fp16)
    if op == "accept":
        nodes = rng.randint(2, 40)
        return dict(op=op, seqs=rng.randint(1, 12), nodes=nodes, keep=rng.randint(1, nodes // 2), ctx=_log(rng, 1, 900),
                    layers=rng.randint(1, 32), hkv=min(hkv, 8), d=d, page=min(page, 64), fp16=fp16)
    seqs = rng.randint(2, 60)
    return dict(op=op, seqs=seqs, gone=rng.randint(1, seqs), ctx=_log(rng, 10, 3000), new=_log(rng, 1, 3000),
                page=page, spare=_log(rng, 6000, 60000))


# ---- sizes that follow from a case --------------------------------------

def _spread(top, n, low=8):
    """n unlike lengths from top down to top/low."""
    return [top - (top - top // low) * s // max(1, n - 1) for s in range(n)]


def _contexts(case):
    return _spread(case["ctx"], case["seqs"])


def _counts(case):
    """New tokens of each sequence."""
    if case["op"] == "append":
        n, s = case["tokens"], case["seqs"]
        cuts = [n * (j * (j + 1)) // (s * (s + 1)) for j in range(s + 1)]
        return [b - a for a, b in zip(cuts, cuts[1:])]
    if case["op"] == "tree":
        return [max(1, case["nodes"] - s % 3) for s in range(case["seqs"])]
    return [max(1, n) for n in _spread(case["new"], case["seqs"], 2)]


def _visible(case):
    """(number of query-key pairs, number of keys read) over all sequences."""
    pairs = keys = 0
    for c, n in zip(_contexts(case), _counts(case)):
        if case["op"] == "tree":
            pairs += n * c + n
            keys += c + n
            continue
        w, k = case["window"], case["sinks"]
        if not w:
            pairs += n * c + n * (n + 1) // 2
            keys += c + n
            continue
        for p in range(c, c + n):
            lo = max(0, p - w + 1)
            pairs += p - lo + 1 + min(k, lo)
        lo = max(0, c - w + 1)
        keys += c + n - lo + min(k, lo)
    return pairs, keys


def work(case):
    op = case["op"]
    if op == "append":
        n = case["tokens"] * case["d"]
        moved = n * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 2 * 2 * moved + case["tokens"] * 8, "flops": 10 * n * (case["hq"] + case["hkv"])}
    if op in ("tree", "window"):
        pairs, keys = _visible(case)
        rows = sum(_counts(case)) * case["hq"]
        return {"bytes": 2 * case["d"] * (2 * rows + 2 * keys * case["hkv"]), "flops": 4 * pairs * case["hq"] * case["d"]}
    if op == "fork":
        part = [c % case["page"] for c in _contexts(case)]
        tokens = sum(part[j % case["seqs"]] for j in range(case["children"]))
        table = sum(_contexts(case)[j % case["seqs"]] // case["page"] for j in range(case["children"]))
        return {"bytes": 2 * 2 * 2 * tokens * case["layers"] * case["hkv"] * case["d"] + 16 * table, "flops": 0}
    if op == "accept":
        moved = sum(j != p for s in range(case["seqs"]) for j, p in enumerate(_path(case, s)))
        return {"bytes": max(64, 2 * 2 * 2 * moved * case["layers"] * case["hkv"] * case["d"]), "flops": 0}
    held = sum(-(-c // case["page"]) for c in _contexts(case)[:case["gone"]])
    new = [case["new"] - j for j in range(case["gone"])]
    want = sum(-(-max(1, n) // case["page"]) for n in new)
    return {"bytes": 12 * (held + want) + 4 * sum(max(1, n) for n in new), "flops": 0}


# ---- inputs -------------------------------------------------------------

def _path(case, s):
    """An accepted path of sequence s's tree: ascending nodes from node 0 (the
    token that was decided last).  Drafted rows that it moves lie behind the
    rows that it fills, so that a pass can be repeated on the same cache."""
    nodes, keep = max(1, case["nodes"] - s % 3), max(1, case["keep"] - s % 2)
    r = random.Random(1000 * s + nodes)
    keep = min(keep, (nodes + 1) // 2)
    tail = sorted(r.sample(range(keep, nodes), keep - 1)) if keep > 1 else []
    return [0] + tail


def _tree(n, r):
    """Ancestor masks (the node itself included) of a random tree of n nodes, parents before children."""
    masks = []
    for i in range(n):
        up = masks[r.randrange(max(0, i - 6), i)] if i else 0
        masks.append(up | 1 << i)
    return [m - (1 << 64) if m >> 63 else m for m in masks]


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device=DEV)


def _pages(case, lens, g, spare=3):
    """(page table, page count): the pages of all sequences in random order; unused entries are -1."""
    P = case["page"]
    need = [-(-n // P) for n in lens]
    total = sum(need) + spare
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return table, total


def _pool(shape, dtype, g):
    """Normal values; big pools repeat a drawn block."""
    n = 1
    for v in shape:
        n *= v
    block = torch.randn(min(n, 1 << 24) + 17, generator=g, device=DEV).to(dtype)
    return block.repeat(-(-n // block.numel()))[:n].view(shape)


def _caches(case, pages, dtype, g, layers=None):
    h, d, P = case["hkv"], case["d"], case["page"]
    lead = (pages,) if layers is None else (layers, pages)
    return _pool(lead + (h, d // 8, P, 8), dtype, g), _pool(lead + (h, P // 8, d, 8), dtype, g)


def _dtype(case):
    return torch.float16 if case.get("fp16") else torch.bfloat16


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    r = random.Random(seed)
    op, dt = case["op"], _dtype(case)
    st = dict(case=case)
    if op == "append":
        n, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        # one fused projection output, read in place
        st["qkv"] = torch.randn((n, (hq + 2 * hkv) * d), generator=g, device=DEV).to(dt)
        st["wq"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
        st["wk"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(dt)
        half = case["rot"] // 2
        st["inv_freq"] = (THETA ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
        first = [r.randrange(case["far"]) for _ in range(case["seqs"])]
        counts = _counts(case)
        table, pages = _pages(case, [case["page"] - 1 + c for c in counts], g)      # wherever in a page each begins
        pos, slots = [], []
        for s, (f, c) in enumerate(zip(first, counts)):
            i = torch.arange(c, device=DEV, dtype=torch.int32)
            pos.append(f + i)
            at = f % case["page"] + i
            slots.append(table[s, (at // case["page"]).long()] * case["page"] + at % case["page"])
        st["positions"], st["slots"] = torch.cat(pos), torch.cat(slots)
        st["k"], st["v"] = _caches(case, pages, dt, g)
        return st
    if op in ("tree", "window"):
        ctx, counts = _contexts(case), _counts(case)
        st["table"], pages = _pages(case, [c + n for c, n in zip(ctx, counts)], g)
        st["lengths"] = _ints(ctx)
        starts = [0]
        for n in counts:
            starts.append(starts[-1] + n)
        st["q_start"], st["max_q"] = _ints(starts), max(counts)
        st["q"] = torch.randn((starts[-1], case["hq"], case["d"]), generator=g, device=DEV).to(dt)
        st["k"], st["v"] = _caches(case, pages, dt, g)
        if op == "tree":
            st["ancestors"] = _ints([m for n in counts for m in _tree(n, r)], torch.int64)
        return st
    if op == "fork":
        ctx = _contexts(case)
        rows = case["seqs"] + case["children"]
        table, pages = _pages(case, ctx, g, case["spare"])
        width = table.shape[1]
        st["table"] = torch.cat([table, table.new_full((case["children"], width), -1)])
        st["lengths"] = _ints(ctx + [0] * case["children"])
        st["parents"] = _ints([j % case["seqs"] for j in range(case["children"])])
        st["children"] = _ints(list(range(case["seqs"], rows)))
        st["refs"] = _count_refs(st["table"], pages)
        st["k"], st["v"] = _caches(case, pages, dt, g, case["layers"])
        return st
    if op == "accept":
        ctx = _contexts(case)
        paths = [_path(case, s) for s in range(case["seqs"])]
        most = max(len(p) for p in paths)
        st["path"] = _ints([p + [0] * (most - len(p)) for p in paths])
        st["counts"] = _ints([len(p) for p in paths])
        st["table"], pages = _pages(case, [c + case["nodes"] for c in ctx], g)
        st["lengths"], st["seq_ids"] = _ints(ctx), _ints(list(range(case["seqs"])))
        st["new_lengths"] = torch.zeros_like(st["lengths"])
        st["k"], st["v"] = _caches(case, pages, dt, g, case["layers"])
        return st
    ctx = _contexts(case)
    table, pages = _pages(case, ctx, g, case["spare"])
    width = max(table.shape[1], -(-case["new"] // case["page"]))
    st["table"] = torch.cat([table, table.new_full((case["seqs"], width - table.shape[1]), -1)], 1)
    st["refs"] = _count_refs(table, pages)
    st["lengths"] = _ints(ctx)
    st["gone"] = _ints(r.sample(range(case["gone"]), case["gone"]))
    new = [max(1, case["new"] - j) for j in range(case["gone"])]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st["q_start"], st["tokens"] = _ints(starts), starts[-1]
    return st


def _count_refs(table, pages):
    refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
    return refs.index_add_(0, table.clamp(min=0).flatten().long(), (table >= 0).flatten().to(torch.int32))


# ---- one pass -----------------------------------------------------------

def _qkv(st):
    """Views of the fused projection: q, k, v [tokens, heads, D]."""
    c = st["case"]
    a, b = c["hq"] * c["d"], c["hkv"] * c["d"]
    x = st["qkv"]
    return (x[:, :a].unflatten(1, (c["hq"], c["d"])), x[:, a:a + b].unflatten(1, (c["hkv"], c["d"])),
            x[:, a + b:].unflatten(1, (c["hkv"], c["d"])))


def run(st):
    return (_run_own if own else _run_plain)[st["case"]["op"]](st)


def _own_append(st):
    import trellis_coded_quantized_amd as tq
    q, k, v = _qkv(st)
    out = tq.qk_norm_rope(q, k, v, st["wq"], st["wk"], st["positions"], st["inv_freq"], st["slots"], st["k"], st["v"],
                          eps=EPS, interleaved=st["case"]["interleaved"])
    return out, st["k"], st["v"]


def _own_tree(st):
    import trellis_coded_quantized_amd as tq
    return tq.tree_attention(st["q"], st["k"], st["v"], st["table"], st["lengths"], st["q_start"], st["ancestors"],
                             st["max_q"])


def _own_window(st):
    import trellis_coded_quantized_amd as tq
    return tq.window_attention(st["q"], st["k"], st["v"], st["table"], st["lengths"], st["q_start"], st["max_q"],
                               window=st["case"]["window"], sinks=st["case"]["sinks"])


def _own_fork(st):
    import trellis_coded_quantized_amd as tq
    granted = tq.cache_fork(st["k"], st["v"], st["table"], st["lengths"], st["refs"], st["parents"], st["children"])
    return granted, st["table"], st["lengths"], st["refs"], st["k"], st["v"]


def _own_accept(st):
    import trellis_coded_quantized_amd as tq
    tq.cache_accept(st["k"], st["v"], st["table"], st["lengths"], st["seq_ids"], st["path"], st["counts"],
                    new_lengths=st["new_lengths"])
    return st["new_lengths"], st["k"], st["v"]


def _own_turnover(st):
    import trellis_coded_quantized_amd as tq
    tq.cache_free(st["table"], st["lengths"], st["refs"], st["gone"])
    slots, granted = tq.cache_reserve(st["table"], st["lengths"], st["refs"], st["case"]["page"], st["gone"],
                                      st["q_start"], st["tokens"])
    return slots, granted, st["table"], st["lengths"], st["refs"]


_run_own = dict(append=_own_append, tree=_own_tree, window=_own_window, fork=_own_fork, accept=_own_accept,
                turnover=_own_turnover)


def _norm_rotate(x, w, cos, sin, interleaved):
    x = x.float()
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, y[..., rot:]), -1)


def _plain_append(st):
    c = st["case"]
    q, k, v = _qkv(st)
    angle = st["positions"].double()[:, None, None] * st["inv_freq"].double()     # far positions need 64 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    out = _norm_rotate(q, st["wq"], cos, sin, c["interleaved"]).to(q.dtype)
    kn = _norm_rotate(k, st["wk"], cos, sin, c["interleaved"]).to(k.dtype)
    page, off = (st["slots"] // c["page"]).long(), (st["slots"] % c["page"]).long()
    st["k"][page, :, :, off] = kn.unflatten(-1, (c["d"] // 8, 8))
    st["v"][page, :, off // 8, :, off % 8] = v
    return out, st["k"], st["v"]


def _attend(st, visible):
    """visible: [seqs, max_q, keys] truth values, keys in order of their cache position."""
    c, table = st["case"], st["table"].clamp(min=0).long()
    seqs, top = table.shape[0], st["max_q"]
    group = c["hq"] // c["hkv"]
    k = st["k"][table].permute(0, 2, 1, 4, 3, 5).flatten(2, 3).flatten(3).float()    # [seqs, hkv, keys, D]
    v = st["v"][table].permute(0, 2, 1, 3, 5, 4).flatten(2, 4).float()
    start = st["q_start"].long()
    rows = (start[:-1, None] + torch.arange(top, device=DEV)).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().unflatten(2, (c["hkv"], group)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    s = torch.matmul(q, k.transpose(2, 3)) * c["d"] ** -0.5                           # [seqs, hkv, top * group, keys]
    s = s.unflatten(2, (top, group)).masked_fill_(~visible[:, None, :, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = (s - m.masked_fill(m == float("-inf"), 0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).unflatten(2, (top, group)) / total.masked_fill(total == 0, 1)
    o = o.permute(0, 2, 1, 3, 4).flatten(2, 3)                                        # [seqs, top, hq, D]
    t = torch.arange(st["q"].shape[0], device=DEV)
    s_of = torch.searchsorted(start, t, right=True) - 1
    return o[s_of, t - start[s_of]].to(st["q"].dtype)


def _keys(st):
    """Key positions [1, 1, keys], contexts [seqs, 1, 1], rows [1, max_q, 1], new tokens [seqs, 1, 1]."""
    j = torch.arange(st["table"].shape[1] * st["case"]["page"], device=DEV)[None, None]
    i = torch.arange(st["max_q"], device=DEV)[None, :, None]
    start = st["q_start"].long()
    return j, st["lengths"].long()[:, None, None], i, (start[1:] - start[:-1])[:, None, None]


def _plain_tree(st):
    j, ctx, i, n = _keys(st)
    start = st["q_start"].long()
    rows = (start[:-1, None] + torch.arange(st["max_q"], device=DEV)).clamp(max=st["q"].shape[0] - 1)
    bits = st["ancestors"][rows][:, :, None]
    node = j - ctx
    drafted = (node >= 0) & (node < n) & ((bits >> node.clamp(0, 63)) & 1).bool()
    return _attend(st, (j < ctx) | drafted)


def _plain_window(st):
    j, ctx, i, n = _keys(st)
    pos = ctx + i
    seen = j <= pos
    if st["case"]["window"]:
        seen = seen & ((pos - j < st["case"]["window"]) | (j < st["case"]["sinks"]))
    return _attend(st, seen)


def _lowest_free(refs):
    """Page numbers, the free ones first, each part ascending."""
    return torch.sort((refs != 0).int(), stable=True).indices.to(torch.int32)


def _release(table, refs, rows):
    held = table[rows]
    refs.index_add_(0, held.clamp(min=0).flatten().long(), -(held >= 0).flatten().int())
    table[rows] = -1


def _plain_fork(st):
    c, table, refs = st["case"], st["table"], st["refs"]
    par, kid = st["parents"].long(), st["children"].long()
    rows, length = table[par], st["lengths"][par]
    _release(table, refs, kid)
    full, part = length // c["page"], length % c["page"] > 0
    at = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)[None]
    src = rows.gather(1, full.long()[:, None])[:, 0]
    rank = (part.int().cumsum(0) - part.int()).long()
    granted = ~part | (rank < (refs == 0).sum())
    new = torch.where(part, _lowest_free(refs)[rank], src)
    child = torch.where(at < full[:, None], rows, torch.where((at == full[:, None]) & part[:, None], new[:, None], -1))
    child = torch.where(granted[:, None], child, -1)
    refs.index_add_(0, child.clamp(min=0).flatten().long(), (child >= 0).flatten().int())
    table[kid] = child
    st["lengths"][kid] = torch.where(granted, length, 0)
    to, of = torch.where(granted & part, new, 0).long(), torch.where(granted & part, src, 0).long()
    st["k"][:, to] = st["k"][:, of]
    st["v"][:, to] = st["v"][:, of]
    return granted.int(), table, st["lengths"], refs, st["k"], st["v"]


def _plain_accept(st):
    P, seq = st["case"]["page"], st["seq_ids"].long()
    ctx = st["lengths"][seq].long()[:, None]
    j = torch.arange(st["path"].shape[1], device=DEV)[None]
    keep = j < st["counts"][:, None]
    to, of = ctx + torch.where(keep, j, 0), ctx + torch.where(keep, st["path"].long(), 0)
    tp, op = (st["table"][seq].long().gather(1, x // P) for x in (to, of))
    to, of = to % P, of % P
    st["k"][:, tp, :, :, to] = st["k"][:, op, :, :, of]
    st["v"][:, tp, :, to // 8, :, to % 8] = st["v"][:, op, :, of // 8, :, of % 8]
    st["new_lengths"].copy_(st["lengths"])
    st["new_lengths"][seq] = st["lengths"][seq] + st["counts"]
    return st["new_lengths"], st["k"], st["v"]


def _plain_turnover(st):
    P, table, refs, seq = st["case"]["page"], st["table"], st["refs"], st["gone"].long()
    _release(table, refs, seq)
    st["lengths"][seq] = 0
    start = st["q_start"].long()
    n = start[1:] - start[:-1]
    want = (n + P - 1) // P
    end = want.cumsum(0)
    granted = end <= (refs == 0).sum()
    free = _lowest_free(refs)
    at = torch.arange(table.shape[1], device=DEV)[None]
    use = (at < want[:, None]) & granted[:, None]
    page = torch.where(use, free[torch.where(use, (end - want)[:, None] + at, 0)], -1)
    table[seq] = page
    refs.index_add_(0, page.clamp(min=0).flatten().long(), (page >= 0).flatten().int())
    t = torch.arange(st["tokens"], device=DEV)
    b = torch.searchsorted(start, t, right=True) - 1
    i = t - start[b]
    p = page[b, i // P]
    slots = torch.where(p >= 0, p * P + (i % P).int(), -1)
    return slots, granted.int(), table, st["lengths"], refs


_run_plain = dict(append=_plain_append, tree=_plain_tree, window=_plain_window, fork=_plain_fork,
                  accept=_plain_accept, turnover=_plain_turnover)


# ---- the definition in 64 bits ------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op not in ("append", "tree", "window"):
        return None                       # copies and whole numbers only
    st = prepare(case, seed)
    if op == "append":
        return _exact_append(case, st)
    outs, P, D = [], case["page"], case["d"]
    starts = st["q_start"].tolist()
    for s, ctx in enumerate(st["lengths"].tolist()):
        n = starts[s + 1] - starts[s]
        total = ctx + n
        tab = st["table"][s, :-(-total // P)].long()
        # one sequence, one key head at a time
        heads = []
        for h in range(case["hkv"]):
            K = st["k"][tab, h].double().transpose(1, 2).reshape(-1, D)[:total]
            V = st["v"][tab, h].double().transpose(2, 3).reshape(-1, D)[:total]
            per = case["hq"] // case["hkv"]
            for a in range(per):
                Q = st["q"][starts[s]:starts[s + 1], h * per + a].double()
                heads.append(_exact_rows(case, st, Q, K, V, ctx, starts[s]))
        outs.append(torch.stack(heads, 1))
    return torch.cat(outs)


def _exact_rows(case, st, Q, K, V, ctx, first):
    out = []
    for at in range(0, Q.shape[0], 512):                  # 512 rows of scores at a time
        q = Q[at:at + 512]
        score = q @ K.T / float(case["d"]) ** 0.5
        key = torch.arange(K.shape[0], device=DEV)
        row = at + torch.arange(q.shape[0], device=DEV)
        if case["op"] == "tree":
            anc = st["ancestors"][first + row]
            see = torch.ones_like(score, dtype=torch.bool)
            for node in range(K.shape[0] - ctx):
                see[:, ctx + node] = (anc >> node) % 2 == 1
        else:
            d = (ctx + row)[:, None] - key[None]
            see = d >= 0
            if case["window"]:
                see &= (d < case["window"]) | (key < case["sinks"])[None]
        score[~see] = -float("inf")
        out.append(torch.softmax(score, 1) @ V)
    return torch.cat(out)


def _exact_append(case, st):
    d, rot, P = case["d"], case["rot"], case["page"]
    x = st["qkv"].double().view(case["tokens"], -1, d)
    w = torch.cat([st["wq"].double().expand(case["hq"], d), st["wk"].double().expand(case["hkv"], d)])
    heads = x[:, :case["hq"] + case["hkv"]]
    heads = heads / (heads.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * w
    if case["interleaved"]:
        lo = torch.arange(0, rot, 2, device=DEV)
        hi = lo + 1
    else:
        lo = torch.arange(rot // 2, device=DEV)
        hi = lo + rot // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       st["positions"].double()[:, None] * st["inv_freq"].double()[None])[:, None]
    z = torch.complex(heads[..., lo], heads[..., hi]) * turn
    heads[..., lo], heads[..., hi] = z.real, z.imag
    k, v = st["k"].double(), st["v"].double()
    slot = st["slots"].long()
    pages = k.shape[0]
    # token-major copies of the pools, one row a slot
    kt = k.permute(0, 3, 1, 2, 4).reshape(pages * P, case["hkv"], d)
    vt = v.permute(0, 2, 4, 1, 3).reshape(pages * P, case["hkv"], d)
    kt[slot], vt[slot] = heads[:, case["hq"]:], x[:, case["hq"] + case["hkv"]:]
    k = kt.view(pages, P, case["hkv"], d // 8, 8).permute(0, 2, 3, 1, 4)
    v = vt.view(pages, P // 8, 8, case["hkv"], d).permute(0, 3, 1, 4, 2)
    return heads[:, :case["hq"]], k, v
