"""Performance cases of block-sparse attention and of attention over trees of drafted tokens.

Five operators of serving steps whose rows read part of a paged history, or more than a line of it:

* ``bounds``: after the step's keys are appended, the smallest and the largest key of every
  channel in each block that the step touched.
* ``select``: per slot and key-value head, the cached blocks whose bounds allow the largest
  scores for the slot's queries, beside the first and the newest ones.
* ``sparse``: attention of decode rows and short runs over the selected blocks alone, in bf16,
  8-bit and 4-bit pools.
* ``tree``: attention of a tree of drafted tokens (every row sees the history, its ancestors
  and itself) over the paged pool, the keys split over many SMs.
* ``accept``: the keys and values of the accepted path move to the front of the slot's drafts.

With ``own`` false ``run`` computes them in elementary torch operations, in 32 bits (the
selection's scores in 64, since close ones decide), rounded once at the end; with ``own`` true
it calls the library. ``exact`` is the definition in 64 bits, written apart from both.
"""

import math
import random

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _case(name, op, heads, dim, more, defaults):
    c = {"op": op, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim, "block_size": 16, "lengths": 1}
    return dict({"name": name} if name else {}, **c) | defaults | more


def _bounds(name, heads, dim, **more):
    return _case(name, "bounds", heads, dim, more, {"pool": "bf16", "tokens": 1, "decode": True})


def _select(name, heads, dim, **more):
    return _case(name, "select", heads, dim, more,
                 {"slots": 1, "rows": 1, "ctx_low": 1, "ctx_high": 1, "top": 8, "first": 1, "last": 2})


def _sparse(name, heads, dim, **more):
    return _case(name, "sparse", heads, dim, more,
                 {"pool": "bf16", "slots": 1, "rows": 1, "ctx_low": 1, "ctx_high": 1, "top": 8, "first": 1, "last": 2})


def _tree(name, heads, dim, **more):
    return _case(name, "tree", heads, dim, more,
                 {"slots": 1, "nodes": 1, "ragged": False, "ctx_low": 1, "ctx_high": 1})


def _accept(name, heads, dim, **more):
    return _case(name, "accept", heads, dim, more, {"slots": 1, "nodes": 8, "path": 4, "ctx_low": 32, "ctx_high": 512})


def listed():
    return [
        # 64 clients' next tokens, each in a block of its own that is partly filled
        _bounds("bounds_decode64", (32, 8), 128, tokens=64, block_size=64),
        # a packed step of many prompts
        _bounds("bounds_packed24500", (64, 8), 128, tokens=24500, decode=False),
        # five clients with long histories: the choice of 128 blocks of 16 among thousands
        _select("select_decode5", (40, 8), 128, slots=5, ctx_low=8192, ctx_high=131072, top=128),
        # a large decode batch, 64 blocks of 32 each
        _select("select_decode256", (64, 8), 128, slots=256, ctx_low=512, ctx_high=16384, block_size=32, top=64),
        # five clients with long histories read 2048 keys each: latency
        _sparse("sparse_decode5", (40, 8), 128, slots=5, ctx_low=8192, ctx_high=131072, top=128),
        # a large decode batch reads 2048 keys per slot
        _sparse("sparse_decode256", (64, 8), 128, slots=256, ctx_low=512, ctx_high=16384, block_size=32, top=64),
        # drafts of four tokens checked at once over an 8-bit pool
        _sparse("sparse_verify4_q8", (32, 8), 128, pool="q8", slots=64, rows=4, ctx_low=1024, ctx_high=8192,
                block_size=64, top=24),
        # five clients with a tree of eight drafted tokens each: latency
        _tree("tree_decode5", (40, 8), 128, slots=5, nodes=8, ctx_low=1024, ctx_high=8192),
        # one client, a large tree at the end of a long history
        _tree("tree_one64", (32, 8), 128, slots=1, nodes=64, ctx_low=32768, ctx_high=32768),
        # many clients with trees of 32 tokens
        _tree("tree_decode64", (64, 8), 128, slots=64, nodes=32, ctx_low=512, ctx_high=8192),
        # five clients keep up to four of eight drafted tokens
        _accept("accept_decode5", (40, 8), 128, slots=5),
        # a large batch keeps up to six of 32 drafted tokens
        _accept("accept_decode256", (64, 8), 128, slots=256, nodes=32, path=6, block_size=32),
    ]


def _between(rng, low, high):
    """A whole number spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


_HEADS = [(4, 2, 64), (8, 8, 64), (14, 2, 64), (16, 1, 64), (20, 4, 128), (40, 8, 128), (32, 8, 128), (64, 8, 128),
          (6, 6, 128), (24, 2, 128)]


def draw(rng):
    hq, hkv, d = rng.choice(_HEADS)
    op = rng.choice(["bounds", "select", "select", "sparse", "sparse", "tree", "tree", "accept"])
    more = {"block_size": rng.choice([16, 32, 64]), "lengths": rng.randrange(1 << 20)}
    pool = rng.choice(["bf16", "bf16", "q8"] + (["q4"] if d == 128 else []))
    if op == "bounds":
        decode = rng.random() < 0.5
        return _bounds(None, (hq, hkv), d, pool=pool, tokens=_between(rng, 1, 512 if decode else 16384), decode=decode,
                       **more)
    if op in ("select", "sparse"):
        rows = rng.choice([1, 1, rng.randint(1, max(1, 16 // (hq // hkv)))])
        low = _between(rng, rows + 1, 4096)
        more |= {"rows": rows, "slots": _between(rng, 1, 128 // rows), "ctx_low": low, "first": rng.randint(0, 2),
                 "last": rng.randint(0, 3), "top": _between(rng, 8, 2048 // more["block_size"])}
        if op == "select":
            high = _between(rng, max(low, 4 * more["top"] * more["block_size"]), 32768)
            return _select(None, (hq, hkv), d, ctx_high=high, **more)
        return _sparse(None, (hq, hkv), d, pool=pool, ctx_high=_between(rng, low, 16384), **more)
    if op == "tree":
        nodes = _between(rng, 1, 128)
        low = _between(rng, nodes + 1, 2048)
        return _tree(None, (hq, hkv), d, nodes=nodes, slots=_between(rng, 1, min(64, 1024 // nodes)), ctx_low=low,
                     ctx_high=_between(rng, low, 8192), ragged=rng.random() < 0.5, **more)
    nodes = rng.randint(2, 64)
    return _accept(None, (hq, hkv), d, nodes=nodes, path=rng.randint(1, max(1, min(16, nodes // 2))),
                   slots=_between(rng, 1, 256), ctx_low=nodes, ctx_high=_between(rng, nodes, 512), **more)


# ---------------------------------------------------------------------------
# What a case's step looks like (host metadata, the same for every seed)
# ---------------------------------------------------------------------------

def _segments(c):
    """[(rows, context)] of the step's slots."""
    r = random.Random(c["lengths"])
    most = c["nodes"] if c["op"] in ("tree", "accept") else c["rows"]
    segs = []
    for _ in range(c["slots"]):
        n = r.randint(1, most) if c.get("ragged") else most
        segs.append((n, max(n, _between(r, c["ctx_low"], c["ctx_high"]))))
    if c["op"] == "select":  # one slot at least has more blocks than are selected
        segs[0] = (most, c["ctx_high"])
    return segs


def _kept(c, n, ctx):
    """Blocks of the slot, and the candidates [a, b) among them; all others are always kept."""
    bs = c["block_size"]
    blocks = -(-ctx // bs)
    b = max(0, (ctx - n) // bs - c["last"])
    return blocks, min(c["first"], b), b


def _chosen_keys(c):
    """Per segment, the keys that its rows read in a sparse step."""
    bs = c["block_size"]
    return [ctx - max(0, -(-ctx // bs) - c["top"]) * bs for _, ctx in _segments(c)]


def _path(c, r, n):
    """Accepted drafts: one index per depth, growing. Those that move come from behind the path, so that a pass can
    be repeated on its own result."""
    m = r.randint(1, min(c["path"], n))
    moved = sorted(r.sample(range(m, n), min(n - m, r.randint(0, m - 1))))
    return list(range(m - len(moved))) + moved


def _tokens(c):
    """bounds: pool rows of the step's tokens."""
    t, bs = c["tokens"], c["block_size"]
    r = np.random.RandomState(c["lengths"])
    if c["decode"]:
        return r.permutation(t + 3)[:t].astype(np.int64) * bs + r.randint(0, bs, t), t + 3
    first = r.randint(0, bs)
    at = np.arange(first, first + t)
    blocks = -(-(first + t) // bs) + 3
    return r.permutation(blocks)[at // bs].astype(np.int64) * bs + at % bs, blocks


def _row_bytes(c):
    d = c["head_dim"]
    return {"bf16": 2 * d, "q8": d + d // 16, "q4": d // 2 + d // 16}[c.get("pool", "bf16")]


def work(c):
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    if c["op"] == "bounds":
        slots, _ = _tokens(c)
        blocks, at = np.unique(slots // bs, return_inverse=True)
        rows = np.zeros(len(blocks), np.int64)
        np.maximum.at(rows, at, slots % bs + 1)
        return {"bytes": int(rows.sum()) * hkv * _row_bytes(c) + len(blocks) * hkv * 4 * d + 8 * len(slots),
                "flops": int(rows.sum()) * hkv * d * 2}
    segs = _segments(c)
    if c["op"] == "select":
        cand = [(n, b - a) for n, ctx in segs for _, a, b in [_kept(c, n, ctx)]]
        return {"bytes": sum(m * hkv * 4 * d + n * hq * d * 2 + 4 * hkv * c["top"] for n, m in cand),
                "flops": sum(4 * m * hq * n * d for n, m in cand)}
    if c["op"] == "sparse":
        keys = _chosen_keys(c)
        rows = sum(n for n, _ in segs)
        return {"bytes": sum(keys) * hkv * 2 * _row_bytes(c) + 4 * rows * hq * d + 4 * len(segs) * hkv * c["top"],
                "flops": sum(4 * d * hq * n * k for (n, _), k in zip(segs, keys))}
    if c["op"] == "tree":
        rows = sum(n for n, _ in segs)
        return {"bytes": sum(ctx for _, ctx in segs) * hkv * 4 * d + 4 * rows * hq * d,
                "flops": sum(4 * d * hq * n * ctx for n, ctx in segs)}
    r = random.Random(c["lengths"] + 1)
    moved = sum(p != i for n, _ in segs for i, p in enumerate(_path(c, r, n)))
    return {"bytes": moved * hkv * 8 * d + 4 * len(segs) * c["path"], "flops": 0}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=BF16)


def _pool(c, g, blocks):
    """Keys and values: (k, v) or, in 8 and 4 bits, (codes, scales) of each; values with an offset per channel."""
    hkv, d, bs = c["kv_heads"], c["head_dim"], c["block_size"]
    if c.get("pool", "bf16") == "bf16":
        return (_normal(g, blocks, hkv, bs, d), _normal(g, blocks, hkv, bs, d).add_(_normal(g, hkv, 1, d), alpha=0.5))
    top = {"q8": 127, "q4": 7}[c["pool"]]

    def codes(shift):
        x = _normal(g, blocks, hkv, bs, d).add_(shift).mul_(top / 3.0).round_().clamp_(-top, top).to(torch.int8)
        if top == 7:
            x = (x[..., 0::2] & 15) | (x[..., 1::2] << 4)
        return x if top == 127 else x.view(torch.uint8)

    def scales():
        e = torch.randint(0, 2, (blocks, hkv, bs, d // 32), generator=g, device="cuda")
        return torch.exp2(e.to(F32) - (6.0 if top == 127 else 2.0)).to(BF16)

    return (codes(0.0), scales(), codes(0.5 * _normal(g, hkv, 1, d)), scales())


def _tables(c):
    """Block tables of the step's slots over a shuffled pool, and the pool's blocks."""
    need = [-(-x // c["block_size"]) for _, x in _segments(c)]
    blocks = sum(need) + 5
    order = np.random.RandomState(c["lengths"]).permutation(blocks)
    tables = np.full((len(need), max(need)), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        tables[i, :m] = order[at:at + m]
        at += m
    return tables, blocks


def _step(c):
    """Host metadata of the step: row offsets, slots and context lengths."""
    segs = _segments(c)
    cu = np.concatenate([[0], np.cumsum([n for n, _ in segs])]).astype(np.int32)
    return cu, np.arange(len(segs), dtype=np.int32), np.array([x for _, x in segs], np.int32)


def prepare(c, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = {"case": c}
    {"bounds": _prepare_bounds, "select": _prepare_select, "sparse": _prepare_sparse, "tree": _prepare_tree,
     "accept": _prepare_accept}[c["op"]](c, g, s)
    return s


def _prepare_bounds(c, g, s):
    slots, blocks = _tokens(c)
    bs = c["block_size"]
    s["pool"] = _pool(c, g, blocks)
    s["slot_mapping"] = _gpu(slots, torch.int64)
    touched, at = np.unique(slots // bs, return_inverse=True)
    rows = np.zeros(len(touched), np.int64)
    np.maximum.at(rows, at, slots % bs + 1)
    s["touched"], s["filled"] = _gpu(touched, torch.int64), _gpu(rows, torch.int64)
    s["bounds"] = _normal(g, blocks, c["kv_heads"], 2, c["head_dim"])
    if own:
        from continuous_batching_paged_pkv_gb300 import binding as B

        s["call"] = B.KeyBoundsCall(s["slot_mapping"], s["pool"][: len(s["pool"]) // 2], s["bounds"],
                                    kv=c["pool"])


def _sparse_plan(c, cu, slots, ctx, tables):
    from continuous_batching_paged_pkv_gb300 import binding as B

    sparse = B.Sparse(top_blocks=c["top"], keep_first=c["first"], keep_last=c["last"])
    items, info = B.pkv_plan_work_sparse(
        cu, slots, ctx, max_slots=len(slots), max_blocks_per_slot=tables.shape[1], block_size=c["block_size"],
        num_q_heads=c["q_heads"], num_kv_heads=c["kv_heads"], head_dim=c["head_dim"], sparse=sparse)
    return B, sparse, _gpu(items, torch.int32), info


def _prepare_select(c, g, s):
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    cu, slots, ctx = _step(c)
    tables, blocks = _tables(c)
    s["q"] = _normal(g, cu[-1], hq, d)
    # keys of a block lie around a centre of their own
    centre, spread = _normal(g, blocks, hkv, 1, d), _normal(g, blocks, hkv, 1, d).abs_().add_(0.3)
    s["bounds"] = torch.cat((centre - spread, centre + spread), 2).contiguous()
    s["tables"] = _gpu(tables, torch.int32)
    s["selected"] = torch.full((len(slots), hkv, c["top"]), -2, dtype=torch.int32, device="cuda")
    kept = np.array([_kept(c, n, x) for n, x in _segments(c)])
    s["kept"] = _gpu(kept, torch.int64)
    s["safe"] = _gpu(np.maximum(tables, 0), torch.int64)
    if own:
        B, sparse, items, info = _sparse_plan(c, cu, slots, ctx, tables)
        s["call"] = B.SelectBlocksCall(
            s["q"], _gpu(cu, torch.int32), _gpu(slots, torch.int32), _gpu(ctx, torch.int32), s["tables"], s["bounds"],
            items, info, s["selected"], torch.empty(max(1, info.workspace_bytes), dtype=torch.uint8, device="cuda"),
            sparse=sparse, block_size=c["block_size"])


def _prepare_sparse(c, g, s):
    hq, hkv, d, bs, top = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"], c["top"]
    cu, slots, ctx = _step(c)
    tables, blocks = _tables(c)
    s["q"] = _normal(g, cu[-1], hq, d)
    s["pool"] = _pool(c, g, blocks)
    s["tables"] = _gpu(tables, torch.int32)
    # any choice that holds the first and the newest blocks, in order
    r = np.random.RandomState(c["lengths"] + 2)
    selected = np.full((len(slots), hkv, top), -1, np.int32)
    for i, (n, x) in enumerate(_segments(c)):
        m, a, b = _kept(c, n, x)
        for h in range(hkv):
            some = np.arange(m)
            if m > top:
                some = np.concatenate((np.arange(a), np.arange(b, m), a + r.permutation(b - a)[: top - a - (m - b)]))
            selected[i, h, : len(some)] = np.sort(some)
    s["selected"] = _gpu(selected, torch.int32)
    s["out"] = torch.empty(cu[-1], hq, d, dtype=BF16, device="cuda")
    # maps of the plain form: the keys of each segment's list
    n = c["rows"]
    keys = _chosen_keys(c)
    s["keys"] = _gpu(keys, torch.int64)
    k = np.arange(max(keys))
    logical = np.maximum(np.take_along_axis(selected, np.broadcast_to(k // bs, (len(slots), hkv, len(k))), 2), 0)
    block = np.take_along_axis(np.broadcast_to(tables[:, None], (len(slots), hkv, tables.shape[1])), logical, 2)
    s["block"], s["slot"] = _gpu(np.maximum(block, 0), torch.int64), _gpu(k % bs, torch.int64)
    s["head"] = torch.arange(hkv, device="cuda")[:, None]
    if own:
        B, sparse, items, info = _sparse_plan(c, cu, slots, ctx, tables)
        s["call"] = B.AttentionSparseCall(
            s["q"], _gpu(cu, torch.int32), _gpu(slots, torch.int32), _gpu(ctx, torch.int32), s["tables"], s["pool"],
            s["selected"], items, info, s["out"],
            torch.empty(max(1, info.workspace_bytes), dtype=torch.uint8, device="cuda"), sparse=sparse, kv=c["pool"])


def _trees(c):
    """Ancestor bits of every packed row, 32 nodes to a word: a node's parent is one of the eight before it."""
    r = random.Random(c["lengths"] + 1)
    segs = _segments(c)
    words = -(-max(n for n, _ in segs) // 32)
    parents = []
    masks = np.zeros((sum(n for n, _ in segs), words), np.uint32)
    row = 0
    for n, _ in segs:
        seen = []
        for i in range(n):
            p = r.randint(max(0, i - 8), i - 1) if i else -1
            parents.append(p)
            seen.append((seen[p] if i else 0) | 1 << i)
            for w in range(words):
                masks[row, w] = seen[i] >> 32 * w & 0xFFFFFFFF
            row += 1
    return parents, masks


def _prepare_tree(c, g, s):
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    cu, slots, ctx = _step(c)
    tables, blocks = _tables(c)
    segs = _segments(c)
    s["q"] = _normal(g, cu[-1], hq, d)
    s["pool"] = _pool(c, g, blocks)
    s["tables"] = _gpu(tables, torch.int32)
    _, masks = _trees(c)
    s["masks"] = torch.from_numpy(masks.view(np.int32)).cuda()
    s["out"] = torch.empty(cu[-1], hq, d, dtype=BF16, device="cuda")
    # maps of the plain form: rows and keys padded to the longest segment's
    n = max(m for m, _ in segs)
    row = np.minimum(cu[:-1, None] + np.arange(n), cu[1:, None] - 1)
    s["rows"] = _gpu(row, torch.int64)
    s["packed"] = _gpu(np.concatenate([i * n + np.arange(m) for i, (m, _) in enumerate(segs)]), torch.int64)
    at = np.minimum(np.arange(ctx.max())[None], ctx[:, None] - 1)
    s["block"] = _gpu(np.take_along_axis(tables, at // bs, 1), torch.int64)
    s["slot"] = _gpu(at % bs, torch.int64)
    s["ctx"], s["old"] = _gpu(ctx, torch.int64), _gpu(ctx - np.diff(cu), torch.int64)
    if own:
        from continuous_batching_paged_pkv_gb300 import binding as B

        items, info = B.pkv_plan_work_tree(cu, slots, ctx, max_slots=len(segs), max_blocks_per_slot=tables.shape[1],
                                           block_size=bs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
        s["call"] = B.AttentionTreeCall(
            s["q"], _gpu(cu, torch.int32), _gpu(slots, torch.int32), _gpu(ctx, torch.int32), s["tables"], s["pool"],
            s["masks"], _gpu(items, torch.int32), info, s["out"],
            torch.empty(max(1, info.workspace_bytes), dtype=torch.uint8, device="cuda"))


def _prepare_accept(c, g, s):
    bs = c["block_size"]
    cu, slots, ctx = _step(c)
    tables, blocks = _tables(c)
    s["pool"], s["tables"] = _pool(c, g, blocks), _gpu(tables, torch.int32)
    r = random.Random(c["lengths"] + 1)
    paths = np.full((len(slots), c["path"]), -1, np.int32)
    moves = []
    for i, (n, x) in enumerate(_segments(c)):
        p = _path(c, r, n)
        paths[i, : len(p)] = p
        for to, at in enumerate(p):
            a, b = x - n + at, x - n + to
            moves.append((tables[i, a // bs], a % bs, tables[i, b // bs], b % bs))
    s["paths"] = _gpu(paths, torch.int32)
    s["moves"] = tuple(_gpu(m, torch.int64) for m in np.array(moves).T)
    if own:
        from continuous_batching_paged_pkv_gb300 import binding as B

        s["call"] = B.AcceptRowsCall(_gpu(cu, torch.int32), _gpu(slots, torch.int32), _gpu(ctx, torch.int32),
                                     s["tables"], s["paths"], s["pool"])


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        s["call"]()
    else:
        {"bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse, "tree": _plain_tree,
         "accept": _plain_accept}[op](s)
    return s["pool"] if op == "accept" else s[{"bounds": "bounds", "select": "selected"}.get(op, "out")]


def _values(pool, kind, which, index):
    """Keys (which 0) or values (1) in 32 bits at an index into [blocks, kv heads, block_size]."""
    if kind == "bf16":
        return pool[which][index].to(F32)
    codes, scales = pool[2 * which][index], pool[2 * which + 1][index].to(F32)
    if kind == "q4":
        codes = codes.view(torch.int8)
        codes = torch.stack(((codes << 4) >> 4, codes >> 4), -1).flatten(-2)
    return codes.to(F32) * scales.repeat_interleave(32, -1)


def _plain_bounds(s):
    c = s["case"]
    k = _values(s["pool"], c["pool"], 0, s["touched"])
    empty = torch.arange(c["block_size"], device="cuda") >= s["filled"][:, None]
    empty = empty[:, None, :, None]
    s["bounds"][s["touched"], :, 0] = k.masked_fill(empty, math.inf).amin(2).to(BF16)
    s["bounds"][s["touched"], :, 1] = k.masked_fill(empty, -math.inf).amax(2).to(BF16)


def _plain_select(s):
    c = s["case"]
    hq, hkv, d, n, top = c["q_heads"], c["kv_heads"], c["head_dim"], c["rows"], c["top"]
    slots = len(s["kept"])
    q = s["q"].to(F64).view(slots, n, hkv, hq // hkv, d).transpose(1, 2).reshape(slots, hkv, -1, d)
    b = s["bounds"][s["safe"]].to(F64).permute(0, 2, 3, 4, 1)  # [slots, kv heads, 2, head_dim, blocks]
    x = torch.matmul(q.clamp(min=0), b[:, :, 1]) + torch.matmul(q.clamp(max=0), b[:, :, 0])
    x = x.amax(2)
    blocks, first, last = (s["kept"][:, i, None, None] for i in range(3))
    at = torch.arange(x.shape[2], device="cuda")
    x = x.masked_fill((at < first) | (at >= last), math.inf).masked_fill(at >= blocks, -math.inf)
    order = x.sort(dim=2, descending=True, stable=True).indices[:, :, :top]  # ties: the lowest index first
    order = order.masked_fill(order >= blocks, x.shape[2]).sort(2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, : order.shape[2]] = order.masked_fill(order >= blocks, -1).to(torch.int32)


def _softmax_product(x, seen, v):
    x = x.masked_fill_(~seen, -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.flatten(2, 3), v).view(*x.shape[:-1], -1)
    return o / torch.where(total == 0, torch.ones_like(total), total)


def _plain_sparse(s):
    c = s["case"]
    hq, hkv, d, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["rows"]
    slots = len(s["keys"])
    k, v = (_values(s["pool"], c["pool"], w, (s["block"], s["head"], s["slot"])) for w in (0, 1))
    q = s["q"].to(F32).view(slots, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).mul_(d ** -0.5).view(slots, hkv, hq // hkv, n, -1)
    end = s["keys"][:, None] - n + 1 + torch.arange(n, device="cuda")  # keys that row i sees
    seen = torch.arange(x.shape[-1], device="cuda") < end[:, :, None]
    o = _softmax_product(x, seen[:, None, None], v)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(slots * n, hq, d))


def _plain_tree(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    slots, n = s["rows"].shape
    k, v = (s["pool"][w][s["block"], :, s["slot"]].to(F32).permute(0, 2, 1, 3) for w in (0, 1))
    q = s["q"][s["rows"]].to(F32).view(slots, n, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).mul_(d ** -0.5).view(slots, hkv, hq // hkv, n, -1)
    at = torch.arange(x.shape[-1], device="cuda") - s["old"][:, None]  # place among the drafts, negative in the history
    node = at.clamp(0, 32 * s["masks"].shape[1] - 1)
    word = torch.gather(s["masks"][s["rows"]], 2, (node // 32)[:, None].expand(-1, n, -1))
    bit = (word >> (node % 32)[:, None]) & 1
    seen = (at < 0)[:, None] | ((bit != 0) & (at < (s["ctx"] - s["old"])[:, None])[:, None])
    o = _softmax_product(x, seen[:, None, None], v)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4).reshape(slots * n, hq, d)[s["packed"]])


def _plain_accept(s):
    block, row, to_block, to_row = s["moves"]
    for x in s["pool"]:
        x[to_block, :, to_row] = x[block, :, row]


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    with torch.no_grad():
        return {"bounds": _exact_bounds, "select": _exact_select, "sparse": _exact_sparse, "tree": _exact_tree,
                "accept": _exact_accept}[c["op"]](c, prepare(c, seed))


def _stored(c, pool, which, blocks, h):
    """Rows of some blocks at one kv head, in 64 bits: [blocks * block_size, head_dim]."""
    d = c["head_dim"]
    if c.get("pool", "bf16") == "bf16":
        return pool[which][blocks, h].double().reshape(-1, d)
    code, scale = pool[2 * which][blocks, h], pool[2 * which + 1][blocks, h].double()
    if c["pool"] == "q4":
        low, high = (code & 15).double(), (code >> 4).double()
        code = torch.stack([torch.where(x > 7, x - 16, x) for x in (low, high)], -1).flatten(-2)
    return (code.double().unflatten(-1, (-1, 32)) * scale[..., None]).reshape(-1, d)


def _exact_bounds(c, s):
    out = s["bounds"].double()
    hkv, bs, d = c["kv_heads"], c["block_size"], c["head_dim"]
    newest = {}
    for at in s["slot_mapping"].tolist():
        newest[at // bs] = max(newest.get(at // bs, 0), at % bs + 1)
    for rows in set(newest.values()):
        some = torch.tensor([b for b, m in newest.items() if m == rows], device="cuda")
        for h in range(hkv):
            k = _stored(c, s["pool"], 0, some, h).view(-1, bs, d)[:, :rows]
            out[some, h, 0], out[some, h, 1] = k.min(1).values, k.max(1).values
    return out


def _exact_select(c, s):
    hq, hkv, n, top = c["q_heads"], c["kv_heads"], c["rows"], c["top"]
    group = hq // hkv
    out = torch.full_like(s["selected"], -1)
    for i, (_, ctx) in enumerate(_segments(c)):
        m, a, b = _kept(c, n, ctx)
        for h in range(hkv):
            some = list(range(m))
            if m > top:
                lo, hi = s["bounds"][s["tables"][i, a:b].long(), h].double().unbind(1)
                q = s["q"][i * n:(i + 1) * n, h * group:(h + 1) * group].double().flatten(0, 1)
                best = torch.stack([torch.maximum(x * lo, x * hi).sum(1) for x in q]).max(0).values.tolist()
                ranked = sorted(range(b - a), key=lambda j: (-best[j], j))
                some = sorted(list(range(a)) + list(range(b, m)) + [a + j for j in ranked[: top - a - (m - b)]])
            out[i, h, : len(some)] = torch.tensor(some, dtype=torch.int32, device="cuda")
    return out


def _exact_sparse(c, s):
    hq, hkv, d, bs, n = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"], c["rows"]
    group = hq // hkv
    out = torch.zeros(len(s["q"]), hq, d, dtype=F64, device="cuda")
    for i, (_, ctx) in enumerate(_segments(c)):
        rows = slice(i * n, (i + 1) * n)
        pos = torch.arange(ctx - n, ctx, device="cuda")
        for h in range(hkv):
            some = s["selected"][i, h]
            some = some[some >= 0].long()
            place = (some[:, None] * bs + torch.arange(bs, device="cuda")).flatten()  # in the sequence
            k, v = (_stored(c, s["pool"], w, s["tables"][i, some].long(), h)[place < ctx] for w in (0, 1))
            seen = place[place < ctx] <= pos[:, None]
            for e in range(h * group, (h + 1) * group):
                x = (s["q"][rows, e].double() @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
                out[rows, e] = torch.softmax(x, -1) @ v
    return out


def _exact_tree(c, s):
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    group = hq // hkv
    parents, _ = _trees(c)
    out = torch.zeros(len(s["q"]), hq, d, dtype=F64, device="cuda")
    row = 0
    for i, (n, ctx) in enumerate(_segments(c)):
        seen = np.zeros((n, ctx), bool)
        for j in range(n):
            if parents[row + j] >= 0:
                seen[j] = seen[parents[row + j]]
            else:
                seen[j, : ctx - n] = True
            seen[j, ctx - n + j] = True
        seen = torch.from_numpy(seen).cuda()
        blocks = s["tables"][i, : -(-ctx // bs)].long()
        for h in range(hkv):
            k, v = (_stored(c, s["pool"], w, blocks, h)[:ctx] for w in (0, 1))
            q = s["q"][row:row + n, h * group:(h + 1) * group].double().transpose(0, 1)
            x = (q @ k.T / math.sqrt(d)).masked_fill(~seen, -math.inf)
            out[row:row + n, h * group:(h + 1) * group] = (torch.softmax(x, -1) @ v).transpose(0, 1)
        row += n
    return out


def _exact_accept(c, s):
    bs = c["block_size"]
    out = tuple(x.double() for x in s["pool"])
    for i, (n, ctx) in enumerate(_segments(c)):
        path = [p for p in s["paths"][i].tolist() if p >= 0]
        at = [(int(s["tables"][i, (ctx - n + p) // bs]), (ctx - n + p) % bs) for p in range(n)]
        for new, old in zip(out, s["pool"]):
            for to, p in enumerate(path):
                new[at[to][0], :, at[to][1]] = old[at[p][0], :, at[p][1]].double()
    return out
