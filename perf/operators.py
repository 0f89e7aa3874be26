"""Performance cases of the rotary cache append and of attention with modified scores.

Two operators of one serving step, in the order a step runs them:

* ``rope``: the step's queries and keys are rotated by their positions (half or interleaved
  pairs, the whole head or its first part, plain or context-extended frequencies); rotated
  keys and the values are appended to the paged pool, rotated queries are left packed.
* ``attention``: grouped-query attention over the paged pool whose scores are capped by a
  tanh, biased by distance, or masked by a window, documents, a bidirectional prefix or
  padding, for single tokens, short runs and prompt chunks, over bf16, 8-bit and 4-bit pools.

With ``own`` false ``run`` computes them in elementary torch operations, in 32 bits (angles
in 64), rounded once at the end; with ``own`` true it calls the library. ``exact`` is the
definition in 64 bits, written apart from both.
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

def _rope(name, tokens, heads, dim, rot, **more):
    c = {"op": "rope", "tokens": tokens, "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim, "rot_dim": rot,
         "interleaved": False, "scaling": "none", "factor": 1.0, "first": 0, "far": 8192, "decode": True,
         "fused": False, "padded": 0, "block_size": 16, "lengths": 1}
    return dict({"name": name} if name else {}, **c) | more


def _attn(name, heads, dim, **more):
    c = {"op": "attention", "pool": "bf16", "q_heads": heads[0], "kv_heads": heads[1], "head_dim": dim,
         "block_size": 16, "slots": 0, "rows": 1, "ctx_low": 1, "ctx_high": 1, "chunk": 0, "chunk_ctx": 0,
         "softcap": 0.0, "window": 0, "alibi": False, "mask": "causal", "padded": 0, "lengths": 1}
    return dict({"name": name} if name else {}, **c) | more


def listed():
    return [
        # five clients' next tokens at far positions of an extended context: latency
        _rope("rope_decode5", 5, (40, 8), 128, 128, scaling="yarn", factor=16.0, far=131072),
        # a large decode batch, interleaved pairs
        _rope("rope_decode256", 256, (64, 8), 128, 128, interleaved=True, far=32768),
        # a prompt chunk whose projections come as one fused row, half of each head rotated
        _rope("rope_chunk2048", 2048, (32, 8), 128, 64, scaling="parts", factor=8.0, first=6144, decode=False,
              fused=True),
        # a packed step of many prompts, the last rows padding
        _rope("rope_packed24500", 24500, (64, 8), 128, 128, scaling="linear", factor=4.0, first=100000, decode=False,
              fused=True, padded=77),
        # five clients with local layers: latency of capped scores in a window
        _attn("attn_decode5_cap_window", (40, 8), 128, slots=5, ctx_low=1024, ctx_high=8192, softcap=50.0,
              window=1024),
        # a large decode batch with distance biases over whole histories
        _attn("attn_decode256_alibi", (64, 8), 128, slots=256, ctx_low=512, ctx_high=8192, alibi=True),
        # a large decode batch over an 8-bit pool, local layers
        _attn("attn_decode256_cap_window_q8", (64, 8), 128, pool="q8", slots=256, ctx_low=512, ctx_high=16384,
              softcap=30.0, window=4096),
        # drafts of four tokens checked at once, local layers
        _attn("attn_verify4_window", (32, 8), 128, slots=64, rows=4, ctx_low=1024, ctx_high=8192, softcap=50.0,
              window=2048),
        # the last chunk of an 8192-token prompt, capped scores over the whole history
        _attn("attn_chunk2048_cap", (32, 8), 128, chunk=2048, chunk_ctx=8192, softcap=50.0),
        # a chunk deep in a long prompt, local layers
        _attn("attn_chunk4096_window", (32, 8), 128, chunk=4096, chunk_ctx=32768, window=4096),
        # documents packed behind one another, one head per key-value head, distance biases, padding at the end
        _attn("attn_documents8192_alibi", (16, 16), 64, chunk=8192, chunk_ctx=8192, alibi=True, mask="documents",
              padded=100),
        # a prompt chunk with a bidirectional prefix beside four decode rows
        _attn("attn_mixed_prefix", (32, 8), 128, block_size=32, slots=4, ctx_low=200, ctx_high=4000, chunk=509,
              chunk_ctx=1533, softcap=30.0, mask="prefix"),
    ]


def _between(rng, low, high):
    """A whole number spread evenly over its logarithm."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


_HEADS = [(4, 2, 64), (8, 8, 64), (14, 2, 64), (16, 1, 64), (20, 4, 128), (40, 8, 128), (32, 8, 128), (64, 8, 128),
          (6, 6, 128), (24, 2, 128)]


def draw(rng):
    hq, hkv, d = rng.choice(_HEADS)
    more = {"block_size": rng.choice([16, 32, 64]), "lengths": rng.randrange(1 << 20)}
    if rng.random() < 0.4:
        decode = rng.random() < 0.5
        rot = rng.choice([d, d, d // 2, d // 4, d - 8, 2 * rng.randint(1, d // 2)])
        scaling = rng.choice(["none", "linear", "ntk", "parts", "yarn"])
        if scaling == "ntk" and rot < 4:
            scaling = "linear"
        tokens = _between(rng, 1, 512 if decode else 16384)
        return _rope(None, tokens, (hq, hkv), d, rot, interleaved=rng.random() < 0.5, scaling=scaling,
                     factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 7.5, 32.0]),
                     first=_between(rng, 1, 500000), far=_between(rng, 64, 1000000), decode=decode,
                     fused=rng.random() < 0.5, padded=min(tokens // 8, rng.randint(0, 50)), **more)
    pool = rng.choice(["bf16", "bf16", "q8"] + (["q4"] if d == 128 else []))
    score = {"softcap": rng.choice([0.0, 15.0, 30.0, 50.0]), "window": rng.choice([0, 0, _between(rng, 1, 4096)]),
             "alibi": rng.random() < 0.35, "mask": rng.choice(["causal", "causal", "documents", "prefix"])}
    kind = rng.choice(["decode", "run", "chunk", "mixed"])
    if kind in ("decode", "run"):
        rows = 1 if kind == "decode" else rng.randint(2, max(2, 16 // (hq // hkv)))
        low = _between(rng, rows + 1, 2048)
        return _attn(None, (hq, hkv), d, pool=pool, slots=_between(rng, 1, 128 // rows), rows=rows, ctx_low=low,
                     ctx_high=_between(rng, low, 8192), **score, **more)
    chunk = _between(rng, 17, 2048)
    slots = rng.randint(1, 8) if kind == "mixed" else 0
    low = _between(rng, 1, 2048)
    return _attn(None, (hq, hkv), d, pool=pool, slots=slots, ctx_low=low, ctx_high=_between(rng, low, 8192),
                 chunk=chunk, chunk_ctx=chunk + rng.choice([0, _between(rng, 1, 6144)]),
                 padded=rng.choice([0, chunk // 16]), **score, **more)


# ---------------------------------------------------------------------------
# What a case's step looks like (host metadata, the same for every seed)
# ---------------------------------------------------------------------------

def _segments(c):
    """[(rows, context)] of the step's slots, the prompt chunk first."""
    r = random.Random(c["lengths"])
    segs = [(c["chunk"], c["chunk_ctx"])] if c["chunk"] else []
    for _ in range(c["slots"]):
        segs.append((c["rows"], max(c["rows"], _between(r, c["ctx_low"], c["ctx_high"]))))
    return segs


def _row_bounds(c):
    """Per packed row: its segment, its position and the keys [lo, hi) that it sees; and the mask rows the library takes."""
    r = random.Random(c["lengths"] + 1)
    seg, pos, begin, end = [], [], [], []
    for s, (n, ctx) in enumerate(_segments(c)):
        p = np.arange(ctx - n, ctx)
        b, e = np.zeros(n, np.int64), p + 1
        if c["mask"] == "documents":
            starts = [0]
            while starts[-1] < ctx:
                starts.append(starts[-1] + _between(r, 16, 2048))
            starts = np.array(starts)
            b = starts[np.searchsorted(starts, p, side="right") - 1]
        elif c["mask"] == "prefix":
            e = np.maximum(e, r.randint(ctx // 4, ctx))
        if c["padded"] and n == c["chunk"]:  # padding rows see nothing
            b[n - c["padded"]:] = ctx
            e[n - c["padded"]:] = 0
        seg.append(np.full(n, s))
        pos.append(p)
        begin.append(b)
        end.append(e)
    seg, pos, begin, end = (np.concatenate(v) for v in (seg, pos, begin, end))
    lo = begin if not c["window"] else np.maximum(begin, pos - c["window"] + 1)
    ctx = np.array([x for _, x in _segments(c)])[seg]
    return seg, pos, np.maximum(lo, 0), np.minimum(end, ctx), begin, end


def _unions(c):
    """Per segment, the keys [lo, hi) that some row of it sees ((0, 0) where none does)."""
    seg, _, lo, hi, _, _ = _row_bounds(c)
    out = []
    for s in range(len(_segments(c))):
        live = (seg == s) & (lo < hi)
        out.append((int(lo[live].min()), int(hi[live].max())) if live.any() else (0, 0))
    return out


def _positions(c):
    if not c["decode"]:
        return np.arange(c["first"], c["first"] + c["tokens"])
    r = np.random.RandomState(c["lengths"])
    return r.randint(0, c["far"], c["tokens"])


def work(c):
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        t, kept = c["tokens"], c["tokens"] - c["padded"]
        return {"bytes": t * (2 * hq * d * 2 + 4 + 8) + kept * 4 * hkv * d * 2,
                "flops": 3 * c["rot_dim"] * (t * hq + kept * hkv)}
    _, _, lo, hi, _, _ = _row_bounds(c)
    row = {"bf16": 2 * d, "q8": d + d // 16, "q4": d // 2 + d // 16}[c["pool"]]
    keys = sum(b - a for a, b in _unions(c))
    return {"bytes": 2 * keys * hkv * row + 4 * len(lo) * hq * d,
            "flops": 4 * d * hq * int(np.maximum(hi - lo, 0).sum())}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _frequencies(c):
    """Rotation per position of each pair (radians, 64 bits) and the rotated values' factor."""
    n, base, s, original = c["rot_dim"], 10000.0, c["factor"], 4096
    i = np.arange(n // 2, dtype=np.float64)
    f = base ** (-2.0 * i / n)
    if c["scaling"] == "linear":
        f = f / s
    elif c["scaling"] == "ntk":
        f = (base * s ** (n / (n - 2))) ** (-2.0 * i / n)
    elif c["scaling"] == "parts":
        g = np.clip((original * f / (2 * math.pi) - 1.0) / (32.0 - 1.0), 0, 1)
        f = f * (g + (1 - g) / s)
    elif c["scaling"] == "yarn":
        at = lambda turns: n * math.log(original / (2 * math.pi * turns)) / (2 * math.log(base))  # noqa: E731
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), n - 1)
        g = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        f = f * ((1 - g) + g / s)
        return f, 0.1 * math.log(s) + 1.0
    return f, 1.0


def _gpu(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def prepare(c, seed):
    return (_prepare_rope if c["op"] == "rope" else _prepare_attention)(c, seed)


def _prepare_rope(c, seed):
    t, hq, hkv, d, bs = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF16)

    if c["fused"]:  # one row of projections per token
        q, k, v = normal(t, hq + 2 * hkv, d).split([hq, hkv, hkv], dim=1)
    else:
        q, k, v = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
    # decode rows land in one row of each of many blocks, a prompt's rows fill blocks one after another
    blocks = (t if c["decode"] else -(-t // bs)) + 3
    slots = np.random.RandomState(c["lengths"]).permutation(blocks)
    slots = slots[np.arange(t) // (1 if c["decode"] else bs)] * bs + np.arange(t) % bs
    kept = t - c["padded"]
    slots[kept:] = -1
    freqs, magnitude = _frequencies(c)
    s = {"case": c, "q": q, "k": k, "v": v, "positions": _gpu(_positions(c), torch.int32),
         "slot_mapping": _gpu(slots, torch.int64), "kept": kept, "freqs": _gpu(freqs, F64), "magnitude": magnitude,
         "block": _gpu(slots[:kept] // bs, torch.int64), "row": _gpu(slots[:kept] % bs, torch.int64),
         "q_out": torch.empty(t, hq, d, dtype=BF16, device="cuda"), "k_pool": normal(blocks, hkv, bs, d),
         "v_pool": normal(blocks, hkv, bs, d)}
    if own:
        from continuous_batching_paged_pkv_gb300 import binding as B

        kind = {"none": B.PKV_ROPE_NONE, "linear": B.PKV_ROPE_LINEAR, "ntk": B.PKV_ROPE_NTK,
                "parts": B.PKV_ROPE_BY_PARTS, "yarn": B.PKV_ROPE_YARN}[c["scaling"]]
        plan = B.pkv_rope_plan(c["rot_dim"], base=10000.0, scaling=kind, factor=c["factor"], original_len=4096,
                               low=1.0, high=32.0)
        s["call"] = B.RopeCacheWriteCall(q, k, v, s["positions"], plan.phase_tensor("cuda"), s["slot_mapping"],
                                         s["q_out"], s["k_pool"], s["v_pool"], rot_dim=c["rot_dim"],
                                         interleaved=c["interleaved"], magnitude=plan.magnitude)
    return s


def _slopes(c):
    return 2.0 ** (-8.0 * np.arange(1, c["q_heads"] + 1) / c["q_heads"])


def _prepare_attention(c, seed):
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    g = torch.Generator("cuda").manual_seed(seed)
    segs = _segments(c)
    seg, pos, lo, hi, begin, end = _row_bounds(c)
    need = [-(-x // bs) for _, x in segs]
    blocks = sum(need) + 5
    order = np.random.RandomState(c["lengths"]).permutation(blocks)
    tables = np.full((len(segs), max(need)), -1, np.int32)
    at = 0
    for i, m in enumerate(need):
        tables[i, :m] = order[at:at + m]
        at += m

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=BF16)

    # scores of a few units, as trained heads have them; values with an offset per channel, as projections leave them
    q = normal(len(seg), hq, d) * (3.0 if c["softcap"] else 1.0)
    s = {"case": c, "q": q, "tables": _gpu(tables, torch.int32)}
    if c["pool"] == "bf16":
        s["pool"] = (normal(blocks, hkv, bs, d), normal(blocks, hkv, bs, d).add_(normal(hkv, 1, d), alpha=0.5))
    else:
        top = {"q8": 127, "q4": 7}[c["pool"]]

        def codes(shift):
            x = torch.randn(blocks, hkv, bs, d, generator=g, device="cuda", dtype=BF16)
            x = x.add_(shift).mul_(top / 3.0).round_().clamp_(-top, top).to(torch.int8)
            if top == 7:
                x = (x[..., 0::2] & 15) | (x[..., 1::2] << 4)
            return x if top == 127 else x.view(torch.uint8)

        def scales():
            e = torch.randint(0, 2, (blocks, hkv, bs, d // 32), generator=g, device="cuda")
            return torch.exp2(e.to(F32) - (6.0 if top == 127 else 2.0)).to(BF16)

        s["pool"] = (codes(0.0), scales(), codes(0.5 * normal(hkv, 1, d)), scales())
    # maps of the plain form: queries padded to [segments, rows], keys gathered from each segment's union
    groups, row0 = [], 0
    union = _unions(c)
    cu = np.concatenate([[0], np.cumsum([n for n, _ in segs])])
    split = 1 if c["chunk"] else 0
    for part in (range(0, split), range(split, len(segs))):
        part = list(part)
        if not part:
            continue
        n = segs[part[0]][0]
        keys = np.arange(max(1, max(union[i][1] - union[i][0] for i in part)))[None] + np.array(
            [[union[i][0]] for i in part])
        rows = np.arange(row0, row0 + n * len(part)).reshape(len(part), n)
        row0 += n * len(part)
        limit = np.array([[segs[i][1] - 1] for i in part])
        at = np.minimum(keys, limit)
        block = np.take_along_axis(tables[part], at // bs, 1)
        groups.append({"rows": _gpu(rows, torch.int64), "keys": _gpu(keys, torch.int64),
                       "block": _gpu(block, torch.int64), "slot": _gpu(at % bs, torch.int64)})
    s["groups"] = groups
    s["lo"], s["hi"], s["pos"] = (_gpu(x, torch.int64) for x in (lo, hi, pos))
    s["slopes"] = _gpu(_slopes(c), F32) if c["alibi"] else None
    s["out"] = torch.empty(len(seg), hq, d, dtype=BF16, device="cuda")
    if own:
        from continuous_batching_paged_pkv_gb300 import binding as B

        ctx = np.array([x for _, x in segs], np.int32)
        rowmask = c["mask"] != "causal" or c["padded"] > 0
        host = {"key_begin": begin.astype(np.int32), "key_end": end.astype(np.int32)} if rowmask else {}
        work_list, info = B.pkv_plan_work_mod(
            cu, np.arange(len(segs)), ctx, max_slots=len(segs), max_blocks_per_slot=tables.shape[1], block_size=bs,
            num_q_heads=hq, num_kv_heads=hkv, head_dim=d, window=c["window"], **host)
        mod = B.ScoreMod(softcap=c["softcap"], window=c["window"], alibi_slopes=s["slopes"],
                         **{k: _gpu(v, torch.int32) for k, v in host.items()})
        room = info.workspace_bytes if c["pool"] == "bf16" else info.workspace_bytes_q8
        s["call"] = B.AttentionModCall(
            q, _gpu(cu, torch.int32), _gpu(np.arange(len(segs)), torch.int32), _gpu(ctx, torch.int32), s["tables"],
            s["pool"], _gpu(work_list, torch.int32), info, s["out"],
            torch.empty(max(1, room), dtype=torch.uint8, device="cuda"), mod=mod, kv=c["pool"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(s):
    if own:
        s["call"]()
    elif s["case"]["op"] == "rope":
        _plain_rope(s)
    else:
        return s["out"].copy_(_plain_attention(s))
    return (s["q_out"], s["k_pool"], s["v_pool"]) if s["case"]["op"] == "rope" else s["out"]


def _rotate(x, cos, sin, rot, interleaved):
    x = x.to(F32)
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head[..., : rot // 2], head[..., rot // 2:]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((turned, rest), -1).to(BF16)


def _plain_rope(s):
    c, kept = s["case"], s["kept"]
    angle = s["positions"].to(F64)[:, None, None] * s["freqs"]
    cos, sin = ((f(angle) * s["magnitude"]).to(F32) for f in (torch.cos, torch.sin))
    s["q_out"].copy_(_rotate(s["q"], cos, sin, c["rot_dim"], c["interleaved"]))
    k = _rotate(s["k"], cos, sin, c["rot_dim"], c["interleaved"])
    s["k_pool"][s["block"], :, s["row"]] = k[:kept]
    s["v_pool"][s["block"], :, s["row"]] = s["v"][:kept]


def _values(pool, kind, block, slot, which):
    """Keys (which 0) or values (1) at the pool rows, in 32 bits: [segments, kv heads, keys, head_dim]."""
    if kind == "bf16":
        x = pool[which][block, :, slot].to(F32)
    else:
        codes, scales = pool[2 * which][block, :, slot], pool[2 * which + 1][block, :, slot].to(F32)
        if kind == "q4":
            codes = codes.view(torch.int8)
            codes = torch.stack(((codes << 4) >> 4, codes >> 4), -1).flatten(-2)
        x = codes.to(F32) * scales.repeat_interleave(32, -1)
    return x.permute(0, 2, 1, 3)


def _plain_attention(s):
    c = s["case"]
    hq, hkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    parts = []
    for m in s["groups"]:  # the prompt chunk, then the slots with equally many rows each
        n, r = m["rows"].shape
        k, v = (_values(s["pool"], c["pool"], m["block"], m["slot"], w) for w in (0, 1))
        q = s["q"][m["rows"]].to(F32).view(n, r, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
        x = torch.matmul(q.reshape(n, hkv, -1, d), k.transpose(2, 3)).mul_(d ** -0.5).view(n, hkv, hq // hkv, r, -1)
        if c["softcap"]:
            x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
        keys, pos = m["keys"][:, None, :], s["pos"][m["rows"]][:, :, None]
        if c["alibi"]:
            away = (keys - pos).abs().to(F32)[:, None, None]
            x = x.sub_(s["slopes"].view(1, hkv, hq // hkv, 1, 1) * away)
        seen = (keys >= s["lo"][m["rows"]][:, :, None]) & (keys < s["hi"][m["rows"]][:, :, None])
        x = x.masked_fill_(~seen[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x = x.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
        total = x.sum(-1, keepdim=True)
        o = torch.matmul(x.view(n, hkv, -1, x.shape[-1]), v).view(n, hkv, hq // hkv, r, d)
        o = o / torch.where(total == 0, torch.ones_like(total), total)
        parts.append(o.permute(0, 3, 1, 2, 4).reshape(n * r, hq, d))
    return torch.cat(parts).to(BF16)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    with torch.no_grad():
        return (_exact_rope if c["op"] == "rope" else _exact_attention)(prepare(c, seed))


def _exact_rope(s):
    c, rot = s["case"], s["case"]["rot_dim"]
    turn = torch.polar(torch.full_like(s["freqs"], s["magnitude"]).expand(c["tokens"], -1),
                       torch.outer(s["positions"].double(), s["freqs"]))

    def turned(x):
        y = x.double().clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if c["interleaved"] else (
            slice(0, rot // 2), slice(rot // 2, rot))
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    pools = [s["k_pool"].double(), s["v_pool"].double()]
    bs = c["block_size"]
    at = s["slot_mapping"][s["slot_mapping"] >= 0]
    for pool, new in zip(pools, (turned(s["k"]), s["v"].double())):
        flat = pool.transpose(1, 2).clone(memory_format=torch.contiguous_format).view(-1, c["kv_heads"], c["head_dim"])
        flat[at] = new[: len(at)]
        pool.copy_(flat.view(-1, bs, c["kv_heads"], c["head_dim"]).transpose(1, 2))
    return turned(s["q"]), pools[0], pools[1]


def _exact_attention(s):
    c = s["case"]
    hq, hkv, d, bs = c["q_heads"], c["kv_heads"], c["head_dim"], c["block_size"]
    group = hq // hkv
    _, _, lo, hi, _, _ = _row_bounds(c)
    slopes, unions = _slopes(c), _unions(c)
    out = torch.zeros(len(lo), hq, d, dtype=F64, device="cuda")

    def stored(which, blocks, h):
        if c["pool"] == "bf16":
            return s["pool"][which][blocks, h].double().reshape(-1, d)
        code, scale = s["pool"][2 * which][blocks, h], s["pool"][2 * which + 1][blocks, h].double()
        if c["pool"] == "q4":
            low, high = (code & 15).double(), (code >> 4).double()
            code = torch.stack([torch.where(n > 7, n - 16, n) for n in (low, high)], -1).flatten(-2)
        return (code.double().unflatten(-1, (-1, 32)) * scale[..., None]).reshape(-1, d)

    row = 0
    for i, (n, ctx) in enumerate(_segments(c)):
        rows = slice(row, row + n)
        row += n
        a, b = unions[i]
        if b <= a:
            continue
        blocks = s["tables"][i, a // bs:-(-b // bs)].long()
        first = a // bs * bs
        j = torch.arange(a, b, device="cuda")
        seen = (j >= _gpu(lo[rows], torch.int64)[:, None]) & (j < _gpu(hi[rows], torch.int64)[:, None])
        away = (j - torch.arange(ctx - n, ctx, device="cuda")[:, None]).abs().double()
        for h in range(hkv):
            k, v = (stored(w, blocks, h)[a - first:b - first] for w in (0, 1))
            for e in range(h * group, (h + 1) * group):
                x = s["q"][rows, e].double() @ k.T / math.sqrt(d)
                if c["softcap"]:
                    x = c["softcap"] * torch.tanh(x / c["softcap"])
                if c["alibi"]:
                    x = x - float(np.float32(slopes[e])) * away
                x = torch.where(seen, x, -math.inf)
                p = torch.softmax(x, -1).nan_to_num(0.0)  # a row that sees nothing gives zeros
                out[rows, e] = p @ v
    return out
