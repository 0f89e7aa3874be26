"""Work lists, masks, truncation and refusals of block-sparse steps and trees of drafts, and pins of their oracle
(no GPU)."""

import ctypes

import numpy as np
import pytest

from oracle import blocks as OB
from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild

SHAPE = dict(max_slots=9, max_blocks_per_slot=200, block_size=16, num_q_heads=8, num_kv_heads=2, head_dim=64)


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def _step(rng, segs, slots=9):
    cu = np.concatenate([[0], np.cumsum([n for n, _ in segs])]).astype(np.int32)
    ss = rng.permutation(slots)[: len(segs)].astype(np.int32)
    ctx = np.zeros(slots, np.int32)
    ctx[ss] = [c for _, c in segs]
    return cu, ss, ctx


def _parts(work, info):
    items = work[:info.work_words].reshape(-1, 4)
    ends = np.cumsum([info.num_decode_items, info.num_prefill_items, info.num_combine_items, info.num_scratch_items])
    assert len(items) == ends[-1]
    return np.split(items, ends[:3])


def _merges(comb, partials):
    """Every partial entry named by exactly one merge row."""
    seen = []
    for _, _, z, first in comb:
        spans, rows = z & 0xFFFF, ((int(z) >> 24) & 0xFF) + 1
        seen += [first + s * rows for s in range(spans)]
    assert sorted(seen) == list(range(partials))


@pytest.mark.parametrize("seed", range(20))
def test_sparse_list(seed):
    rng = np.random.default_rng(seed)
    hq, hkv, d = [(4, 2, 64), (8, 8, 128), (40, 8, 128), (16, 1, 64)][seed % 4]
    bs = [16, 32, 64][seed % 3]
    most = max(1, 16 // (hq // hkv))
    segs = [(int(rng.integers(0, most + 1)), 0) for _ in range(6)]
    segs = [(n, n + int(rng.integers(0 if n else 1, 6000))) for n, _ in segs]
    sp = B.Sparse(top_blocks=int(rng.integers(8, 60)), keep_first=int(rng.integers(0, 3)), keep_last=int(rng.integers(0, 3)))
    cu, ss, ctx = _step(rng, segs)
    before = int(rng.integers(0, 3)) * 5  # rows of other segments in front
    work, info = B.pkv_plan_work_sparse(cu + before, ss, ctx, max_slots=9, max_blocks_per_slot=-(-6020 // bs), block_size=bs,
                                        num_q_heads=hq, num_kv_heads=hkv, head_dim=d, sparse=sp)
    assert info.modified == 2
    dec, pre, comb, scr = _parts(work, info)
    _merges(comb, info.num_partials)
    cand = {}
    for s, (n, L) in enumerate(segs):
        if n == 0:
            assert not any((x[:, 0] == s).any() for x in (dec, pre, comb, scr))
            continue
        blocks, a, b = OB.always(L, n, bs, sp.keep_first, sp.keep_last)
        read = min(blocks, sp.top_blocks)
        keys = L - (blocks - read) * bs
        got = np.zeros(-(-keys // 16), int)
        for _, slot, w, first in dec[dec[:, 0] == s]:
            w = int(w) & 0xFFFFFFFF
            k0 = (w & 0x7FFFFF) * 16 + (w >> 23 & 15)
            got[k0:k0 + (w >> 27)] += 1
            assert slot == ss[s] and (first >= 0) == (len(dec[dec[:, 0] == s]) > 1)
        assert (got == 1).all()
        (sel,) = pre[pre[:, 0] == s]
        assert sel[3] == (b - a if blocks > sp.top_blocks else 0)
        cand[s] = (sel[2], sel[3])
        parts = sorted(tuple(x) for x in scr[scr[:, 0] == s].tolist())
        assert [p[2] for p in parts] == list(range(0, sel[3], 128)) and all(p[3] == sel[2] for p in parts)
    taken = sorted((f, f + -(-c // 128) * 128) for f, c in cand.values() if c)
    assert all(x[1] == y[0] for x, y in zip(taken, taken[1:])) and all(f % 128 == 0 for f, _ in taken)
    assert info.scratch_blocks == sum(-(-c // 128) * 128 for _, c in cand.values()) == 128 * len(scr)
    need = info.scratch_blocks * hkv * 12
    assert info.workspace_bytes >= need and (info.workspace_bytes == 0 or info.workspace_bytes >= 256)


@pytest.mark.parametrize("seed", range(20))
def test_tree_list(seed):
    rng = np.random.default_rng(seed)
    hq, hkv, d = [(4, 2, 64), (8, 8, 128), (24, 4, 128), (16, 1, 64)][seed % 4]
    segs = [(int(rng.integers(0, [3, 40, 257][seed % 3])), 0) for _ in range(6)]
    segs = [(n, n + int(rng.integers(0 if n else 1, 9000))) for n, _ in segs]
    cu, ss, ctx = _step(rng, segs)
    work, info = B.pkv_plan_work_tree(cu + 7, ss, ctx, max_slots=9, max_blocks_per_slot=600, block_size=16,
                                      num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    assert info.modified == 3 and info.decode_rows_max == max(n for n, _ in segs)
    dec, pre, comb, scr = _parts(work, info)
    assert len(pre) == len(scr) == 0
    _merges(comb, info.num_partials)
    per = 128 // (hq // hkv)
    step = 2 if info.decode_rows_max > per else 1
    for s, (n, L) in enumerate(segs):
        mine = dec[dec[:, 0] == s]
        got = np.zeros((-(-n // per), -(-L // 128)), int)
        for _, slot, w, first in mine:
            w = int(w) & 0xFFFFFFFF
            span, q0 = (w >> 16 & 0xFF) + 1, w >> 24
            got[q0:q0 + step, (w & 0xFFFF) * span:][:, :span] += 1
            assert slot == ss[s] and (first < 0 or first + n <= info.num_partials)
        assert (got == 1).all()


@pytest.mark.parametrize("plan", ["sparse", "tree"])
def test_plan_refusals(plan):
    def status(cu=(0, 1), ss=(0,), ctx=None, sp=B.Sparse(8), **shape):
        c = np.zeros(9, np.int32)
        c[0] = 100
        args = (np.array(cu, np.int32), np.array(ss, np.int32), c if ctx is None else ctx)
        try:
            if plan == "sparse":
                B.pkv_plan_work_sparse(*args, **(SHAPE | shape), sparse=sp)
            else:
                B.pkv_plan_work_tree(*args, **(SHAPE | shape))
        except B.PkvError as e:
            return B.STATUS_NAMES[e.status]
        return "PKV_OK"

    assert status() == "PKV_OK"
    assert status(cu=(0, 0)) == "PKV_OK"
    assert status(cu=(-1, 0)) == "PKV_ERR_INVALID_ARG"
    assert status(cu=(5, 4)) == "PKV_ERR_INVALID_ARG"
    assert status(ss=(9,)) == "PKV_ERR_OUT_OF_RANGE" and status(ss=(-1,)) == "PKV_ERR_OUT_OF_RANGE"
    assert status(cu=(0, 1, 2), ss=(0, 0)) == "PKV_ERR_INVALID_ARG"
    assert status(cu=(0, 101)) in ("PKV_ERR_INVALID_ARG", "PKV_ERR_UNSUPPORTED")
    assert status(ctx=np.full(9, 3201, np.int32)) == "PKV_ERR_OUT_OF_RANGE"
    assert status(ctx=np.full(9, -1, np.int32)) == "PKV_ERR_INVALID_ARG"
    assert status(num_q_heads=7) == "PKV_ERR_INVALID_ARG" and status(num_kv_heads=0) == "PKV_ERR_INVALID_ARG"
    assert status(num_q_heads=34) == "PKV_ERR_UNSUPPORTED" and status(head_dim=96) == "PKV_ERR_UNSUPPORTED"
    assert status(block_size=8) == "PKV_ERR_UNSUPPORTED" and status(max_slots=0) == "PKV_ERR_INVALID_ARG"
    full = np.full(9, 3000, np.int32)
    if plan == "sparse":
        assert status(cu=(0, 4), ctx=full) == "PKV_OK" and status(cu=(0, 5), ctx=full) == "PKV_ERR_UNSUPPORTED"
        assert status(sp=B.Sparse(0)) == "PKV_ERR_INVALID_ARG"
        # 3000 keys: 188 blocks, the last one with the step's row; 2 first and 4 last of 6
        assert status(ctx=full, sp=B.Sparse(7, 2, 4)) == "PKV_OK"
        assert status(ctx=full, sp=B.Sparse(6, 2, 4)) == "PKV_ERR_INVALID_ARG"
        assert status(sp=B.Sparse(6, 9, 9)) == "PKV_ERR_INVALID_ARG" and status(sp=B.Sparse(7, 9, 9)) == "PKV_OK"
        with pytest.raises(ValueError):
            B.Sparse(8, -1).marshal()
    else:
        assert status(cu=(0, 256), ctx=full) == "PKV_OK" and status(cu=(0, 257), ctx=full) == "PKV_ERR_UNSUPPORTED"


def test_sparse_attention_refuses_other_lists():
    """A list of another planner, counts that do not fit, missing buffers: refused before any launch."""
    L = B._lib()
    one, info = B.pkv_plan_work_sparse([0, 1], [0], np.full(9, 3000, np.int32), **SHAPE, sparse=B.Sparse(8))
    sp = B.Sparse(8).marshal()
    p = ctypes.c_void_p(1 << 20)  # never followed

    def attend(info, sparse=sp, q=p, k=p, v=p, sel=p, out=p, ws=p, ws_bytes=1 << 30, d=64, bs=16, hq=8, total=1):
        return B.STATUS_NAMES[L.pkv_attention_sparse(
            q, p, 1, total, p, p, p, 9, 200, bs, k, v, 4000, hq, 2, d, 0.0, None if sparse is None else ctypes.byref(sparse),
            sel, p, ctypes.byref(info), out, ws, ws_bytes, None, None)]

    def select(info, sparse=sp, b=p, sel=p, ws=p, ws_bytes=1 << 30):
        return B.STATUS_NAMES[L.pkv_select_blocks(p, p, 1, 1, p, p, p, 9, 200, 16, b, 4000, 8, 2, 64,
                                                  None if sparse is None else ctypes.byref(sparse), p,
                                                  ctypes.byref(info), sel, ws, ws_bytes, None, None)]

    bad = "PKV_ERR_INVALID_ARG"
    plain = B.pkv_plan_work([0, 1], [0], np.full(9, 3000, np.int32), **SHAPE)[1]
    tree = B.pkv_plan_work_tree([0, 1], [0], np.full(9, 3000, np.int32), **SHAPE)[1]
    for f in (attend, select):
        assert f(plain) == bad and f(tree) == bad
        assert f(info, sparse=None) == bad and f(info, sparse=B.SparseArgs(0, 0, 0)) == bad
        assert f(info, sparse=B.SparseArgs(8, -1, 0)) == bad
        assert f(info, sel=None) == bad and f(info, sel=ctypes.c_void_p(1 << 20 | 2)) == bad
        assert f(info, ws=None) == "PKV_ERR_WORKSPACE_TOO_SMALL" and f(info, ws_bytes=255) == "PKV_ERR_WORKSPACE_TOO_SMALL"
        assert f(info, ws=ctypes.c_void_p(1 << 20 | 16)) == "PKV_ERR_WORKSPACE_TOO_SMALL"
        for field in ("num_decode_items", "num_scratch_items", "num_partials", "scratch_blocks", "decode_rows_max"):
            wrong = B.WorkInfo.from_buffer_copy(info)
            setattr(wrong, field, -1)
            assert f(wrong) == bad
    assert attend(info, q=None) == bad and attend(info, k=None) == bad and attend(info, out=None) == bad
    assert attend(info, k=ctypes.c_void_p(1 << 20 | 8)) == bad and select(info, b=None) == bad
    assert attend(info, d=96) == "PKV_ERR_UNSUPPORTED" and attend(info, bs=8) == "PKV_ERR_UNSUPPORTED"
    wide = B.WorkInfo.from_buffer_copy(info)
    wide.decode_rows_max = 5
    assert attend(wide) == bad
    assert attend(info, total=0) == "PKV_OK"  # nothing to do, nothing launched
    empty = B.pkv_plan_work_sparse([0, 0], [0], np.full(9, 3000, np.int32), **SHAPE, sparse=B.Sparse(8))[1]
    assert attend(empty, q=None) == "PKV_OK" and select(empty) == "PKV_OK"
    # an old call refuses the new lists
    assert L.pkv_attention(p, p, 1, 1, p, p, p, 9, 200, 16, p, p, 4000, 8, 2, 64, 0.0, p, ctypes.byref(info), p, p,
                           1 << 30, None, None) == 1


def test_sparse_list_limits():
    """2^20 blocks to choose among are planned, more are refused."""
    shape = dict(max_slots=1, max_blocks_per_slot=2 ** 21, block_size=16, num_q_heads=8, num_kv_heads=2, head_dim=64)
    fixed = 2  # the first block and that of the step's row
    for blocks, ok in ((2 ** 20 + fixed, True), (2 ** 20 + fixed + 1, False)):
        args = ([0, 1], [0], np.array([blocks * 16], np.int32))
        if ok:
            info = B.pkv_plan_work_sparse(*args, **shape, sparse=B.Sparse(64, 1, 0))[1]
            assert info.num_scratch_items == 2 ** 20 // 128
            continue
        with pytest.raises(B.PkvError) as e:
            B.pkv_plan_work_sparse(*args, **shape, sparse=B.Sparse(64, 1, 0))
        assert B.STATUS_NAMES[e.value.status] == "PKV_ERR_UNSUPPORTED"


def test_tree_attention_refuses_what_does_not_fit():
    """Other planners' lists, masks that are too narrow or too wide, missing or odd buffers: refused before any launch."""
    L = B._lib()
    ctx = np.full(9, 3000, np.int32)
    info = B.pkv_plan_work_tree([0, 40], [0], ctx, **SHAPE)[1]
    p = ctypes.c_void_p(1 << 20)  # never followed

    def attend(info=info, q=p, k=p, v=p, masks=p, words=2, out=p, ws=p, ws_bytes=1 << 30, d=64, bs=16, hq=8, total=40, cu=p):
        return B.STATUS_NAMES[L.pkv_attention_tree(q, cu, 1, total, p, p, p, 9, 200, bs, k, v, 4000, hq, 2, d, 0.0, masks, words,
                                                   p, ctypes.byref(info), out, ws, ws_bytes, None, None)]

    bad = "PKV_ERR_INVALID_ARG"
    for other in (B.pkv_plan_work([0, 1], [0], ctx, **SHAPE)[1],
                  B.pkv_plan_work_sparse([0, 1], [0], ctx, **SHAPE, sparse=B.Sparse(8))[1]):
        assert attend(other) == bad
    assert attend(words=1) == bad and attend(words=0) == bad and attend(words=9) == bad
    for field in ("q", "k", "v", "masks", "out", "cu"):
        assert attend(**{field: None}) == bad
    for field in ("q", "k", "v", "out"):
        assert attend(**{field: ctypes.c_void_p(1 << 20 | 8)}) == bad
    assert attend(masks=ctypes.c_void_p(1 << 20 | 2)) == bad
    assert attend(d=96) == "PKV_ERR_UNSUPPORTED" and attend(bs=8) == "PKV_ERR_UNSUPPORTED"
    assert attend(ws=None) == "PKV_ERR_WORKSPACE_TOO_SMALL" and attend(ws_bytes=255) == "PKV_ERR_WORKSPACE_TOO_SMALL"
    assert attend(ws=ctypes.c_void_p(1 << 20 | 16)) == "PKV_ERR_WORKSPACE_TOO_SMALL"
    for field in ("num_decode_items", "num_prefill_items", "num_scratch_items", "num_partials", "decode_rows_max"):
        wrong = B.WorkInfo.from_buffer_copy(info)
        setattr(wrong, field, -1)
        assert attend(wrong) == bad
    assert attend(total=0) == "PKV_OK"
    empty = B.pkv_plan_work_tree([0, 0], [0], ctx, **SHAPE)[1]
    assert attend(empty, q=None, masks=None) == "PKV_OK"


def test_bounds_and_accept_refusals():
    L = B._lib()
    p = ctypes.c_void_p(1 << 20)
    bounds = lambda m=p, n=1, k=p, nb=10, bs=16, h=2, d=64, b=p: B.STATUS_NAMES[  # noqa: E731
        L.pkv_key_bounds(m, n, k, nb, bs, h, d, b, None, None)]
    bad = "PKV_ERR_INVALID_ARG"
    assert bounds(n=0, m=None, k=None, b=None) == "PKV_OK"
    assert bounds(n=-1) == bad and bounds(nb=0) == bad and bounds(h=0) == bad and bounds(bs=0) == bad
    assert bounds(m=None) == bad and bounds(k=None) == bad and bounds(b=None) == bad
    assert bounds(b=ctypes.c_void_p(1 << 20 | 8)) == bad and bounds(m=ctypes.c_void_p(1 << 20 | 4)) == bad
    assert bounds(nb=2 ** 62) == bad and bounds(d=96) == "PKV_ERR_UNSUPPORTED"
    q = lambda bits, d, s=p: B.STATUS_NAMES[getattr(L, f"pkv_key_bounds_q{bits}")](p, 1, p, s, 10, 16, 2, d, p, None, None)  # noqa: E731,E501
    assert L.pkv_key_bounds_q4(p, 1, p, p, 10, 16, 2, 64, p, None, None) == 3
    assert L.pkv_key_bounds_q8(p, 1, p, None, 10, 16, 2, 64, p, None, None) == 1

    def accept(arrays=(1 << 20,), sizes=(128,), segs=1, path=4, paths=p, nb=10, cu=p, h=2):
        a = (ctypes.c_void_p * len(arrays))(*arrays)
        s = (ctypes.c_int64 * len(sizes))(*sizes)
        return B.STATUS_NAMES[L.pkv_accept_rows(cu, segs, 8, p, p, p, 9, 200, 16, h, paths, path, a, s, len(arrays), nb,
                                                None, None)]

    assert accept(segs=0, cu=None) == "PKV_OK" and accept(path=0) == "PKV_OK"
    assert accept(segs=-1) == bad and accept(path=-1) == bad and accept(cu=None) == bad and accept(paths=None) == bad
    assert accept(arrays=(None,)) == bad and accept(arrays=(1 << 20 | 8,)) == bad
    assert accept(sizes=(0,)) == bad and accept(sizes=(6,)) == bad and accept(nb=0) == bad and accept(h=0) == bad
    assert accept(arrays=(1 << 20,) * 5, sizes=(128,) * 5) == bad and accept(nb=2 ** 60) == bad


def test_tree_masks():
    rng = np.random.default_rng(1)
    for words in (1, 2, 8):
        sizes = [0, 1, int(rng.integers(1, 32 * words)), 32 * words]
        cu = np.concatenate([[3], 3 + np.cumsum(sizes)]).astype(np.int32)
        parents = np.full(cu[-1], 99, np.int32)
        for a, b in zip(cu, cu[1:]):
            for r in range(a, b):
                parents[r] = rng.integers(-1, r - a) if r > a else -1
        masks, depths = B.pkv_tree_masks(parents, cu, words)
        assert (masks[:3] == 0).all() and (depths[:3] == 0).all()
        for a, b in zip(cu, cu[1:]):
            if b == a:
                continue
            seen = OB.tree_seen(parents[a:b], b - a + 5)[:, 5:]
            bits = np.unpackbits(masks[a:b].view(np.uint8), axis=1, bitorder="little")[:, : b - a]
            assert (bits == seen).all() and (depths[a:b] == seen.sum(1) - 1).all()
    assert B.pkv_tree_masks([-1, 0], [0, 2])[0].shape == (2, 1)
    for parents, cu, words, status in (([0], [0, 1], 1, 1), ([-2], [0, 1], 1, 1), ([-1, 1], [0, 2], 1, 1),
                                       ([-1] * 33, [0, 33], 1, 2), ([-1], [0, 1], 0, 1), ([-1], [0, 1], 9, 1)):
        with pytest.raises(B.PkvError) as e:
            B.pkv_tree_masks(parents, cu, words)
        assert e.value.status == status


def test_truncate():
    pool = B.Pool(20, 16, 4, 8)
    assert pool.admit(0, 64) == 0
    pool.lower([(0, 50)])
    before = pool.block_tables()
    pool.truncate(0, 40)
    assert pool.slot_length(0) == 40 and pool.slot_blocks(0) == 4 and (pool.block_tables() == before).all()
    low = pool.lower([(0, 3)])  # the next rows overwrite the rest
    assert low.slot_mapping.tolist() == [int(before[0, 2]) * 16 + r for r in (8, 9, 10)]
    for slot, n, status in ((0, 44, 1), (0, -1, 1), (1, 0, 1), (4, 0, 2), (-1, 0, 2)):
        with pytest.raises(B.PkvError) as e:
            pool.truncate(slot, n)
        assert e.value.status == status
    pool.truncate(0, 0)
    assert pool.slot_length(0) == 0 and pool.slot_blocks(0) == 4
    pool.release(0)
    assert pool.stats().free_blocks == 20


@pytest.mark.parametrize("donor", [False, True])
def test_truncate_leaves_other_tables_blocks_alone(donor):
    """Blocks that two tables hold behind the cut are given up: no later row of either slot lands in them."""
    pool = B.Pool(20, 16, 4, 8)
    assert pool.admit(0, 0) == 0
    pool.lower([(0, 70)])
    assert pool.adopt(1, 0, 60) == 0
    cut, other = (0, 1) if donor else (1, 0)
    held = pool.block_tables()[other]
    held = held[held >= 0].tolist()
    pool.truncate(cut, 20)
    assert pool.slot_blocks(cut) == 2 and pool.block_tables()[other][: len(held)].tolist() == held
    low = pool.lower([(cut, 50)])
    copies = pool.take_copies()
    assert [c.tolist()[0] for c in copies] == [held[1]]
    assert not set(low.slot_mapping // 16) & set(held)
    pool.release(0)
    pool.release(1)
    assert pool.stats().free_blocks == 20


def test_oracle_choice_by_hand():
    lo = np.array([[-1.0, 0], [0, 0], [2, -3], [0, 0], [1, 1], [0, 0]])
    hi = np.array([[1.0, 0], [0, 0], [3, -1], [0, 0], [1, 2], [0, 0]])
    q = np.array([[[1.0, 0.5]], [[-1.0, 0.0]]])  # bounds by block: 1, 0, 2.5, 0, 2, 0
    args = dict(L=90, bs=16, keep_first=1, keep_last=0)
    assert OB.always(90, 2, 16, 1, 0) == (6, 1, 5)
    assert OB.choose(q, lo, hi, top=3, **args) == [0, 2, 5]
    assert OB.choose(q, lo, hi, top=4, **args) == [0, 2, 4, 5]
    assert OB.choose(q, lo, hi, top=5, **args) == [0, 1, 2, 4, 5]  # 1 and 3 tie: the lower place
    assert OB.choose(q, lo, hi, top=6, **args) == [0, 1, 2, 3, 4, 5]


def test_oracle_attention_by_hand():
    v = np.arange(8.0).reshape(4, 1, 2)
    seen = np.array([[1, 0, 0, 1], [0, 0, 0, 0], [0, 1, 0, 0]], bool)
    out, tol = OB.attention(np.zeros((3, 1, 2)), np.zeros((4, 1, 2)), v, seen, 1.0)
    assert np.allclose(out[:, 0], [[3, 4], [0, 0], [2, 3]]) and (tol[1] == 0).all() and (tol[0] > 0).all()
    assert OB.tree_seen([-1, 0, 0, 2], 6).astype(int).tolist() == [
        [1, 1, 1, 0, 0, 0], [1, 1, 1, 1, 0, 0], [1, 1, 1, 0, 1, 0], [1, 1, 1, 0, 1, 1]]


def test_tree_list_limits():
    """Contexts of 65535 spans of 8192 keys are planned, longer ones refused; the spans cover the longest."""
    shape = dict(max_slots=1, max_blocks_per_slot=2 ** 24, block_size=64, num_q_heads=8, num_kv_heads=2, head_dim=64)
    longest = 65535 * 8192
    work, info = B.pkv_plan_work_tree([0, 3], [0], np.array([longest], np.int32), **shape)
    dec, _, comb, _ = _parts(work, info)
    assert info.num_partials == 3 * 65535 and (comb[:, 2] & 0xFFFF == 65535).all()
    assert (dec[:, 2] >> 16 == 63).all() and sorted(dec[:, 2] & 0xFFFF) == list(range(65535))
    for keys in (longest + 1, 2 ** 30 - 1):
        with pytest.raises(B.PkvError) as e:
            B.pkv_plan_work_tree([0, 3], [0], np.array([keys], np.int32), **shape)
        assert B.STATUS_NAMES[e.value.status] == "PKV_ERR_UNSUPPORTED"


def test_blocks_are_copied_in_up_to_five_arrays():
    """A quantised pool's four arrays and the bounds of its keys go in one call."""
    L, p = B._lib(), ctypes.c_void_p(1 << 20)
    for n, status in ((4, 0), (5, 0), (6, 1), (0, 1)):
        arrays, sizes = (ctypes.c_void_p * 6)(*[1 << 20] * 6), (ctypes.c_int64 * 6)(*[1024] * 6)
        assert L.pkv_copy_blocks(p, 0, arrays, sizes, n, 10, None, None) == status


def test_bounds_refuse_more_warps_than_a_grid_holds():
    """2^31 - 1 tokens of 65 heads would wrap to a small grid, those of 32 not launch at all."""
    L, p = B._lib(), ctypes.c_void_p(1 << 20)
    for heads in (32, 65, 65536):
        assert B.STATUS_NAMES[L.pkv_key_bounds(p, 2 ** 31 - 1, p, 10, 16, heads, 64, p, None, None)] == "PKV_ERR_UNSUPPORTED"


def test_tree_masks_read_no_parents_behind_the_last_row():
    """Offsets that fall again are refused before the rows that they seem to name are looked up: the parents stand at
    the end of a page that nothing follows."""
    code = """
import ctypes, mmap
import numpy as np
from continuous_batching_paged_pkv_gb300 import binding as B
page = mmap.PAGESIZE
area = mmap.mmap(-1, 2 * page)
at = ctypes.addressof(ctypes.c_char.from_buffer(area))
libc = ctypes.CDLL(None)
libc.mprotect.argtypes = [ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int]
assert libc.mprotect(at + page, page, 0) == 0
parents = np.frombuffer(area, np.int32, page // 4)
parents[:] = -1
cu = np.array([0, 250, 2], np.int32)
status = B._lib().pkv_tree_masks(at + page - 8, cu.ctypes.data, 2, 8, None, None)
raise SystemExit(0 if status == 1 else 1)
"""
    import subprocess
    import sys
    from pathlib import Path

    run = subprocess.run([sys.executable, "-c", code], cwd=Path(__file__).resolve().parents[1], timeout=300)
    assert run.returncode == 0


@pytest.mark.parametrize("undo", ["truncate", "release"])
def test_a_step_taken_back_before_its_copies_ran(undo):
    """A copy into a block that was given back meanwhile is dropped, and no block is the destination of two; a copy
    into a block that the slot keeps stays."""
    pool = B.Pool(20, 16, 4, 8)
    pool.admit(0, 0)
    pool.lower([(0, 40)])
    for cut in (35, 8):
        pool.adopt(1, 0, 40)
        pool.lower([(1, 1)])
        (_, src), (_, dst) = pool.block_tables()[:2, 1:3].tolist()
        if undo == "truncate":
            pool.truncate(1, cut)
        else:
            pool.release(1)
            pool.adopt(1, 0, 40)
        keeps = undo == "truncate" and cut == 35
        assert pool.slot_blocks(1) == (3 if keeps or undo == "release" else 1)
        pool.adopt(2, 0, 40)
        pool.lower([(2, 1)])
        copies = pool.take_copies().tolist()
        again = int(pool.block_tables()[2, 2])
        assert copies == ([[src, dst], [src, again]] if keeps else [[src, again]]) and (again == dst) == (not keeps)
        pool.release(1)
        pool.release(2)
    pool.release(0)
    assert pool.stats().free_blocks == 20
