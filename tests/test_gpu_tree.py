"""Attention of trees of drafted tokens on the GPU against ``oracle.blocks`` (float64), element by element within the
oracle's tolerance, and a whole verification step: tree, accepted path, cut slot, next step."""

import zlib

import numpy as np
import pytest

import oracle
from oracle import blocks as OB
from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild
from continuous_batching_paged_pkv_gb300 import runtime as R
from continuous_batching_paged_pkv_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    libbuild.build()
    oracle.build()


HEADS = [(4, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (6, 6, 128), (16, 1, 64), (14, 2, 64)]


def _seed(*what):
    return zlib.crc32("/".join(map(str, what)).encode()) % 1000


def _parents(rng, sizes, kind="tree"):
    """Per packed row: a line, a star, a random tree, a forest."""
    out = []
    for n in sizes:
        for i in range(n):
            if i == 0:
                out.append(-1)
            elif kind == "line":
                out.append(i - 1)
            elif kind == "star":
                out.append(0)
            elif kind == "forest":
                out.append(int(rng.integers(-1, i)))
            else:
                out.append(int(rng.integers(max(0, i - 6), i)))
    return out


def _call(ds, masks, out=None, workspace=None, fill=0xFF):
    w, low = ds.w, ds.lowered
    work, info = B.pkv_plan_work_tree(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=w.max_slots,
                                      max_blocks_per_slot=w.max_blocks_per_slot, block_size=w.block_size,
                                      num_q_heads=w.num_q_heads, num_kv_heads=w.num_kv_heads, head_dim=w.head_dim)
    ws = torch.full((max(256, info.workspace_bytes),), fill, dtype=torch.uint8, device="cuda")
    m = torch.from_numpy(np.ascontiguousarray(masks).view(np.int32)).cuda()
    return B.AttentionTreeCall(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, (ds.k_pool, ds.v_pool), m,
                               torch.from_numpy(work).cuda(), info, ds.out if out is None else out, ws, scale=ds.scale,
                               device_status=ds.status), info


def _bits(masks, n):
    return np.unpackbits(np.ascontiguousarray(masks).view(np.uint8), axis=1, bitorder="little")[:, :n].astype(bool)


def _expect(w, masks):
    q = W.bf16_bits_to_f32(w.q).astype(np.float64)
    out, tol, row = np.zeros(q.shape), np.zeros(q.shape), 0
    for s in w.segments:
        rows = slice(row, row + s.q_len)
        row += s.q_len
        k, v = (W.bf16_bits_to_f32(h[s.slot]).astype(np.float64) for h in (w.hist_k, w.hist_v))
        bits = _bits(masks[rows], s.q_len)
        bits = np.pad(bits, ((0, 0), (0, s.q_len - bits.shape[1])))
        seen = np.concatenate([np.ones((s.q_len, s.ctx - s.q_len), bool), bits], 1)
        out[rows], tol[rows] = OB.attention(q[rows], k[: s.ctx], v[: s.ctx], seen, w.scale)
    return out, tol


def _check(ds, masks, what):
    want, tol = _expect(ds.w, masks)
    got = R.out_f32(ds)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), f"{what}: {off.max():.3e} beyond the tolerance, {(off > 0).mean():.2%} of the values"


SHAPES = {
    "one": [(1, 1)],
    "small": [(1, 1), (3, 3), (8, 100), (1, 129), (5, 128), (2, 700)],
    "middle": [(16, 16), (31, 300), (33, 1000), (64, 64), (1, 2000)],
    "large": [(128, 128), (129, 700), (256, 1500), (100, 2049)],
    "long": [(7, 20000), (40, 9000)],
}


@pytest.mark.parametrize("i", range(len(HEADS)))
@pytest.mark.parametrize("case", list(SHAPES))
def test_shapes(case, i):
    hq, hkv, d = HEADS[i]
    rng = np.random.default_rng(i)
    w = W.random_step(_seed(case, i), SHAPES[case], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=[16, 32, 64][i % 3])
    ds = R.prepare(w)
    R.run_cache_write(ds)
    sizes = [n for n, _ in SHAPES[case]]
    for kind in ("tree", "forest"):
        masks, _ = B.pkv_tree_masks(_parents(rng, sizes, kind), ds.lowered.cu_seqlens_q)
        call, _ = _call(ds, masks)
        call()
        assert B.pkv_check_device_status(ds.status) == 0
        _check(ds, masks, f"{case} {hq}/{hkv}/{d} {kind}")


@pytest.mark.parametrize("d", [64, 128])
def test_a_line_is_plain_attention(d):
    w = W.random_step(3, [(8, 900), (1, 300), (64, 2000)], num_q_heads=8, num_kv_heads=2, head_dim=d)
    ds = R.prepare(w)
    R.run_step(ds)
    plain = R.out_f32(ds)
    masks, depths = B.pkv_tree_masks(_parents(None, [8, 1, 64], "line"), ds.lowered.cu_seqlens_q)
    _call(ds, masks)[0]()
    _check(ds, masks, "line")
    assert np.abs(R.out_f32(ds) - plain).max() < 2e-2
    pos = B.pkv_plan_positions(ds.lowered.cu_seqlens_q, ds.lowered.seq_slot, ds.lowered.context_lens)
    first = np.repeat([892, 299, 1936], [8, 1, 64])
    assert (first + depths == pos).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("words", [1, 2, 8])
def test_any_masks(words, d):
    """Masks that are no trees: random rows, themselves or not, rows that see nothing, bits behind the segment."""
    rng = np.random.default_rng(words)
    n = 32 * words
    shapes = [(n, n), (n - 5, n + 100), (1, 1), (min(n, 20), 20), (3, 600)]
    w = W.random_step(50 + words, shapes, num_q_heads=8, num_kv_heads=2, head_dim=d)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    masks = rng.integers(0, 2 ** 32, (w.total_q, words), dtype=np.uint32)
    masks[rng.random(w.total_q) < 0.3] = 0
    masks[rng.random(w.total_q) < 0.2] = 0xFFFFFFFF
    masks[n + n - 5] = 0  # the segment of one row: it sees nothing
    _call(ds, masks)[0]()
    assert B.pkv_check_device_status(ds.status) == 0
    _check(ds, masks, f"{words} words")
    empty = np.concatenate([[not _bits(masks[a:b][r:r + 1], b - a).any() and s.ctx == s.q_len for r in range(b - a)]
                            for s, a, b in zip(w.segments, ds.lowered.cu_seqlens_q, ds.lowered.cu_seqlens_q[1:])])
    assert empty.any() and (R.out_f32(ds)[empty] == 0).all()


@pytest.mark.parametrize("size", [0.0, 12.0])
def test_peaked_and_flat_scores(size):
    w = W.random_step(6, [(40, 1900), (8, 300)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    w.q = W.f32_to_bf16_bits(W.bf16_bits_to_f32(w.q) * size)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [40, 8]), ds.lowered.cu_seqlens_q)
    _call(ds, masks)[0]()
    _check(ds, masks, str(size))


def test_scores_that_rise_along_the_history():
    """Every tile raises the running maximum: the output is rescaled again and again."""
    for d in (64, 128):
        w = W.random_step(7, [(16, 3000), (40, 1000)], num_q_heads=8, num_kv_heads=2, head_dim=d)
        for slot in w.hist_k:
            k = W.bf16_bits_to_f32(w.hist_k[slot])
            k[..., 0] = np.linspace(-60, 60, len(k))[:, None]
            w.hist_k[slot][...] = W.f32_to_bf16_bits(k)
        q = W.bf16_bits_to_f32(w.q)
        q[..., 0] = 8.0
        w.q = W.f32_to_bf16_bits(q)
        ds = R.prepare(w)
        R.run_cache_write(ds)
        masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [16, 40]), ds.lowered.cu_seqlens_q)
        _call(ds, masks)[0]()
        _check(ds, masks, str(d))


def test_behind_the_chunks_of_a_mixed_step():
    """Prompt chunks first, trees behind them: one call each on parts of the same packed step."""
    shapes = [(70, 300), (200, 200), (9, 1000), (40, 640)]
    w = W.random_step(8, shapes, num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    ds.out.fill_(5.0)
    low = ds.lowered
    parents = [0] * 270 + _parents(np.random.default_rng(0), [9, 40])
    masks, _ = B.pkv_tree_masks(parents, low.cu_seqlens_q[2:])
    shape = dict(max_slots=w.max_slots, max_blocks_per_slot=w.max_blocks_per_slot, block_size=16, num_q_heads=32,
                 num_kv_heads=8, head_dim=128)
    work, info = B.pkv_plan_work_tree(low.cu_seqlens_q[2:], low.seq_slot[2:], low.context_lens, **shape)
    ws = torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda")
    B.pkv_attention_tree(ds.q, ds.cu_seqlens_q[2:].contiguous(), ds.seq_slot[2:].contiguous(), ds.context_lens,
                         ds.block_tables, ds.k_pool, ds.v_pool, torch.from_numpy(masks.view(np.int32)).cuda(),
                         torch.from_numpy(work).cuda(), info, ds.out, ws, scale=ds.scale, device_status=ds.status)
    trees = ds.out.clone()
    assert (trees[:270] == 5).all()
    work, info = B.pkv_plan_work(low.cu_seqlens_q[:3], low.seq_slot[:2], low.context_lens, **shape)
    B.pkv_attention(ds.q[:270], ds.cu_seqlens_q[:3].contiguous(), ds.seq_slot, ds.context_lens, ds.block_tables, ds.k_pool,
                    ds.v_pool, torch.from_numpy(work).cuda(), info, ds.out[:270], scale=ds.scale, device_status=ds.status)
    assert B.pkv_check_device_status(ds.status) == 0 and torch.equal(ds.out[270:], trees[270:])
    line, _ = B.pkv_tree_masks(_parents(None, [70, 200], "line") + parents[270:], low.cu_seqlens_q, masks.shape[1] + 5)
    _check(ds, line, "mixed")


def test_captured_replayed_and_on_another_stream():
    w = W.random_step(9, [(8, 3000), (64, 500), (1, 1)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [8, 64, 1]), ds.lowered.cu_seqlens_q)
    call, info = _call(ds, masks)
    assert info.num_combine_items > 0

    def step():
        R.run_cache_write(ds)
        call()

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for scale in (1.0, -0.5):
        ds.q.mul_(scale)
        ds.v_new.mul_(scale)
        step()
        torch.cuda.synchronize()
        want = ds.out.clone()
        ds.out.fill_(3.0)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(ds.out, want) and B.pkv_check_device_status(ds.status) == 0


def test_calls_one_behind_another_with_one_workspace():
    """Two steps' calls in a row over the same workspace: the second's partials wait for the first's merge."""
    w = W.random_step(10, [(16, 6000)] * 4, num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [16] * 4), ds.lowered.cu_seqlens_q)
    call, _ = _call(ds, masks)
    call()
    torch.cuda.synchronize()
    want = ds.out.clone()
    for _ in range(20):
        call()
    torch.cuda.synchronize()
    assert torch.equal(ds.out, want)


def test_results_do_not_depend_on_the_rest_of_the_step():
    """A tree alone (one query tile per CTA) and beside larger ones (two): the same bits."""
    rng = np.random.default_rng(0)
    for d in (64, 128):
        shapes = [(8, 3000), (64, 2500), (30, 500), (1, 900)]
        w = W.random_step(11, shapes, num_q_heads=8, num_kv_heads=2, head_dim=d)
        ds = R.prepare(w)
        R.run_cache_write(ds)
        cu = ds.lowered.cu_seqlens_q
        masks, _ = B.pkv_tree_masks(_parents(rng, [n for n, _ in shapes]), cu)
        _call(ds, masks)[0]()
        out = ds.out.clone()
        for order in ([0], [1], [2], [3], [3, 0], list(rng.permutation(4))):
            q = torch.cat([ds.q[cu[s]:cu[s + 1]] for s in order])
            m = np.concatenate([masks[cu[s]:cu[s + 1]] for s in order])
            c2 = np.concatenate([[0], np.cumsum([shapes[s][0] for s in order])]).astype(np.int32)
            work, info = B.pkv_plan_work_tree(c2, ds.lowered.seq_slot[order], ds.lowered.context_lens, max_slots=w.max_slots,
                                              max_blocks_per_slot=w.max_blocks_per_slot, block_size=16, num_q_heads=8,
                                              num_kv_heads=2, head_dim=d)
            o2 = torch.empty_like(q)
            B.pkv_attention_tree(q, torch.from_numpy(c2).cuda(), ds.seq_slot[torch.tensor(order).cuda()].contiguous(),
                                 ds.context_lens, ds.block_tables, ds.k_pool, ds.v_pool,
                                 torch.from_numpy(m.view(np.int32)).cuda(), torch.from_numpy(work).cuda(), info, o2,
                                 torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda"), scale=w.scale)
            for i, s in enumerate(order):
                assert torch.equal(o2[c2[i]:c2[i + 1]], out[cu[s]:cu[s + 1]]), (d, order, s)


def test_bad_blocks_and_lists_are_reported():
    w = W.random_step(12, [(8, 3000), (40, 500)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [8, 40]), ds.lowered.cu_seqlens_q)
    call, _ = _call(ds, masks)
    tables = ds.block_tables.clone()
    for bad in (-1, w.num_blocks, 2 ** 30):
        ds.block_tables[0, 7] = bad
        call()
        assert B.pkv_check_device_status(ds.status) == 2
        ds.block_tables.copy_(tables)
    for lens in ([2000, 500], [3000, 39], [0, 500]):  # a list made for longer contexts
        ds.context_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        call()
        assert B.pkv_check_device_status(ds.status) & 4
    ds.context_lens.copy_(torch.tensor([3000, 500], dtype=torch.int32))
    call()
    assert B.pkv_check_device_status(ds.status) == 0
    _check(ds, masks, "mended")


def test_calls_refuse_what_does_not_fit():
    w = W.random_step(13, [(40, 300)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    masks, _ = B.pkv_tree_masks(_parents(None, [40], "line"), ds.lowered.cu_seqlens_q)
    with pytest.raises(ValueError):
        _call(ds, masks[:39])
    with pytest.raises(ValueError):
        _call(ds, masks, out=ds.out[:, :4].contiguous())
    with pytest.raises(B.PkvError) as e:  # a word too few for 40 rows
        _call(ds, masks[:, :1])[0]()
    assert e.value.status == 1
    with pytest.raises(B.PkvError) as e:
        _call(ds, np.zeros((40, 9), np.uint32))[0]()
    assert e.value.status == 1


def test_a_verification_step():
    """Drafts as a tree; the best path is kept, the slot cut there, and the next step sees what a plain run sees."""
    rng = np.random.default_rng(5)
    bs, hq, hkv, d, hist, n = 16, 8, 2, 64, 75, 13
    parents = np.array(_parents(rng, [n], "tree"), np.int32)
    path = [n - 1]
    while parents[path[-1]] >= 0:
        path.append(int(parents[path[-1]]))
    path = path[::-1]
    x = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    k, v, qt, q1 = x(hist + n + 1, hkv, d), x(hist + n + 1, hkv, d), x(n, hq, d), x(1, hq, d)
    shape = dict(max_slots=1, max_blocks_per_slot=16, block_size=bs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731

    def write(pool, kv, rows, count):
        low = pool.lower([(0, count)])
        B.pkv_cache_write(k[rows].contiguous(), v[rows].contiguous(), dev(low.slot_mapping), *kv)
        return low

    def attend(low, pool, kv, q):
        work, info = B.pkv_plan_work(low.cu_seqlens_q, low.seq_slot, low.context_lens, **shape)
        out = torch.empty_like(q)
        ws = torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda")
        B.pkv_attention(q, dev(low.cu_seqlens_q), dev(low.seq_slot), dev(low.context_lens), dev(pool.block_tables()), *kv,
                        dev(work), info, out, ws)
        return out

    kv = R.empty_pool(32, hkv, bs, d, "cuda")
    pool = B.Pool(32, bs, 1, 16)
    pool.admit(0, 0)
    write(pool, kv, slice(0, hist), hist)
    low = write(pool, kv, slice(hist, hist + n), n)
    masks, depths = B.pkv_tree_masks(parents, low.cu_seqlens_q)
    work, info = B.pkv_plan_work_tree(low.cu_seqlens_q, low.seq_slot, low.context_lens, **shape)
    meta = [dev(a) for a in (low.cu_seqlens_q, low.seq_slot, low.context_lens, pool.block_tables())]
    out = torch.empty_like(qt)
    B.pkv_attention_tree(qt, *meta, *kv, dev(masks.view(np.int32)), dev(work), info, out,
                         torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda"))
    B.pkv_accept_rows(*meta, torch.tensor([path], dtype=torch.int32, device="cuda"), kv, total_q=n)
    pool.truncate(0, hist + len(path))
    low = write(pool, kv, slice(hist + n, hist + n + 1), 1)
    got = attend(low, pool, kv, q1)

    # the same tokens in a line
    kept = list(range(hist)) + [hist + p for p in path] + [hist + n]
    kv2 = R.empty_pool(32, hkv, bs, d, "cuda")
    pool2 = B.Pool(32, bs, 1, 16)
    pool2.admit(0, 0)
    write(pool2, kv2, kept[:hist], hist)
    low2 = write(pool2, kv2, kept[hist:-1], len(path))
    line = attend(low2, pool2, kv2, qt[path].contiguous())
    low2 = write(pool2, kv2, kept[-1:], 1)
    assert torch.equal(got, attend(low2, pool2, kv2, q1))
    # the path's rows of the tree are those of the line
    q64, k64, v64 = (t.double().cpu().numpy() for t in (qt[path], k[kept[:-1]], v[kept[:-1]]))
    want, tol = OB.attention(q64, k64, v64, OB.tree_seen(list(range(-1, len(path) - 1)), len(kept) - 1), d ** -0.5)
    for o in (out[path], line):
        assert (np.abs(o.double().cpu().numpy() - want) <= tol).all()
    assert (depths[path] == np.arange(len(path))).all()


def test_bounds_behind_an_accepted_path():
    """A tree whose accepted rows move over block ends: bounds made anew for those rows, and the choice that follows."""
    bs, hq, hkv, d, hist, n = 16, 8, 2, 128, 250, 40
    path = [0, 2, 3, 9, 11, 12, 20, 21, 33, 39]
    x = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    k, v, q = x(hist + n + 1, hkv, d), x(hist + n + 1, hkv, d), x(1, hq, d)
    kv, status = R.empty_pool(32, hkv, bs, d, "cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    bounds = torch.full((32, hkv, 2, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool = B.Pool(32, bs, 1, 20)
    pool.admit(0, 0)

    def write(first, count):
        low = pool.lower([(0, count)])
        m = dev(low.slot_mapping)
        B.pkv_cache_write(k[first:first + count], v[first:first + count], m, *kv)
        B.pkv_key_bounds(m, kv[0], bounds, device_status=status)
        return low

    write(0, hist)
    low = write(hist, n)
    meta = [dev(a) for a in (low.cu_seqlens_q, low.seq_slot, low.context_lens, pool.block_tables())]
    B.pkv_accept_rows(*meta, torch.tensor([path + [-1]], dtype=torch.int32, device="cuda"), kv, total_q=n, device_status=status)
    kept = low.slot_mapping.copy()
    kept[len(path):] = -1
    B.pkv_key_bounds(dev(kept), kv[0], bounds, device_status=status)
    pool.truncate(0, hist + len(path))
    low = write(hist + n, 1)
    keys = k[list(range(hist)) + [hist + p for p in path] + [hist + n]].double().cpu().numpy()
    want = np.stack([OB.bounds(keys[i:i + bs]) for i in range(0, len(keys), bs)])  # [blocks, 2, heads, D]
    table = pool.block_tables()[0][: len(want)]
    assert np.array_equal(bounds[torch.from_numpy(table).cuda().long()].double().cpu().numpy(), want.transpose(0, 2, 1, 3))

    sparse = B.Sparse(6, 1, 1)
    work, info = B.pkv_plan_work_sparse(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=1, max_blocks_per_slot=20,
                                        block_size=bs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, sparse=sparse)
    sel = torch.empty(1, hkv, 6, dtype=torch.int32, device="cuda")
    ws, out = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda"), torch.empty_like(q)
    meta = [dev(a) for a in (low.cu_seqlens_q, low.seq_slot, low.context_lens, pool.block_tables())]
    B.pkv_select_blocks(q, *meta, bounds, dev(work), info, sel, ws, sparse=sparse, block_size=bs, device_status=status)
    B.pkv_attention_sparse(q, *meta, *kv, sel, dev(work), info, out, ws, sparse=sparse, device_status=status)
    assert B.pkv_check_device_status(status) == 0
    vals = v[list(range(hist)) + [hist + p for p in path] + [hist + n]].double().cpu().numpy()
    q64, g = q.double().cpu().numpy(), hq // hkv
    for h in range(hkv):
        places = OB.choose(q64[:, h * g:(h + 1) * g], want[:, 0, h], want[:, 1, h], len(keys), bs, 6, 1, 1)
        assert sel[0, h].tolist() == places
        seen = np.isin(np.arange(len(keys)) // bs, places)[None]
        o, tol = OB.attention(q64[:, h * g:(h + 1) * g], keys[:, h:h + 1], vals[:, h:h + 1], seen, d ** -0.5)
        assert (np.abs(out[:, h * g:(h + 1) * g].double().cpu().numpy() - o) <= tol).all()


def test_two_streams_at_once():
    """Trees on one stream and a block-sparse step on another, each with a workspace of its own."""
    w = W.random_step(14, [(16, 6000), (40, 3000)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    w1 = W.random_step(15, [(1, 9000), (2, 5000)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds, d1 = R.prepare(w), R.prepare(w1)
    for s in (ds, d1):
        R.run_cache_write(s)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [16, 40]), ds.lowered.cu_seqlens_q)
    tree, _ = _call(ds, masks)
    low, sparse = d1.lowered, B.Sparse(64)
    work, info = B.pkv_plan_work_sparse(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=w1.max_slots,
                                        max_blocks_per_slot=w1.max_blocks_per_slot, block_size=16, num_q_heads=32,
                                        num_kv_heads=8, head_dim=128, sparse=sparse)
    bounds = torch.randn(w1.num_blocks, 8, 2, 128, device="cuda").sort(2).values.bfloat16()
    sel = torch.empty(2, 8, 64, dtype=torch.int32, device="cuda")
    ws, work = torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda"), torch.from_numpy(work).cuda()
    meta = (d1.cu_seqlens_q, d1.seq_slot, d1.context_lens, d1.block_tables)

    def choose_and_attend():
        B.pkv_select_blocks(d1.q, *meta, bounds, work, info, sel, ws, sparse=sparse, block_size=16, device_status=d1.status)
        B.pkv_attention_sparse(d1.q, *meta, d1.k_pool, d1.v_pool, sel, work, info, d1.out, ws, sparse=sparse,
                               device_status=d1.status)

    tree()
    choose_and_attend()
    torch.cuda.synchronize()
    want = [t.clone() for t in (ds.out, sel, d1.out)]
    ds.out.fill_(9.0)
    d1.out.fill_(9.0)
    sel.fill_(0)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(a):
            tree()
        with torch.cuda.stream(b):
            choose_and_attend()
    torch.cuda.synchronize()
    for got, t in zip((ds.out, sel, d1.out), want):
        assert torch.equal(got, t)
    assert B.pkv_check_device_status(ds.status) == 0 and B.pkv_check_device_status(d1.status) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("slots", [1, 40])
def test_keys_and_queries_that_are_not_numbers_reach_the_rows_that_see_them(slots, d):
    """NaN exactly in the rows that see a NaN key or hold a NaN query, in one span and in several (a lone slot has
    more); zeros in rows that see nothing, whatever their query; every other row as without them."""
    rng = np.random.default_rng(d + slots)
    shapes = [(9, 2500)] if slots == 1 else [(20, 20), (12, 3000), (40, 40), (256, 300), (1, 1)]
    w = W.random_step(60 + slots, shapes, num_q_heads=8, num_kv_heads=2, head_dim=d, max_slots=slots)
    sizes = [n for n, _ in shapes]
    cu = np.concatenate([[0], np.cumsum(sizes)])
    masks, _ = B.pkv_tree_masks(_parents(rng, sizes, "forest"), cu.astype(np.int32))
    masks[rng.random(w.total_q) < 0.2] = 0  # rows that see the history alone, or nothing
    q = W.bf16_bits_to_f32(w.q)
    bad_q = rng.random(q.shape[:2]) < 0.1
    clean = w.q.copy()
    q[bad_q] = np.nan
    w.q = W.f32_to_bf16_bits(q)
    expect_nan = np.zeros(q.shape[:2], bool)
    for i, (s, a) in enumerate(zip(w.segments, cu)):
        seen = np.concatenate([np.ones((s.q_len, s.ctx - s.q_len), bool), _bits(masks[a:a + s.q_len], s.q_len)], 1)
        # NaN in one channel of some of the step's own keys
        bad_k = np.zeros((s.ctx, 2), bool)
        bad_k[s.ctx - s.q_len:] = rng.random((s.q_len, 2)) < 0.15
        k = W.bf16_bits_to_f32(w.hist_k[s.slot])
        k[: s.ctx][bad_k, 5] = np.nan
        w.hist_k[s.slot][...] = W.f32_to_bf16_bits(k)
        reach = (seen.astype(int) @ bad_k.astype(int)) > 0  # [rows, kv heads]
        expect_nan[a:a + s.q_len] = np.repeat(reach, 4, 1) | (bad_q[a:a + s.q_len] & seen.any(1)[:, None])
    ds = R.prepare(w)
    R.run_cache_write(ds)
    call, info = _call(ds, masks)
    assert info.num_combine_items > 0
    call()
    assert B.pkv_check_device_status(ds.status) == 0
    got = R.out_f32(ds)
    assert np.array_equal(np.isnan(got), np.repeat(expect_nan[..., None], d, 2))
    w.q = clean
    for slot in w.hist_k:  # no row compared below sees these
        w.hist_k[slot][...] = W.f32_to_bf16_bits(np.nan_to_num(W.bf16_bits_to_f32(w.hist_k[slot])))
    want, tol = _expect(w, masks)
    rows = ~expect_nan & ~bad_q
    assert expect_nan.any() and rows.any() and (np.abs(got - want) <= tol)[rows].all()
    assert (got[bad_q & ~expect_nan] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_a_key_that_is_not_a_number_in_the_history_reaches_every_row(d):
    """Alone in its span, at the end of one and in the middle of another."""
    for at in (0, 255, 1100):
        w = W.random_step(70, [(5, 1200), (3, 1200)], num_q_heads=4, num_kv_heads=2, head_dim=d)
        k = W.bf16_bits_to_f32(w.hist_k[0])
        k[at, 1] = np.nan
        w.hist_k[0][...] = W.f32_to_bf16_bits(k)
        ds = R.prepare(w)
        R.run_cache_write(ds)
        masks, _ = B.pkv_tree_masks(_parents(None, [5, 3], "star"), ds.lowered.cu_seqlens_q)
        _call(ds, masks)[0]()
        nan = np.isnan(R.out_f32(ds))
        assert nan[:5, 2:].all() and not nan[:5, :2].any() and not nan[5:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_chunks_modified_chunks_and_trees_one_behind_another(d):
    """Kernels of different shares of tensor memory start under one another's ends: small grids, no call in between."""
    w = W.random_step(80, [(100, 700), (33, 2000), (256, 256)], num_q_heads=8, num_kv_heads=2, head_dim=d)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    low, meta = ds.lowered, (ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, ds.k_pool, ds.v_pool)
    shape = dict(max_slots=w.max_slots, max_blocks_per_slot=w.max_blocks_per_slot, block_size=16, num_q_heads=8, num_kv_heads=2,
                 head_dim=d)
    work, info = B.pkv_plan_work_mod(low.cu_seqlens_q, low.seq_slot, low.context_lens, window=300, **shape)
    work = torch.from_numpy(work).cuda()
    ws = torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(ds.out) for _ in range(3)]
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [100, 33, 256]), low.cu_seqlens_q)
    tree, _ = _call(ds, masks, out=outs[2])

    def plain():
        B.pkv_attention(ds.q, *meta, ds.work, ds.info, outs[0], ds.workspace, scale=ds.scale, device_status=ds.status)

    def modified():
        B.pkv_attention_mod(ds.q, *meta, work, info, outs[1], ws, mod=B.ScoreMod(window=300), scale=ds.scale,
                            device_status=ds.status)

    calls = (plain, modified, tree)
    for call in calls:
        call()
        torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    for order in ((0, 1, 2), (1, 0, 2), (0, 2, 1), (2, 0, 0, 1, 1, 2, 2)):
        for o in outs:
            o.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(5):
            for i in order:
                calls[i]()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), order
    assert B.pkv_check_device_status(ds.status) == 0


@pytest.mark.parametrize("d", [64, 128])
def test_trees_beside_idle_slots(d):
    """Few live slots of many: longer spans, the same attention."""
    shapes = [(8, 8200), (64, 9000), (1, 30), (33, 2000)]
    w = W.random_step(90, shapes, num_q_heads=8, num_kv_heads=2, head_dim=d, max_slots=64, slots=[63, 0, 31, 8])
    ds = R.prepare(w)
    R.run_cache_write(ds)
    masks, _ = B.pkv_tree_masks(_parents(np.random.default_rng(0), [n for n, _ in shapes]), ds.lowered.cu_seqlens_q)
    _call(ds, masks)[0]()
    assert B.pkv_check_device_status(ds.status) == 0
    _check(ds, masks, f"idle {d}")
