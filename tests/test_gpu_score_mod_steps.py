"""Modified scores among their neighbours: other segments of the step, other calls on the stream, other lists."""

import numpy as np
import pytest

import oracle
from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild
from continuous_batching_paged_pkv_gb300 import runtime as R
from continuous_batching_paged_pkv_gb300 import workloads as W
from tests import test_gpu_score_mod as score_mod

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    libbuild.build()
    oracle.build()


def _slopes(hq):
    return 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)


def _run(w, mod, kv="bf16"):
    ds = R.prepare(w, kv=kv, mod=mod)
    R.run_step(ds)
    torch.cuda.synchronize()
    assert B.pkv_check_device_status(ds.status) == 0
    return R.out_f32(ds), ds


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("rows", [509, 203, 33])
def test_a_capped_chunk_does_not_depend_on_the_rows_behind_it(rows, biased, d):
    """A chunk whose last warp is partly filled: the same bits alone, before another chunk whose queries lie far beyond
    the cap (their rows are in the chunk's last query tile), and before such decode rows."""
    heads = dict(num_q_heads=32, num_kv_heads=8, head_dim=d)
    mod = B.ScoreMod(softcap=50.0, alibi_slopes=_slopes(32) if biased else None)
    first = W.random_step(31, [(rows, rows + 700)], max_slots=4, **heads)
    want, _ = _run(first, mod)
    for behind in ([(40, 90)], [(1, 700), (1, 64)], [(64, 64), (1, 300), (1, 41)]):
        w = W.random_step(32, [(rows, rows + 700)] + behind, max_slots=4, **heads)
        w.hist_k[0], w.hist_v[0] = first.hist_k[0], first.hist_v[0]
        q = 30.0 * W.bf16_bits_to_f32(w.q)
        q[:rows] = W.bf16_bits_to_f32(first.q)
        w.q = W.f32_to_bf16_bits(q)
        got, _ = _run(w, mod)
        differ = (got[:rows] != want).any((1, 2)).nonzero()[0]
        assert not len(differ), f"behind it {behind}: rows {differ} differ"


@pytest.mark.parametrize("modified", [False, True])
@pytest.mark.parametrize("kv,heads", [("q8", (32, 8, 128)), ("q4", (32, 8, 128)), ("q8", (8, 8, 64))])
def test_a_widened_history_does_not_depend_on_what_the_workspace_held(heads, modified, kv):
    """Prompt chunks over a block-scaled pool read a scratch pool through a scratch block table that the kernel before
    fills: the same bits whatever an earlier call left there, called one behind another and replayed."""
    hq, hkv, d = heads
    w = W.random_step(43, [(40, 1500), (90, 600), (33, 2100), (200, 200), (1, 700)], num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    mod = B.ScoreMod(window=900) if modified else None
    want, ds = _run(w, mod, kv)
    graph = torch.cuda.CUDAGraph()
    fills = (0, 255, 1)
    got = torch.empty((2 * len(fills),) + tuple(ds.out.shape), dtype=ds.out.dtype, device="cuda")

    def calls(at):
        for i, fill in enumerate(fills):
            ds.workspace.fill_(fill)
            R.run_attention(ds)
            got[at + i].copy_(ds.out)

    calls(0)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        calls(len(fills))
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert B.pkv_check_device_status(ds.status) == 0
    assert all(np.array_equal(o.float().cpu().numpy(), want) for o in got)


@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("heads", [(32, 8, 128), (8, 8, 64)])
@pytest.mark.parametrize("shapes", [[(1, 2500), (1, 900), (1, 40)], [(2, 2500), (1, 130)], [(300, 2300), (40, 90)],
                                    [(200, 1800), (1, 1200), (1, 60)]])
def test_rows_that_see_no_new_key_keep_the_order_of_calls(shapes, heads, kv):
    """Calls whose rows see only cached keys, or none, between calls and appends that write the same output and pool,
    on one stream without a host wait: the same bits as with one."""
    hq, hkv, d = heads
    w = W.random_step(41, shapes, num_q_heads=hq, num_kv_heads=hkv, head_dim=d)
    first = np.concatenate([np.full(s.q_len, s.ctx - s.q_len) for s in w.segments])
    mods = [B.ScoreMod(window=700), B.ScoreMod(key_end=first // 3), B.ScoreMod(key_end=np.zeros_like(first)),
            B.ScoreMod(key_end=first)]
    steps = [R.prepare(w, kv=kv, mod=m) for m in mods]
    base = steps[0]
    room = torch.empty(max([1] + [int(max(s.info.workspace_bytes_q8, s.info.workspace_bytes)) for s in steps]),
                       dtype=torch.uint8, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    news = [tuple(torch.randn(base.k_new.shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
            for _ in range(2)]
    for s in steps[1:]:
        s.k_pool, s.v_pool, s.k_scales, s.v_scales, s.out, s.status = (base.k_pool, base.v_pool, base.k_scales,
                                                                       base.v_scales, base.out, base.status)
    for s in steps:
        s.workspace = room

    def run(s, new, wait):
        if new is not None:
            s.k_new, s.v_new = news[new]
            R.run_cache_write(s)
        if wait:
            torch.cuda.synchronize()
        R.run_attention(s)
        if wait:
            torch.cuda.synchronize()

    # (step, which rows it appends first, whether its output is looked at)
    chain = [(0, 0, False), (2, None, True), (1, None, False), (0, None, True), (1, 1, False), (0, 0, True), (0, None, False),
             (1, None, True), (3, 1, False), (2, 0, False), (0, 1, True), (3, None, False), (2, None, True)]
    rounds = 6

    def outputs(wait, seen):
        base.out.fill_(3.0)
        for _ in range(rounds):
            for i, new, keep in chain:
                run(steps[i], new, wait)
                if keep:
                    seen.append(base.out.clone())
        return seen

    want, got, graph, replayed = outputs(True, []), outputs(False, []), torch.cuda.CUDAGraph(), []
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        outputs(False, replayed)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert (want[0] == 0).all() and B.pkv_check_device_status(base.status) == 0
    for i, (a, b, c) in enumerate(zip(want, got, replayed)):
        assert torch.equal(a, b) and torch.equal(a, c), f"output {i}"


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("q8", 64), ("q8", 128)])
@pytest.mark.parametrize("modified", [False, True])
def test_chunk_items_outside_the_segment_are_reported_not_followed(modified, kv, d):
    """Query tiles past the segment's rows, also those whose first row leaves 32 bits, and wrong segments and slots."""
    w = W.random_step(5, [(150, 400), (40, 90)], num_q_heads=8, num_kv_heads=2, head_dim=d)
    mod = B.ScoreMod(window=90, key_begin=np.zeros(190, np.int64), alibi_slopes=_slopes(8)) if modified else None
    want, ds = _run(w, mod, kv)
    good = ds.work.clone()
    at = 4 * ds.info.num_decode_items
    tiles = 32  # rows of a tile: 128 / group
    assert good[at] == 0 and good[at + 2] % 2 == 0
    for word, value in ((2, 5), (2, 6), (2, 2 ** 31 - 1), (2, 2 ** 31 // tiles), (2, 2 ** 32 // tiles), (2, 2 ** 32 // tiles + 2),
                        (2, 3 * 2 ** 31 // tiles), (2, -2), (0, 2), (0, -1), (0, 1), (1, 1), (1, 2 ** 31 - 1), (1, -1)):
        bad = good.clone()
        bad[at + word] = value
        ds.work.copy_(bad)
        R.run_attention(ds)
        assert B.pkv_check_device_status(ds.status) & 4, (word, value)
    ds.work.copy_(good)
    ds.out.zero_()
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) == 0
    assert np.array_equal(R.out_f32(ds), want)


@pytest.mark.parametrize("kv,d", [("q8", 64), ("q8", 128), ("q4", 128)])
def test_chunk_bounds_wider_than_the_widened_history_are_reported(kv, d):
    """Also where an earlier call has left block IDs of the scratch pool in the workspace's block table."""
    w = W.random_step(6, [(60, 900), (33, 700)], num_q_heads=8, num_kv_heads=2, head_dim=d)
    _, whole = _run(w, B.ScoreMod(), kv)
    want, ds = _run(w, B.ScoreMod(key_begin=np.full(93, 640)), kv)
    narrow = ds.mod.key_begin.clone()
    for at, begin in ((slice(0, 60), 100), (slice(0, 1), 0), (slice(60, 93), 500)):
        for fill in (0, None):
            whole.workspace.fill_(0)
            if fill is None:
                R.run_attention(whole)
            ds.workspace = whole.workspace
            ds.mod.key_begin.copy_(narrow)
            ds.mod.key_begin[at] = begin
            R.run_attention(ds)
            assert B.pkv_check_device_status(ds.status) & 2, (at, begin, fill)
            assert B.pkv_check_device_status(whole.status) == 0
    ds.mod.key_begin.copy_(narrow)
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) == 0
    assert np.array_equal(R.out_f32(ds), want)


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("q8", 64), ("q4", 128)])
def test_rows_with_a_gap_between_their_keys(kv, d):
    """A run and a chunk whose rows' intervals leave a gap: right results, whatever finite values lie in the gap, and
    with NaN and blocks outside the pool before the first and behind the last key that a row sees."""
    w = W.random_step(7, [(2, 1500), (60, 2500)], num_q_heads=8, num_kv_heads=2, head_dim=d)
    low = np.arange(60) < 30
    mod = B.ScoreMod(key_begin=np.concatenate([[33, 1000], np.where(low, 100, 2000)]),
                     key_end=np.concatenate([[100, 1100], np.where(low, 150, 2050)]))
    want, ds = _run(w, mod, kv)
    score_mod.check(want, w, kv, mod, "a gap")
    tables, arrays = ds.block_tables, [t for t in (ds.k_pool, ds.v_pool, ds.k_scales, ds.v_scales) if t is not None]
    for slot, first, gap, last in ((0, 33, (100, 1000), 1100), (1, 100, (150, 2000), 2050)):
        inside = tables[slot, -(-gap[0] // 16):gap[1] // 16].long()
        for t in arrays:
            t[inside] = 7 if t.dtype != torch.bfloat16 else 1e30 if kv == "bf16" else 0.25
        dead = [*range(0, first // 16), *range(-(-last // 16), tables.shape[1])]
        for t in (arrays if kv == "bf16" else arrays[2:]):
            t[tables[slot, first // 16].long(), :, :first % 16] = float("nan")
            if last % 16:
                t[tables[slot, last // 16].long(), :, last % 16:] = float("nan")
        tables[slot, dead] = torch.tensor([-1, 1 << 30] * len(dead), dtype=torch.int32, device="cuda")[:len(dead)]
    ds.out.fill_(float("nan"))
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) == 0
    got = R.out_f32(ds)
    score_mod.check(got, w, kv, mod, "other keys in the gap")
    # (decode over codes scales its weights by the largest value scale that it has loaded)
    rows = slice(None) if kv == "bf16" else slice(2, None)
    assert np.array_equal(got[rows], want[rows])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("shapes", [[(1, 60), (1, 900)], [(2, 50), (2, 1300)], [(150, 700)]])
def test_a_row_whose_logits_are_all_minus_infinity(shapes, d):
    """0 / 0 by the definition, in every path alike; zeros are for rows that see no key."""
    w = W.random_step(9, shapes, num_q_heads=8, num_kv_heads=2, head_dim=d)
    q = W.bf16_bits_to_f32(w.q).copy()
    q[..., 0] = 1.0
    w.q = W.f32_to_bf16_bits(q)
    pos = np.concatenate([np.arange(s.ctx - s.q_len, s.ctx) for s in w.segments])
    end = np.where(pos % 2 == 0, 0, pos + 1)
    for mod in (None, B.ScoreMod(), B.ScoreMod(window=40), B.ScoreMod(alibi_slopes=_slopes(8)), B.ScoreMod(key_end=end),
                B.ScoreMod(key_end=end, softcap=5.0)):
        _, ds = _run(w, mod)
        ds.k_pool[:, 0, :, 0] = float("-inf")
        R.run_attention(ds)
        got = R.out_f32(ds)
        assert B.pkv_check_device_status(ds.status) == 0
        blind = mod is not None and mod.key_end is not None and end == 0
        if mod is None or not mod.softcap:
            assert np.array_equal(np.isnan(got[:, :4]), np.broadcast_to(~np.atleast_1d(blind)[:, None, None], got[:, :4].shape)), mod
        else:
            assert np.isfinite(got).all()
        assert np.isfinite(got[:, 4:]).all() and (got[np.broadcast_to(blind, len(pos))] == 0).all(), mod
