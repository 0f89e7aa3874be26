"""Attention with modified scores on the GPU against ``oracle.scoremod`` (float64), element by element within the
tolerance that the oracle derives beside the result."""

import zlib

import numpy as np
import pytest

import oracle
from oracle import kvquant as KQ
from oracle import scoremod as SM
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


def _slopes(hq):
    return 2.0 ** (-8.0 * np.arange(1, hq + 1) / hq)


def make_mod(kind, w, seed):
    """Modification `kind` for the step w."""
    rng = np.random.default_rng(seed)
    pos = np.concatenate([np.arange(s.ctx - s.q_len, s.ctx) for s in w.segments])
    ctx = np.concatenate([np.full(s.q_len, s.ctx) for s in w.segments])
    hq = w.num_q_heads
    if kind == "none":
        return B.ScoreMod()
    if kind == "cap":
        return B.ScoreMod(softcap=5.0)
    if kind.startswith("window"):
        return B.ScoreMod(window=int(kind[6:]))
    if kind == "alibi":
        return B.ScoreMod(alibi_slopes=_slopes(hq))
    if kind == "documents":
        return B.ScoreMod(key_begin=pos - pos % 37)
    if kind == "prefix":
        return B.ScoreMod(key_end=np.maximum(pos + 1, ctx * 2 // 3), softcap=20.0)
    if kind == "padding":
        end = pos + 1
        end[rng.random(len(pos)) < 0.4] = 0
        return B.ScoreMod(key_end=end, alibi_slopes=_slopes(hq))
    if kind == "nothing":
        return B.ScoreMod(key_begin=ctx, key_end=np.zeros_like(pos))
    if kind == "around":  # biases to both sides of a row, steep, flat and growing
        return B.ScoreMod(alibi_slopes=_slopes(hq) * rng.choice([-0.05, 0.1, 1.0, 4.0], hq),
                          key_begin=np.where(rng.random(len(pos)) < 0.5, 0, rng.integers(0, ctx)),
                          key_end=np.where(rng.random(len(pos)) < 0.3, pos + 1, rng.integers(1, ctx + 3)))
    if kind == "everything":
        begin = rng.integers(-3, ctx + 3)
        begin[rng.random(len(pos)) < 0.5] = 0
        return B.ScoreMod(softcap=3.0, window=211, alibi_slopes=_slopes(hq) * rng.choice([-0.01, 1.0], hq),
                          key_begin=begin, key_end=rng.integers(-3, ctx + 40))
    raise KeyError(kind)


def _histories(w, kv):
    """Per slot (k, v, magnitudes for the tolerance) as the pool holds them."""
    out = {}
    for s in w.segments:
        one = []
        for h in (w.hist_k[s.slot], w.hist_v[s.slot]):
            if kv == "bf16":
                one.append((W.bf16_bits_to_f32(h).astype(np.float64), None))
            else:
                codes, scales = KQ.quantize(h, int(kv[1]))
                val = KQ.dequantize(codes, scales)
                d = np.repeat(W.bf16_bits_to_f32(scales).astype(np.float64), 32, -1)
                one.append((val, (np.abs(codes.astype(np.float64)) + 1152) * d))
        out[s.slot] = one
    return out


def expect(w, kv, mod):
    hist, outs, tols, row = _histories(w, kv), [], [], 0
    q = W.bf16_bits_to_f32(w.q).astype(np.float64)
    for s in w.segments:
        rows = slice(row, row + s.q_len)
        row += s.q_len
        pos = np.arange(s.ctx - s.q_len, s.ctx)
        lo, hi = SM.bounds(pos, s.ctx, window=mod.window, key_begin=None if mod.key_begin is None else mod.key_begin[rows],
                           key_end=None if mod.key_end is None else mod.key_end[rows])
        (k, km), (v, vm) = hist[s.slot]
        o, t = SM.attention(q[rows], k, v, pos, lo, hi, w.scale, softcap=mod.softcap, slopes=mod.alibi_slopes, k_mag=km,
                            v_mag=vm)
        outs.append(o)
        tols.append(t)
    return np.concatenate(outs), np.concatenate(tols)


def check(got, w, kv, mod, what):
    want, tol = expect(w, kv, mod)
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), (f"{what}: {off.max():.3e} beyond the tolerance at "
                              f"{np.unravel_index(off.argmax(), off.shape)}, {(off > 0).mean():.2%} of the values")


def run(w, kv, mod):
    ds = R.prepare(w, kv=kv, mod=mod)
    R.run_step(ds)
    torch.cuda.synchronize()
    assert B.pkv_check_device_status(ds.status) == 0
    return R.out_f32(ds), ds


SHAPES = {
    "decode": [(1, 1), (1, 17), (1, 256), (1, 257), (1, 513), (1, 1300)],
    "runs": [(2, 257), (3, 259), (2, 2), (4, 4), (2, 700)],
    "chunk": [(130, 300)],
    "chunks": [(33, 100), (7, 7), (200, 200), (300, 1111)],
    "mixed": [(40, 333), (1, 700), (1, 64), (17, 17), (2, 300)],
}
KINDS = ["none", "cap", "window1", "window5", "window100", "window400", "alibi", "documents", "prefix", "padding", "nothing",
         "around", "everything"]
HEADS = [(4, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (6, 6, 128), (16, 1, 64)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", sorted(SHAPES))
def test_shapes(case, kind):
    for i, (hq, hkv, d) in enumerate(HEADS):
        seed = zlib.crc32(f"{case}/{kind}/{i}".encode()) % 1000
        w = W.random_step(seed, SHAPES[case], num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=[16, 32, 64][i % 3])
        mod = make_mod(kind, w, seed)
        got, _ = run(w, "bf16", mod)
        check(got, w, "bf16", mod, f"{hq}/{hkv}/{d}")


@pytest.mark.parametrize("kv", ["q8", "q4"])
@pytest.mark.parametrize("kind", ["cap", "window100", "alibi", "documents", "padding", "nothing", "around", "everything"])
def test_quantised_pools(kind, kv):
    for i, (hq, hkv, d) in enumerate([(32, 8, 128), (40, 8, 128), (16, 1, 128)] + ([(4, 2, 64), (8, 8, 64)] if kv == "q8" else [])):
        for case in ("decode", "runs", "mixed"):
            seed = zlib.crc32(f"{case}/{kind}/{i}/{kv}".encode()) % 1000
            w = W.random_step(seed, SHAPES[case], num_q_heads=hq, num_kv_heads=hkv, head_dim=d,
                              block_size=[16, 32, 64][(i + 1) % 3])
            mod = make_mod(kind, w, seed)
            got, _ = run(w, kv, mod)
            check(got, w, kv, mod, f"{case} {hq}/{hkv}/{d}")


@pytest.mark.parametrize("kind", ["cap", "everything", "alibi"])
def test_peaked_scores(kind):
    """Queries eight times as large: logits far beyond the cap, weights near one."""
    w = W.random_step(6, [(1, 900), (64, 700), (2, 300)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    w.q = W.f32_to_bf16_bits(W.bf16_bits_to_f32(w.q) * 8.0)
    mod = make_mod(kind, w, 6)
    for kv in ("bf16", "q8"):
        got, _ = run(w, kv, mod)
        check(got, w, kv, mod, kv)


@pytest.mark.parametrize("sign", [-1.0, 1.0])
def test_scores_all_far_below_zero(sign):
    """Every logit near -200 or 200 times a head's slope: the softmax is relative to the row's own largest."""
    w = W.random_step(8, [(1, 600), (40, 400)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    rng = np.random.default_rng(0)
    for slot in w.hist_k:
        k = W.bf16_bits_to_f32(w.hist_k[slot])
        k[..., 0] = 40.0 * sign
        w.hist_k[slot][...] = W.f32_to_bf16_bits(k + 0.0 * rng.random())
    q = W.bf16_bits_to_f32(w.q)
    q[..., 0] = -40.0
    w.q = W.f32_to_bf16_bits(q)
    for mod in (B.ScoreMod(), B.ScoreMod(alibi_slopes=np.full(8, 0.4)), B.ScoreMod(window=90), B.ScoreMod(softcap=300.0)):
        got, _ = run(w, "bf16", mod)
        check(got, w, "bf16", mod, str(mod))


@pytest.mark.parametrize("cap", [2.0 ** -20, 0.01, 700.0, 4096.0])
def test_caps_from_the_least_to_the_largest(cap):
    for d in (64, 128):
        w = W.random_step(12, SHAPES["mixed"], num_q_heads=8, num_kv_heads=2, head_dim=d)
        for mod in (B.ScoreMod(softcap=cap), B.ScoreMod(softcap=cap, alibi_slopes=_slopes(8), window=150)):
            got, _ = run(w, "bf16", mod)
            check(got, w, "bf16", mod, str(mod))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_keys_that_nobody_sees_are_not_read(kv, d):
    """Blocks before the rows' windows are given back (entries -1) and the rest of the unseen rows hold NaN."""
    bs = 16
    segs = [(1, 777), (3, 500), (50, 600)]
    w = W.random_step(3, segs, num_q_heads=8, num_kv_heads=4, head_dim=d, block_size=bs)
    mod = B.ScoreMod(window=70)
    want, ds = run(w, kv, mod)
    tables = ds.block_tables
    scales = ds.k_pool if kv == "bf16" else ds.k_scales
    vscales = ds.v_pool if kv == "bf16" else ds.v_scales
    for s in w.segments:
        lo = s.ctx - s.q_len - 70 + 1
        dead = lo // bs
        ids = tables[s.slot, :dead].long()
        for t in (scales, vscales):
            t[ids] = float("nan")
            t[tables[s.slot, dead], :, :lo % bs] = float("nan")
        tables[s.slot, :dead] = torch.tensor([-1, 1 << 30] * dead, dtype=torch.int32, device="cuda")[:dead]
        end = s.ctx % bs
        if end:
            for t in (scales, vscales):
                t[tables[s.slot, s.ctx // bs], :, end:] = float("nan")
    ds.out.fill_(float("nan"))
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) == 0
    assert np.array_equal(R.out_f32(ds), want)


def test_unseen_keys_may_hold_nan():
    """Keys (not values) that are not finite reach only the rows that see them, also inside a tile."""
    w = W.random_step(5, [(1, 300), (60, 290)], num_q_heads=8, num_kv_heads=4, head_dim=128)
    mod = B.ScoreMod(key_begin=np.concatenate([[130], np.where(np.arange(60) < 30, 0, 240)]))
    want, ds = run(w, "bf16", mod)
    bt = ds.block_tables
    ds.k_pool[bt[0, 129 // 16], :, 129 % 16] = float("nan")
    ds.k_pool[bt[1, 5], :, 3] = float("inf")
    R.run_attention(ds)
    got = R.out_f32(ds)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[31:], want[31:])


def test_results_do_not_depend_on_the_batch():
    """A row in a batch and alone, on other blocks (the tables' shape is the same): the same bits."""
    heads = dict(num_q_heads=32, num_kv_heads=8, head_dim=128)
    segs = [(1, 1500), (200, 900), (2, 640), (1, 3000)]
    w = W.random_step(11, segs, **heads)
    mod = lambda n: B.ScoreMod(softcap=20.0, window=600, alibi_slopes=_slopes(32) / 4)  # noqa: E731
    whole, _ = run(w, "bf16", mod(0))
    row = 0
    for i, s in enumerate(w.segments):
        alone = W.random_step(50 + i, [(s.q_len, s.ctx)], max_slots=4, **heads)
        alone.hist_k[0], alone.hist_v[0] = w.hist_k[s.slot], w.hist_v[s.slot]
        alone.q = w.q[row:row + s.q_len]
        got, _ = run(alone, "bf16", mod(0))
        assert np.array_equal(got, whole[row:row + s.q_len]), f"segment {i}"
        row += s.q_len


def test_streams_graphs_and_shared_workspaces():
    """Bound calls on another stream, and two captured steps that share one workspace, replayed in turn."""
    heads = dict(num_q_heads=40, num_kv_heads=8, head_dim=128)
    steps = []
    for seed, kind in ((1, "cap"), (2, "everything")):
        w = W.random_step(seed, [(1, 2000), (64, 500), (3, 777)], **heads)
        mod = make_mod(kind, w, seed)
        want, ds = run(w, "bf16", mod)
        steps.append((w, mod, want, ds))
    room = torch.empty(max(int(s[3].info.workspace_bytes) for s in steps), dtype=torch.uint8, device="cuda")
    calls = [B.AttentionModCall(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables,
                                (ds.k_pool, ds.v_pool), ds.work, ds.info, ds.out, room, mod=ds.mod, scale=ds.scale,
                                device_status=ds.status) for _, _, _, ds in steps]
    side = torch.cuda.Stream()
    for (_, _, want, ds), call in zip(steps, calls):
        ds.out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert np.array_equal(R.out_f32(ds), want)
    graphs = []
    for call in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    for _ in range(3):
        for (_, _, want, ds), g in zip(steps, graphs):
            ds.out.zero_()
            g.replay()
    torch.cuda.synchronize()
    for _, _, want, ds in steps:
        assert np.array_equal(R.out_f32(ds), want)
        assert B.pkv_check_device_status(ds.status) == 0


def test_rows_beyond_the_output_are_left():
    w = W.random_step(4, [(1, 300), (20, 90)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    mod = make_mod("cap", w, 0)
    want, ds = run(w, "bf16", mod)
    big = torch.full((30, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    B.pkv_attention_mod(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, ds.k_pool, ds.v_pool, ds.work,
                        ds.info, big[4:25], ds.workspace, mod=ds.mod, scale=ds.scale)
    assert np.array_equal(big[4:25].float().cpu().numpy(), want)
    assert (big[:4] == 7).all() and (big[25:] == 7).all()


def test_bad_blocks_are_reported():
    w = W.random_step(4, [(1, 300), (20, 90)], num_q_heads=8, num_kv_heads=2, head_dim=128)
    _, ds = run(w, "bf16", make_mod("cap", w, 0))
    ds.block_tables[0, 3] = w.num_blocks
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) & 2
    ds.block_tables[0, 3] = -7
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) & 2


def test_a_list_of_another_step_is_reported_not_followed():
    """Items that name partials past the workspace, or spans past the context, are skipped and set the status."""
    heads = dict(num_q_heads=8, num_kv_heads=2, head_dim=128)
    w = W.random_step(4, [(1, 900), (2, 600)], **heads)
    _, ds = run(w, "bf16", make_mod("cap", w, 0))
    good = ds.work.clone()
    nd, nc = ds.info.num_decode_items, ds.info.num_combine_items
    for at, word in ((3, ds.info.num_partials), (3, 2 ** 31 - 1), (2, 0x7FFFFF | 16 << 27), (2, 17 << 27), (2, 31 << 27),
                     (0, 2), (1, 5), (nd * 4 + 3, ds.info.num_partials - 2), (nd * 4 + 2, 65535), (nd * 4 + 2, 0)):
        assert nc > 0
        bad = good.clone()
        bad[at] = word if word < 2 ** 31 else word - 2 ** 32
        ds.work.copy_(bad)
        R.run_attention(ds)
        assert B.pkv_check_device_status(ds.status) & 4, (at, word)
    ds.work.copy_(good)
    ds.out.zero_()
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) == 0
    check(R.out_f32(ds), w, "bf16", make_mod("cap", w, 0), "after the bad lists")


def test_bounds_wider_than_the_plan_are_reported():
    w = W.random_step(4, [(1, 900), (1, 300)], num_q_heads=8, num_kv_heads=2, head_dim=128)
    mod = B.ScoreMod(key_begin=np.array([700, 280]))
    _, ds = run(w, "bf16", mod)
    ds.mod.key_begin.copy_(torch.tensor([700, 100], dtype=torch.int32))
    R.run_attention(ds)
    assert B.pkv_check_device_status(ds.status) & 4


def test_pools_past_2_31_elements():
    """Rotation, append and windowed attention in the last blocks of pools of 2.2e9 elements each."""
    hq, hkv, d, bs, nb, n = 16, 8, 128, 16, 134300, 300
    kp = torch.empty(nb, hkv, bs, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    g = torch.Generator("cuda").manual_seed(1)
    q, k, v = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda", dtype=torch.bfloat16).split([hq, hkv, hkv], 1)
    pool = B.Pool(nb, bs, 2, 32, free_order=np.arange(nb - 40, nb, dtype=np.int32))
    assert pool.admit(1, n) == B.PKV_OK
    low = pool.lower([(1, n)])
    assert low.slot_mapping.max() * hkv * d > 2 ** 31
    plan = B.pkv_rope_plan(d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qr, out = torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda"), torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda")
    pos = R._i32(np.arange(n), "cuda")
    B.pkv_rope_cache_write(q, k, v, pos, plan.phase_tensor("cuda"), R._i64(low.slot_mapping, "cuda"), qr, kp, vp, rot_dim=d,
                           device_status=status)
    work, info = B.pkv_plan_work_mod(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=2, max_blocks_per_slot=32,
                                     block_size=bs, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, window=77)
    room = torch.empty(max(1, info.workspace_bytes), dtype=torch.uint8, device="cuda")
    B.pkv_attention_mod(qr, R._i32(low.cu_seqlens_q, "cuda"), R._i32(low.seq_slot, "cuda"), R._i32(low.context_lens, "cuda"),
                        R._i32(pool.block_tables(), "cuda"), kp, vp, R._i32(work, "cuda"), info, out, room,
                        mod=B.ScoreMod(window=77), device_status=status)
    assert B.pkv_check_device_status(status) == 0
    kr = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
    B.pkv_rope(k, pos, plan.phase_tensor("cuda"), kr, rot_dim=d)
    f = lambda t: t.float().cpu().numpy()  # noqa: E731
    p = np.arange(n)
    want, tol = SM.attention(f(qr), f(kr), f(v), p, *SM.bounds(p, n, window=77), d ** -0.5)
    assert (np.abs(f(out) - want) <= tol).all()


def test_arguments_are_checked():
    w = W.random_step(4, [(1, 300), (20, 90)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    _, ds = run(w, "bf16", make_mod("documents", w, 0))
    base = dict(mod=ds.mod, scale=ds.scale)
    args = [ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, (ds.k_pool, ds.v_pool), ds.work, ds.info,
            ds.out, ds.workspace]

    def refused(i=None, value=None, **kw):
        a = list(args)
        if i is not None:
            a[i] = value
        with pytest.raises((ValueError, B.PkvError)):
            B.AttentionModCall(*a, **(base | kw))()

    refused(0, ds.q.float())
    refused(0, ds.q.cpu())
    refused(8, ds.out[:5])
    refused(6, ds.work[:4])
    refused(3, ds.context_lens[:1])
    refused(5, (ds.k_pool, ds.v_pool[:3]))
    refused(kv="q8")
    refused(kv="fp8")
    for mod in (B.ScoreMod(softcap=-1.0), B.ScoreMod(softcap=4097.0), B.ScoreMod(softcap=1e-7), B.ScoreMod(window=-2), B.ScoreMod(alibi_slopes=torch.ones(7, device="cuda")),
                B.ScoreMod(alibi_slopes=torch.ones(8, dtype=torch.float64, device="cuda")),
                B.ScoreMod(key_begin=ds.mod.key_begin[:5]), B.ScoreMod(key_end=ds.mod.key_begin.long())):
        refused(mod=mod)
    _, ds = run(w, "bf16", make_mod("cap", w, 0))  # two spans: partials in the workspace
    with pytest.raises(B.PkvError):
        B.pkv_attention_mod(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, ds.k_pool, ds.v_pool,
                            ds.work, ds.info, ds.out, ds.workspace[:64], mod=ds.mod)


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_a_step_of_rotation_append_and_attention(kv):
    """Rotation, append and windowed, capped attention as a serving step runs them: two steps of one slot beside others."""
    hq, hkv, d, bs, hist = 16, 4, 64, 16, 500
    g = torch.Generator("cuda").manual_seed(3)
    plan = B.pkv_rope_plan(d, scaling=B.PKV_ROPE_LINEAR, factor=2.0)
    ph = plan.phase_tensor("cuda")
    pool = B.Pool(200, bs, 4, 60)
    arrays = R.empty_pool(200, hkv, bs, d, "cuda") if kv == "bf16" else R.empty_pool_q8(200, hkv, bs, d, "cuda")
    seen = {s: [] for s in range(3)}
    for s in range(3):
        assert pool.admit(s, hist + 40) == B.PKV_OK
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mod = B.ScoreMod(softcap=10.0, window=200)
    for plan_step in ([(0, 300), (1, 77), (2, 2)], [(1, 1), (0, 130), (2, 3)], [(2, 1), (0, 1), (1, 2)]):
        low = pool.lower(plan_step)
        n = int(low.cu_seqlens_q[-1])
        qkv = torch.randn(n, hq + 2 * hkv, d, generator=g, device="cuda", dtype=torch.bfloat16)
        q, k, v = qkv.split([hq, hkv, hkv], 1)
        pos = B.pkv_plan_positions(low.cu_seqlens_q, low.seq_slot, low.context_lens)
        work, info = B.pkv_plan_work_mod(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=4,
                                         max_blocks_per_slot=60, block_size=bs, num_q_heads=hq, num_kv_heads=hkv,
                                         head_dim=d, window=200)
        dpos, slots = R._i32(pos, "cuda"), R._i64(low.slot_mapping, "cuda")
        out, qr = (torch.empty(n, hq, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        room = torch.empty(max(1, info.workspace_bytes_q8), dtype=torch.uint8, device="cuda")
        meta = (R._i32(low.cu_seqlens_q, "cuda"), R._i32(low.seq_slot, "cuda"), R._i32(low.context_lens, "cuda"),
                R._i32(pool.block_tables(), "cuda"))
        dwork = R._i32(work, "cuda")
        kr = torch.empty(n, hkv, d, dtype=torch.bfloat16, device="cuda")
        if kv == "bf16":
            B.pkv_rope_cache_write(q, k, v, dpos, ph, slots, qr, *arrays, rot_dim=d, device_status=status)
            B.pkv_attention_mod(qr, *meta, *arrays, dwork, info, out, room, mod=mod, device_status=status)
        else:
            B.pkv_rope(q, dpos, ph, qr, rot_dim=d)
            B.pkv_rope(k, dpos, ph, kr, rot_dim=d)
            B.pkv_cache_write_q8(kr, v.contiguous(), slots, *arrays, device_status=status)
            B.pkv_attention_mod_q8(qr, *meta, *arrays, dwork, info, out, room, mod=mod, device_status=status)
        assert B.pkv_check_device_status(status) == 0
        B.pkv_rope(k, dpos, ph, kr, rot_dim=d)
        bits = lambda t: t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)  # noqa: E731
        kb, vb, qb = bits(kr), bits(v), bits(qr)
        for (s, m), a in zip(plan_step, low.cu_seqlens_q):
            rows = slice(int(a), int(a) + m)
            seen[s].append((kb[rows], vb[rows]))
            hk, hv = (np.concatenate([x[i] for x in seen[s]]) for i in (0, 1))
            mags = (None, None)
            if kv == "bf16":
                keys, vals = (W.bf16_bits_to_f32(x) for x in (hk, hv))
            else:
                (kc, ks), (vc, vs) = KQ.quantize(hk), KQ.quantize(hv)
                keys, vals = KQ.dequantize(kc, ks), KQ.dequantize(vc, vs)
                mags = tuple((np.abs(c.astype(np.float64)) + 1152) * np.repeat(W.bf16_bits_to_f32(x), 32, -1)
                             for c, x in ((kc, ks), (vc, vs)))
            p = np.arange(len(hk) - m, len(hk))
            want, tol = SM.attention(W.bf16_bits_to_f32(qb[rows]), keys, vals, p, *SM.bounds(p, len(hk), window=200),
                                     d ** -0.5, softcap=10.0, k_mag=mags[0], v_mag=mags[1])
            off = np.abs(out[rows].float().cpu().numpy() - want) - tol
            assert (off <= 0).all(), f"slot {s}: {off.max():.3e} beyond the tolerance"
