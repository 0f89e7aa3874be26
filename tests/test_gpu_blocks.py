"""Key bounds, block selection, block-sparse attention and accepted rows on the GPU against ``oracle.blocks``
(float64). Bounds, choices and moves have to be equal; attention is held to the oracle's element-wise tolerance."""

import zlib

import numpy as np
import pytest

import oracle
from oracle import blocks as OB
from oracle import kvquant as KQ
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


HEADS = [(4, 2, 64), (32, 8, 128), (40, 8, 128), (8, 8, 64), (16, 1, 128), (6, 6, 128), (16, 1, 64)]


def _seed(*what):
    return zlib.crc32("/".join(map(str, what)).encode()) % 1000


def _values(w, kv):
    """Per slot ((k, magnitudes), (v, magnitudes)) in float64 as the pool holds them."""
    out = {}
    for s in w.segments:
        one = []
        for h in (w.hist_k[s.slot], w.hist_v[s.slot]):
            if kv == "bf16":
                one.append((W.bf16_bits_to_f32(h).astype(np.float64), None))
            else:
                codes, scales = KQ.quantize(h, int(kv[1]))
                d = np.repeat(W.bf16_bits_to_f32(scales).astype(np.float64), 32, -1)
                one.append((KQ.dequantize(codes, scales), (np.abs(codes.astype(np.float64)) + 1152) * d))
        out[s.slot] = one
    return out


def _pool(ds):
    return (ds.k_pool, ds.v_pool) if ds.kv == "bf16" else (ds.k_pool, ds.k_scales, ds.v_pool, ds.v_scales)


def _whole_mapping(ds):
    """Pool rows of every position of every slot, in order."""
    t, bs = ds.pool.block_tables(), ds.w.block_size
    rows = [t[s.slot][np.arange(s.ctx) // bs].astype(np.int64) * bs + np.arange(s.ctx) % bs for s in ds.w.segments]
    return torch.from_numpy(np.concatenate(rows)).cuda()


def _new_bounds(ds):
    return torch.full((ds.w.num_blocks, ds.w.num_kv_heads, 2, ds.w.head_dim), 77.0, dtype=torch.bfloat16, device="cuda")


def _bounds(ds, mapping=None):
    b = _new_bounds(ds)
    keys = _pool(ds)[: 1 if ds.kv == "bf16" else 2]
    B.KeyBoundsCall(_whole_mapping(ds) if mapping is None else mapping, keys, b, kv=ds.kv, device_status=ds.status)()
    return b


def _plan(ds, sparse):
    w, low = ds.w, ds.lowered
    work, info = B.pkv_plan_work_sparse(low.cu_seqlens_q, low.seq_slot, low.context_lens, max_slots=w.max_slots,
                                        max_blocks_per_slot=w.max_blocks_per_slot, block_size=w.block_size,
                                        num_q_heads=w.num_q_heads, num_kv_heads=w.num_kv_heads, head_dim=w.head_dim,
                                        sparse=sparse)
    return (torch.from_numpy(work).cuda(), info,
            torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda"))


def _select_call(ds, sparse, plan, bounds):
    work, info, ws = plan
    sel = torch.full((len(ds.w.segments), ds.w.num_kv_heads, sparse.top_blocks), -9, dtype=torch.int32, device="cuda")
    return sel, B.SelectBlocksCall(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, bounds, work, info,
                                   sel, ws, sparse=sparse, block_size=ds.w.block_size, device_status=ds.status)


def _attend_call(ds, sparse, plan, sel):
    work, info, ws = plan
    return B.AttentionSparseCall(ds.q, ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, _pool(ds), sel, work,
                                 info, ds.out, ws, sparse=sparse, kv=ds.kv, scale=ds.scale, device_status=ds.status)


def _want_choice(w, sparse, lohi, q=None):
    """Oracle's choice; lohi(slot, head) -> (lo, hi) [blocks, D] in logical order."""
    q = W.bf16_bits_to_f32(w.q).astype(np.float64) if q is None else q
    g = w.num_q_heads // w.num_kv_heads
    out = np.full((len(w.segments), w.num_kv_heads, sparse.top_blocks), -1)
    row = 0
    for i, s in enumerate(w.segments):
        for h in range(w.num_kv_heads):
            c = OB.choose(q[row:row + s.q_len, h * g:(h + 1) * g], *lohi(s.slot, h), s.ctx, w.block_size, sparse.top_blocks,
                          sparse.keep_first, sparse.keep_last)
            out[i, h, : len(c)] = c
        row += s.q_len
    return out


def _want_attention(w, kv, sel):
    q = W.bf16_bits_to_f32(w.q).astype(np.float64)
    vals, g, bs = _values(w, kv), w.num_q_heads // w.num_kv_heads, w.block_size
    out, tol, row = np.zeros(q.shape), np.zeros(q.shape), 0
    for i, s in enumerate(w.segments):
        rows = slice(row, row + s.q_len)
        row += s.q_len
        (k, km), (v, vm) = vals[s.slot]
        for h in range(w.num_kv_heads):
            places = sel[i, h][sel[i, h] >= 0]
            keys = np.concatenate([np.arange(p * bs, min(s.ctx, (p + 1) * bs)) for p in places])
            pick = lambda x: None if x is None else x[keys, h:h + 1]  # noqa: E731
            seen = keys <= np.arange(s.ctx - s.q_len, s.ctx)[:, None]
            o, t = OB.attention(q[rows, h * g:(h + 1) * g], pick(k), pick(v), seen, w.scale, k_mag=pick(km), v_mag=pick(vm))
            out[rows, h * g:(h + 1) * g], tol[rows, h * g:(h + 1) * g] = o, t
    return out, tol


def _check(ds, sel, what):
    want, tol = _want_attention(ds.w, ds.kv, sel)
    got = R.out_f32(ds)
    assert np.isfinite(got).all(), what
    off = np.abs(got - want) - tol
    assert (off <= 0).all(), f"{what}: {off.max():.3e} beyond the tolerance"


# ---------------------------------------------------------------------------
# Bounds
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "q8", "q4"])
def test_bounds(kv):
    for i, (hq, hkv, d) in enumerate(HEADS):
        if kv == "q4" and d != 128:
            continue
        bs = [16, 32, 64][i % 3]
        w = W.random_step(_seed("bounds", kv, i), [(1, 1), (40, 333), (1, 64), (3, 17), (17, 17), (200, 256)], num_q_heads=hq,
                          num_kv_heads=hkv, head_dim=d, block_size=bs)
        ds = R.prepare(w, kv=kv)
        R.run_cache_write(ds)
        vals = _values(w, kv)
        # of the whole history, and of the blocks that this step's rows touch alone (rows never written are NaN)
        for mapping, first in ((None, lambda s: 0), (ds.slot_mapping, lambda s: (s.ctx - s.q_len) // bs)):
            got = _bounds(ds, mapping).to(torch.float64).cpu().numpy()
            want = np.full(got.shape, 77.0)
            for s in w.segments:
                for j in range(first(s), -(-s.ctx // bs)):
                    k = vals[s.slot][0][0][j * bs: min(s.ctx, (j + 1) * bs)]
                    want[w.blocks[s.slot][j]] = OB.bounds(k).transpose(1, 0, 2)
            assert np.array_equal(got, want), (kv, hq, hkv, d)
        assert B.pkv_check_device_status(ds.status) == 0


def test_bounds_forget_rows_behind_the_last_one():
    """After a cut the block's bounds are those of the rows that are left, not of what stood there."""
    w = W.random_step(3, [(30, 30)], num_q_heads=4, num_kv_heads=2, head_dim=64, block_size=32)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    b = _bounds(ds, ds.slot_mapping[:11].contiguous())
    k = _values(w, "bf16")[0][0][0]
    assert np.array_equal(b[int(w.blocks[0][0])].double().cpu().numpy(), OB.bounds(k[:11]).transpose(1, 0, 2))


def test_bounds_skip_and_report():
    w = W.random_step(4, [(40, 40)], num_q_heads=4, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    m = ds.slot_mapping.clone()
    m[20:] = -1
    whole = _bounds(ds)
    got = _bounds(ds, m)
    assert torch.equal(got[int(w.blocks[0][0])], whole[int(w.blocks[0][0])])
    k = _values(w, "bf16")[0][0][0]
    assert np.array_equal(got[int(w.blocks[0][1])].double().cpu().numpy(), OB.bounds(k[16:20]).transpose(1, 0, 2))
    assert (got[int(w.blocks[0][2])] == 77).all() and B.pkv_check_device_status(ds.status) == 0
    m[:] = w.num_blocks * 16
    assert (_bounds(ds, m) == 77).all() and B.pkv_check_device_status(ds.status) == 1


@pytest.mark.parametrize("tokens", [1, 31, 33, 5000])
def test_bounds_of_any_number_of_tokens(tokens):
    w = W.random_step(5, [(tokens, tokens + 7)], num_q_heads=2, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    whole, part = _bounds(ds), _bounds(ds, ds.slot_mapping)
    assert torch.equal(whole, part)


# ---------------------------------------------------------------------------
# Selection
# ---------------------------------------------------------------------------

def _lohi(ds, bounds):
    b = bounds.double().cpu().numpy()
    return lambda slot, h: (b[ds.w.blocks[slot]][:, h, 0], b[ds.w.blocks[slot]][:, h, 1])


@pytest.mark.parametrize("case", ["decode", "runs", "long"])
@pytest.mark.parametrize("i", range(len(HEADS)))
def test_choice(case, i):
    hq, hkv, d = HEADS[i]
    most = max(1, 16 // (hq // hkv))
    bs = [16, 32, 64][i % 3]
    shapes = {"decode": [(1, 1), (1, 17), (1, 700), (1, 5000), (1, 16), (1, 2048)],
              "runs": [(min(3, most), 900), (min(2, most), 2), (most, 4001), (most, 640), (1, 333)],
              "long": [(1, 40000), (most, 30011)]}[case]
    w = W.random_step(_seed("choice", case, i), shapes, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    bounds = _bounds(ds)
    for sparse in (B.Sparse(9, 1, 2), B.Sparse(24, 0, 0), B.Sparse(40, 2, 3), B.Sparse(5000, 1, 1)):
        sel, call = _select_call(ds, sparse, _plan(ds, sparse), bounds)
        call()
        assert B.pkv_check_device_status(ds.status) == 0
        assert np.array_equal(sel.cpu().numpy(), _want_choice(w, sparse, _lohi(ds, bounds))), (hq, hkv, d, sparse)


def _choice_over(lo, hi, q, sparse, bs=16, ctx=None):
    """Selection of one segment over bounds [blocks, hkv, D] given in logical order; q [n, hq, D]. Returns (got, want)."""
    n, hq, d = q.shape
    nb, hkv, _ = lo.shape
    ctx = nb * bs if ctx is None else ctx
    table = np.random.RandomState(0).permutation(nb + 3)[:nb].astype(np.int32)
    bounds = torch.zeros(nb + 3, hkv, 2, d, dtype=torch.bfloat16, device="cuda")
    bounds[torch.from_numpy(table).long().cuda()] = torch.from_numpy(np.stack([lo, hi], 2)).cuda().to(torch.bfloat16)
    exact = bounds.double().cpu().numpy()[table]
    cu, ss, cl = np.array([0, n], np.int32), np.zeros(1, np.int32), np.array([ctx], np.int32)
    work, info = B.pkv_plan_work_sparse(cu, ss, cl, max_slots=1, max_blocks_per_slot=nb, block_size=bs, num_q_heads=hq,
                                        num_kv_heads=hkv, head_dim=d, sparse=sparse)
    sel = torch.full((1, hkv, sparse.top_blocks), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    B.pkv_select_blocks(qd, *(torch.from_numpy(x).cuda() for x in (cu, ss, cl)), torch.from_numpy(table[None]).cuda(), bounds,
                        torch.from_numpy(work).cuda(), info, sel,
                        torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda"), sparse=sparse,
                        block_size=bs, device_status=status)
    assert B.pkv_check_device_status(status) == 0
    qf, g = qd.double().cpu().numpy(), hq // hkv
    want = [OB.choose(qf[:, h * g:(h + 1) * g], exact[:, h, 0], exact[:, h, 1], ctx, bs, sparse.top_blocks,
                      sparse.keep_first, sparse.keep_last) for h in range(hkv)]
    return sel.cpu().numpy()[0], np.array([x + [-1] * (sparse.top_blocks - len(x)) for x in want])


@pytest.mark.parametrize("blocks", [20, 300, 1500, 9000])
@pytest.mark.parametrize("kind", ["same", "zero q", "few values", "close", "wide", "cancel"])
def test_choice_among_equal_and_close_scores(kind, blocks):
    """Equal scores go to the lowest place; scores that 32 bits cannot tell apart are told apart."""
    rng = np.random.default_rng(_seed(kind, blocks))
    hq, hkv, d = 4, 1, 64
    q = rng.standard_normal((1, hq, d))
    lo = rng.standard_normal((blocks, hkv, d)) - 1
    hi = lo + rng.random((blocks, hkv, d))
    if kind == "same":
        lo[:], hi[:] = lo[0], hi[0]
    elif kind == "zero q":
        q[:] = 0
    elif kind == "few values":
        lo[:] = rng.choice([-1.0, -0.5], (blocks, hkv, 1))
        hi[:] = rng.choice([0.5, 1.0, 2.0], (blocks, hkv, 1))
        q[:] = 1
    elif kind == "close":  # differences of 2^-30 of the score
        lo[:], hi[:] = -1, 1
        q[:] = 1
        q[..., 0] = 2.0 ** -20
        hi[..., 0] = 1 + rng.integers(0, 100, (blocks, hkv)) * 2.0 ** -7
    elif kind == "wide":
        q *= 2.0 ** rng.integers(-40, 40, (1, hq, d))
        hi = np.abs(hi) * 2.0 ** rng.integers(-40, 40, (blocks, hkv, d))
        lo = -hi
    else:  # large terms that cancel: what is left decides
        q[:] = 1
        q[..., 1] = -1
        hi[..., 0] = lo[..., 0] = 2.0 ** 12
        hi[..., 1] = lo[..., 1] = 2.0 ** 12
    for sparse in (B.Sparse(8, 1, 1), B.Sparse(17, 0, 0)):
        got, want = _choice_over(lo, hi, q, sparse)
        assert np.array_equal(got, want), (kind, blocks, sparse)


def test_choice_of_one_and_of_all_but_one():
    rng = np.random.default_rng(0)
    lo = rng.standard_normal((400, 2, 128))
    hi, q = lo + 1, rng.standard_normal((1, 8, 128))
    for sparse in (B.Sparse(1, 0, 0), B.Sparse(2, 0, 0), B.Sparse(399, 3, 3), B.Sparse(400, 0, 0), B.Sparse(9, 4, 4)):
        for ctx in (6400, 6399, 6385):
            got, want = _choice_over(lo, hi, q, sparse, ctx=ctx)
            assert np.array_equal(got, want), (sparse, ctx)


def test_choice_among_many_blocks():
    """More candidates than a CTA holds in registers, in both sizes of CTA."""
    rng = np.random.default_rng(2)
    for blocks in (2049, 8193, 40000):
        lo = rng.standard_normal((blocks, 1, 64))
        got, want = _choice_over(lo, lo + rng.random((blocks, 1, 64)), rng.standard_normal((2, 4, 64)), B.Sparse(300, 1, 1))
        assert np.array_equal(got, want)


def test_choice_with_values_that_are_not_finite():
    """Scores that are not numbers rank last; infinities neither fault nor leave a place out or name one twice."""
    rng = np.random.default_rng(3)
    lo = rng.standard_normal((200, 1, 64))
    hi, q = lo + 1, np.abs(rng.standard_normal((1, 2, 64))) + 0.1
    bad = hi.copy()
    bad[::3, 0, 5] = np.nan
    got, _ = _choice_over(lo, bad, q, B.Sparse(40, 0, 0))
    assert not set(got[0][:-1]) & set(range(0, 199, 3)) and (np.diff(got[0]) > 0).all()
    for value in (np.inf, -np.inf):
        for at in (lo, hi, q):
            x = at.copy()
            x[..., 7] = value
            a = [x if y is at else y for y in (lo, hi, q)]
            got, _ = _choice_over(*a, B.Sparse(40, 1, 1))
            assert (np.diff(got[0]) > 0).all() and got.min() >= 0 and got.max() == 199


# ---------------------------------------------------------------------------
# Attention over the chosen blocks
# ---------------------------------------------------------------------------

def _any_choice(w, sparse, seed):
    """A list that keeps what is always kept and any others."""
    rng = np.random.default_rng(seed)
    out = np.full((len(w.segments), w.num_kv_heads, sparse.top_blocks), -1, np.int32)
    for i, s in enumerate(w.segments):
        m, a, b = OB.always(s.ctx, s.q_len, w.block_size, sparse.keep_first, sparse.keep_last)
        for h in range(w.num_kv_heads):
            some = np.arange(m)
            if m > sparse.top_blocks:
                free = sparse.top_blocks - a - (m - b)
                some = np.sort(np.concatenate([np.arange(a), np.arange(b, m), a + rng.permutation(b - a)[:free]]))
            out[i, h, : len(some)] = some
    return out


@pytest.mark.parametrize("kv", ["bf16", "q8", "q4"])
@pytest.mark.parametrize("i", range(len(HEADS)))
def test_attention(kv, i):
    hq, hkv, d = HEADS[i]
    if kv == "q4" and d != 128:
        pytest.skip("4-bit pools hold heads of 128")
    most, bs = max(1, 16 // (hq // hkv)), [16, 32, 64][(i + len(kv)) % 3]
    for case, shapes in (("decode", [(1, 1), (1, 17), (1, 700), (1, 5000), (1, 16), (1, 2050)]),
                         ("runs", [(min(3, most), 900), (min(2, most), 2), (most, 4001), (most, 641), (1, 333)]),
                         ("one", [(1, 3001)])):
        w = W.random_step(_seed("sparse", kv, i, case), shapes, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=bs)
        ds = R.prepare(w, kv=kv)
        R.run_cache_write(ds)
        for sparse in (B.Sparse(5, 1, 1), B.Sparse(17, 0, 0), B.Sparse(90, 2, 3)):
            sel = _any_choice(w, sparse, i)
            plan = _plan(ds, sparse)
            plan[2].fill_(0xFF)  # the workspace needs no start value
            _attend_call(ds, sparse, plan, torch.from_numpy(sel).cuda())()
            assert B.pkv_check_device_status(ds.status) == 0
            _check(ds, sel, f"{kv} {hq}/{hkv}/{d} {case} {sparse}")


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_blocks_that_are_not_chosen_may_hold_anything(kv):
    """Keys, values and scales that are no numbers in every block that the step does not read."""
    w = W.random_step(17, [(1, 3000), (3, 1111), (1, 90)], num_q_heads=8, num_kv_heads=2, head_dim=128)
    ds = R.prepare(w, kv=kv)
    R.run_cache_write(ds)
    sparse = B.Sparse(7, 1, 1)
    sel = _any_choice(w, sparse, 3)
    sel[:] = sel[:, :1]  # the same blocks for both heads
    read = {int(w.blocks[s.slot][p]) for i, s in enumerate(w.segments) for p in sel[i, 0] if p >= 0}
    rest = torch.tensor([b for b in range(w.num_blocks) if b not in read], device="cuda")
    for a in _pool(ds):
        a[rest] = float("nan") if a.is_floating_point() else 127
    plan = _plan(ds, sparse)
    _attend_call(ds, sparse, plan, torch.from_numpy(sel).cuda())()
    assert B.pkv_check_device_status(ds.status) == 0
    _check(ds, sel, kv)


def test_all_blocks_are_plain_attention():
    w = W.random_step(9, [(1, 3000), (4, 777), (1, 1)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    R.run_step(ds)
    plain = R.out_f32(ds)
    sparse = B.Sparse(w.max_blocks_per_slot)
    ds.out.fill_(5.0)
    _attend_call(ds, sparse, _plan(ds, sparse), torch.from_numpy(_any_choice(w, sparse, 0)).cuda())()
    _check(ds, _any_choice(w, sparse, 0), "all")
    assert np.abs(R.out_f32(ds) - plain).max() < 2e-2


def test_rows_of_other_segments_stay():
    """The sparse segments are the last ones of a packed step: the rows in front are neither read nor written."""
    w = W.random_step(10, [(40, 300), (1, 1000), (2, 900)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    ds.out.fill_(5.0)
    sparse, low = B.Sparse(12), ds.lowered
    shape = dict(max_slots=w.max_slots, max_blocks_per_slot=w.max_blocks_per_slot, block_size=16, num_q_heads=8, num_kv_heads=2,
                 head_dim=64)
    work, info = B.pkv_plan_work_sparse(low.cu_seqlens_q[1:], low.seq_slot[1:], low.context_lens, **shape, sparse=sparse)
    plan = torch.from_numpy(work).cuda(), info, torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda")
    ds.cu_seqlens_q, ds.seq_slot = ds.cu_seqlens_q[1:].contiguous(), ds.seq_slot[1:].contiguous()
    bounds = _bounds(ds)
    head, w.segments = w.segments[0], w.segments[1:]
    sel, call = _select_call(ds, sparse, plan, bounds)
    call()
    _attend_call(ds, sparse, plan, sel)()
    assert B.pkv_check_device_status(ds.status) == 0
    got = R.out_f32(ds)
    assert (got[:40] == 5).all()
    w.q = w.q[40:]
    assert np.array_equal(sel.cpu().numpy(), _want_choice(w, sparse, _lohi(ds, bounds)))
    want, tol = _want_attention(w, "bf16", sel.cpu().numpy())
    assert (np.abs(got[40:] - want) <= tol).all()


def test_bad_places_are_reported():
    w = W.random_step(11, [(1, 2000), (1, 500)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    sparse = B.Sparse(12)
    good = _any_choice(w, sparse, 1)
    for bad in (-1, 125, 10 ** 6, -2 ** 31):
        sel = good.copy()
        sel[0, 1, 3] = bad
        _attend_call(ds, sparse, _plan(ds, sparse), torch.from_numpy(sel).cuda())()
        assert B.pkv_check_device_status(ds.status) == 2
        want, tol = _want_attention(w, "bf16", np.where(sel > 124, -1, sel))
        assert (np.abs(R.out_f32(ds) - want) <= tol).all()  # the block is left out, the rest stands


def test_lists_that_do_not_fit_the_step_are_reported():
    """A list made for longer contexts: the items past the step's own are skipped."""
    w = W.random_step(12, [(1, 2000), (1, 500)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    bounds, sparse = _bounds(ds), B.Sparse(12)
    plan = _plan(ds, sparse)
    ds.context_lens[0] = 100
    sel, call = _select_call(ds, sparse, plan, bounds)
    call()
    assert B.pkv_check_device_status(ds.status) == 4 and (sel[0] == -1).all() and (sel[1] >= 0).all()
    _attend_call(ds, sparse, plan, torch.from_numpy(_any_choice(w, sparse, 0)).cuda())()
    assert B.pkv_check_device_status(ds.status) & 4


# ---------------------------------------------------------------------------
# Accepted rows
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "q8", "q4"])
def test_accepted_rows(kv):
    for i, (hq, hkv, d) in enumerate([(4, 2, 64), (32, 8, 128)]):
        if kv == "q4" and d == 64:
            continue
        rng = np.random.default_rng(i)
        shapes = [(8, 100), (1, 50), (100, 100), (64, 333), (16, 16), (5, 70)]
        w = W.random_step(20 + i, shapes, num_q_heads=hq, num_kv_heads=hkv, head_dim=d, block_size=[16, 32][i])
        ds = R.prepare(w, kv=kv)
        R.run_cache_write(ds)
        paths = np.full((len(shapes), 70), -1, np.int32)
        for s, (n, _) in enumerate(shapes):
            m = int(rng.integers(0, min(n, 70) + 1)) if s else 4
            paths[s, :m] = np.sort(rng.permutation(n)[:m])
        paths[2, :70] = np.arange(30, 100)  # overlapping, longer than one round
        want = [a.view(torch.int16 if a.dtype == torch.bfloat16 else a.dtype).cpu().numpy().copy() for a in _pool(ds)]
        for s, seg in zip(range(len(shapes)), w.segments):
            t, at0 = w.blocks[seg.slot], seg.ctx - seg.q_len
            at = lambda p: (t[(at0 + p) // w.block_size], slice(None), (at0 + p) % w.block_size)  # noqa: E731
            for a in want:
                old = a.copy()
                for depth, p in enumerate(paths[s]):
                    if p < 0:
                        break
                    a[at(depth)] = old[at(p)]
        B.pkv_accept_rows(ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables, torch.from_numpy(paths).cuda(),
                          _pool(ds), device_status=ds.status)
        assert B.pkv_check_device_status(ds.status) == 0
        for a, b in zip(_pool(ds), want):
            assert np.array_equal(a.view(torch.int16 if a.dtype == torch.bfloat16 else a.dtype).cpu().numpy(), b)


@pytest.mark.parametrize("path", [[3, 2], [0, 0, 1], [1, 8], [2 ** 31 - 1]])
def test_paths_that_do_not_grow_end_there(path):
    w = W.random_step(30, [(8, 100)], num_q_heads=4, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    want = R.pool_bits(ds)[0].copy()
    at = lambda p: (w.blocks[0][(92 + p) // 16], slice(None), (92 + p) % 16)  # noqa: E731
    if path[0] < 8:
        want[at(0)] = want[at(path[0])]
    B.pkv_accept_rows(ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables,
                      torch.tensor([path + [-1]], dtype=torch.int32, device="cuda"), [ds.k_pool], device_status=ds.status)
    assert B.pkv_check_device_status(ds.status) == 4
    assert np.array_equal(R.pool_bits(ds)[0], want)


def test_attention_behind_a_move_sees_the_moved_rows():
    """pkv_attention reads history before it waits for the kernel before it: a move must be over by then."""
    w = W.random_step(31, [(1, 257)] * 60, num_q_heads=8, num_kv_heads=2, head_dim=128)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    path = torch.tensor([[0]] * 60, dtype=torch.int32, device="cuda")
    for _ in range(3):
        # the last 8 rows of every slot as a segment: its nodes 3, 5, 7 move to the front
        cu8 = torch.arange(0, 481, 8, dtype=torch.int32, device="cuda")
        path = torch.tensor([[3, 5, 7]] * 60, dtype=torch.int32, device="cuda")
        B.pkv_accept_rows(cu8, ds.seq_slot, ds.context_lens, ds.block_tables, path, [ds.k_pool, ds.v_pool])
        R.run_attention(ds)
        torch.cuda.synchronize()
        got = ds.out.clone()
        R.run_attention(ds)
        assert torch.equal(got, ds.out)


# ---------------------------------------------------------------------------
# Together
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_a_sparse_step_captured_and_replayed(kv):
    """Cache write, bounds, choice and attention in one graph, replayed on new queries and keys; twice on a side
    stream, with the same workspace for choice and attention."""
    w = W.random_step(40, [(1, 5000), (2, 900), (1, 40), (1, 1300)], num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w, kv=kv)
    R.run_cache_write(ds)
    bounds, sparse = _bounds(ds), B.Sparse(20, 1, 2)
    plan = _plan(ds, sparse)
    sel, select = _select_call(ds, sparse, plan, bounds)
    attend = _attend_call(ds, sparse, plan, sel)
    touch = B.KeyBoundsCall(ds.slot_mapping, _pool(ds)[: 1 if kv == "bf16" else 2], bounds, kv=kv, device_status=ds.status)

    def step():
        R.run_cache_write(ds)
        touch()
        select()
        attend()

    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for scale in (1.0, -2.0):
        ds.q.mul_(scale)
        ds.k_new.mul_(scale)
        step()
        torch.cuda.synchronize()
        want_sel, want = sel.clone(), ds.out.clone()
        sel.fill_(-5)
        ds.out.fill_(3.0)
        with torch.cuda.stream(side):
            side.wait_stream(torch.cuda.default_stream())
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(sel, want_sel) and torch.equal(ds.out, want)
        assert B.pkv_check_device_status(ds.status) == 0
        q = ds.q.double().cpu().numpy()
        assert np.array_equal(sel.cpu().numpy(), _want_choice(w, sparse, _lohi(ds, bounds), q))


def test_results_do_not_depend_on_the_rest_of_the_step():
    """A slot alone and among others, in any order: the same choice and the same bits."""
    rng = np.random.default_rng(0)
    shapes = [(1, 3000), (2, 900), (1, 40), (1, 1300)]
    w = W.random_step(41, shapes, num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    bounds, sparse, low = _bounds(ds), B.Sparse(20, 1, 2), ds.lowered
    plan = _plan(ds, sparse)
    sel, call = _select_call(ds, sparse, plan, bounds)
    call()
    _attend_call(ds, sparse, plan, sel)()
    cu, out = low.cu_seqlens_q, ds.out.clone()
    for order in ([0], [1], [2], [3], list(rng.permutation(4))):
        q = torch.cat([ds.q[cu[s]:cu[s + 1]] for s in order])
        c2 = np.concatenate([[0], np.cumsum([shapes[s][0] for s in order])]).astype(np.int32)
        work, info = B.pkv_plan_work_sparse(c2, low.seq_slot[order], low.context_lens, max_slots=w.max_slots,
                                            max_blocks_per_slot=w.max_blocks_per_slot, block_size=16, num_q_heads=32,
                                            num_kv_heads=8, head_dim=128, sparse=sparse)
        ws = torch.empty(max(256, info.workspace_bytes), dtype=torch.uint8, device="cuda")
        s2, o2 = torch.empty_like(sel[: len(order)]), torch.empty_like(q)
        meta = (torch.from_numpy(c2).cuda(), ds.seq_slot[torch.tensor(order).cuda()].contiguous(), ds.context_lens,
                ds.block_tables)
        wk = torch.from_numpy(work).cuda()
        B.pkv_select_blocks(q, *meta, bounds, wk, info, s2, ws, sparse=sparse, block_size=16)
        B.pkv_attention_sparse(q, *meta, ds.k_pool, ds.v_pool, s2, wk, info, o2, ws, sparse=sparse, scale=w.scale)
        for i, s in enumerate(order):
            assert torch.equal(s2[i], sel[s]) and torch.equal(o2[c2[i]:c2[i + 1]], out[cu[s]:cu[s + 1]])


def test_calls_refuse_what_does_not_fit():
    w = W.random_step(42, [(1, 300)], num_q_heads=8, num_kv_heads=2, head_dim=64)
    ds = R.prepare(w)
    bounds, sparse = _new_bounds(ds), B.Sparse(8)
    plan = _plan(ds, sparse)
    sel, _ = _select_call(ds, sparse, plan, bounds)
    meta = (ds.cu_seqlens_q, ds.seq_slot, ds.context_lens, ds.block_tables)
    with pytest.raises(ValueError):
        B.pkv_select_blocks(ds.q, *meta, bounds, plan[0], plan[1], sel[:, :1].contiguous(), plan[2], sparse=sparse, block_size=16)
    with pytest.raises(ValueError):
        B.pkv_select_blocks(ds.q.float(), *meta, bounds, plan[0], plan[1], sel, plan[2], sparse=sparse, block_size=16)
    with pytest.raises(ValueError):
        B.pkv_attention_sparse(ds.q, *meta, ds.k_pool, ds.v_pool, sel.cpu(), plan[0], plan[1], ds.out, plan[2], sparse=sparse)
    with pytest.raises(ValueError):
        B.pkv_attention_sparse(ds.q, *meta, ds.k_pool, ds.v_pool, sel, plan[0][:4], plan[1], ds.out, plan[2], sparse=sparse)
    with pytest.raises(B.PkvError) as e:
        B.pkv_attention_sparse(ds.q, *meta, ds.k_pool, ds.v_pool, sel, plan[0], plan[1], ds.out, None, sparse=sparse)
    assert e.value.status == B.PKV_ERR_WORKSPACE_TOO_SMALL
    with pytest.raises(ValueError):
        B.pkv_key_bounds(ds.slot_mapping, ds.k_pool, bounds[:, :, :, :32].contiguous())
    with pytest.raises(ValueError):
        B.pkv_accept_rows(*meta, torch.zeros(2, 4, dtype=torch.int32, device="cuda"), [ds.k_pool])


@pytest.mark.parametrize("kv", ["bf16", "q8", "q4"])
def test_bounds_of_a_block_that_is_copied_on_write(kv):
    """Bounds are one more array of the pool: a partly filled block is adopted and then branches. The copy has the
    block's bounds; the step that follows makes those of its rows; the other table's block keeps its own."""
    bs, hq, hkv, d, shared = 16, 8, 2, 128, 90
    x = lambda n: torch.randn(n, hkv, d, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    arrays = R.empty_pool(40, hkv, bs, d, "cuda") if kv == "bf16" else R.empty_pool_q8(40, hkv, bs, d, "cuda", int(kv[1]))
    bounds = torch.full((40, hkv, 2, d), 77.0, dtype=torch.bfloat16, device="cuda")
    keys, status = arrays[: len(arrays) // 2], torch.zeros(1, dtype=torch.int32, device="cuda")
    write = {"bf16": B.pkv_cache_write, "q8": B.pkv_cache_write_q8, "q4": B.pkv_cache_write_q4}[kv]
    pool = B.Pool(40, bs, 3, 12)
    pool.admit(0, 0)
    stored = {}

    def append(slot, n):
        low = pool.lower([(slot, n)])
        pairs = pool.take_copies()
        if len(pairs):
            B.pkv_copy_blocks(dev(pairs), [*arrays, bounds], device_status=status)
            src, dst = pairs[0].tolist()
            assert torch.equal(bounds[dst], bounds[src])
        k, m = x(n), dev(low.slot_mapping)
        write(k, x(n), m, *arrays, device_status=status)
        B.KeyBoundsCall(m, keys, bounds, kv=kv, device_status=status)()
        bits = k.view(torch.int16).cpu().numpy().view(np.uint16)
        stored[slot] = np.concatenate([stored[slot], bits]) if slot in stored else bits
        return len(pairs)

    assert append(0, shared) == 0
    pool.adopt(1, 0, shared)
    stored[1] = stored[0].copy()
    assert append(1, 30) == 1 and append(0, 3) == 0 and append(1, 1) == 0
    for slot in (0, 1):
        vals = W.bf16_bits_to_f32(stored[slot]) if kv == "bf16" else KQ.dequantize(*KQ.quantize(stored[slot], int(kv[1])))
        vals = vals.astype(np.float64)
        table = pool.block_tables()[slot]
        for j in range(-(-len(vals) // bs)):
            want = OB.bounds(vals[j * bs:(j + 1) * bs]).transpose(1, 0, 2)
            assert np.array_equal(bounds[int(table[j])].double().cpu().numpy(), want), (slot, j)
    assert B.pkv_check_device_status(status) == 0


@pytest.mark.parametrize("kind", ["any", "same", "few values"])
@pytest.mark.parametrize("blocks", [2049, 2500, 12000])
def test_choice_of_one_long_slot_among_short_ones(blocks, kind):
    """The segments' mean sets the size of the CTAs: small ones then choose among more candidates than they hold, here
    with and without scores that have to be told apart."""
    rng = np.random.default_rng(_seed(blocks, kind))
    hq, hkv, d, bs, slots, sparse = 8, 2, 64, 16, 40, B.Sparse(24, 1, 1)
    counts = [30, 26, 1, blocks, 25] + [28] * 15
    table = np.full((slots, blocks), -1, np.int32)
    order, at, ss = rng.permutation(sum(counts)).astype(np.int32), 0, rng.permutation(slots)[: len(counts)].astype(np.int32)
    for s, m in zip(ss, counts):
        table[s, :m] = order[at:at + m]
        at += m
    lo = rng.standard_normal((at, hkv, d))
    if kind != "any":
        lo[:] = rng.choice([-1.0, -0.5], (at, hkv, 1)) if kind == "few values" else lo[0]
    bounds = torch.from_numpy(np.stack([lo, lo + (rng.random(lo.shape) if kind == "any" else 1.0)], 2)).cuda().bfloat16()
    q = torch.from_numpy(rng.standard_normal((len(counts), hq, d))).cuda().bfloat16()
    if kind == "few values":
        q[:] = 1
    cu, ctx = np.arange(len(counts) + 1, dtype=np.int32), np.zeros(slots, np.int32)
    ctx[ss] = np.array(counts) * bs - 3
    work, info = B.pkv_plan_work_sparse(cu, ss, ctx, max_slots=slots, max_blocks_per_slot=blocks, block_size=bs,
                                        num_q_heads=hq, num_kv_heads=hkv, head_dim=d, sparse=sparse)
    assert info.scratch_blocks <= 1024 * info.num_prefill_items
    sel = torch.full((len(counts), hkv, 24), -9, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.pkv_select_blocks(q, *(torch.from_numpy(x).cuda() for x in (cu, ss, ctx, table)), bounds, torch.from_numpy(work).cuda(),
                        info, sel, torch.empty(info.workspace_bytes, dtype=torch.uint8, device="cuda"), sparse=sparse,
                        block_size=bs, device_status=status)
    assert B.pkv_check_device_status(status) == 0
    q64, exact, got = q.double().cpu().numpy(), bounds.double().cpu().numpy(), sel.cpu().numpy()
    for i, (s, m) in enumerate(zip(ss, counts)):
        for h in range(hkv):
            c = OB.choose(q64[i:i + 1, 4 * h:4 * h + 4], *exact[table[s, :m]][:, h].transpose(1, 0, 2), ctx[s], bs, 24, 1, 1)
            assert got[i, h].tolist() == c + [-1] * (24 - len(c)), (i, h)


@pytest.mark.parametrize("kv", ["bf16", "q8", "q4"])
def test_a_sparse_step_beside_idle_slots(kv):
    """A server's slots are mostly more than a step's: the cut of the keys follows the slots, the results do not."""
    w = W.random_step(43, [(1, 5000), (2, 900), (1, 40), (1, 1300)], num_q_heads=32, num_kv_heads=8, head_dim=128,
                      max_slots=64, slots=[60, 3, 17, 34])
    ds = R.prepare(w, kv=kv)
    R.run_cache_write(ds)
    bounds, sparse = _bounds(ds), B.Sparse(100, 1, 2)
    plan = _plan(ds, sparse)
    sel, call = _select_call(ds, sparse, plan, bounds)
    call()
    _attend_call(ds, sparse, plan, sel)()
    assert B.pkv_check_device_status(ds.status) == 0
    want = _want_choice(w, sparse, _lohi(ds, bounds))
    assert np.array_equal(sel.cpu().numpy(), want)
    _check(ds, want, kv)


def test_attention_started_with_a_move_sees_every_moved_row():
    """Long moves over rows that are new in every round, and attention that reads them as history: launched one behind
    the other and in one graph, against the same calls with a synchronisation between them."""
    w = W.random_step(32, [(1, 400)] * 60, num_q_heads=32, num_kv_heads=8, head_dim=128)
    ds = R.prepare(w)
    R.run_cache_write(ds)
    cu = torch.arange(0, 60 * 140 + 1, 140, dtype=torch.int32, device="cuda")  # the last 140 rows of every slot
    path = torch.arange(40, 130, dtype=torch.int32, device="cuda").expand(60, 90).contiguous()
    move = B.AcceptRowsCall(cu, ds.seq_slot, ds.context_lens, ds.block_tables, path, [ds.k_pool, ds.v_pool],
                            device_status=ds.status)
    move()
    R.run_attention(ds)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        move()
        R.run_attention(ds)

    def apart():
        move()
        torch.cuda.synchronize()
        R.run_attention(ds)

    def together():
        move()
        R.run_attention(ds)

    for _ in range(4):
        fresh = [torch.randn_like(t) for t in (ds.k_pool, ds.v_pool)]
        results = []
        for run in (apart, together, graph.replay):
            for t, f in zip((ds.k_pool, ds.v_pool), fresh):
                t.copy_(f)
            ds.out.fill_(9.0)
            torch.cuda.synchronize()
            run()
            torch.cuda.synchronize()
            results.append([t.clone() for t in (ds.out, ds.k_pool, ds.v_pool)])
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other))
    assert B.pkv_check_device_status(ds.status) == 0
