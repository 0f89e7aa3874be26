"""Work lists and refusals of attention with modified scores, and pins of its oracle (no GPU)."""

import ctypes
import math
import subprocess
import sys

import numpy as np
import pytest

import oracle
from oracle import scoremod as SM
from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild
from tests.conftest import ROOT


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


def _masks(rng, segs):
    """Random bounds per packed row: whole, documents, prefixes, empty rows, out-of-range values."""
    total = sum(n for n, _ in segs)
    begin = rng.integers(-5, max(c for _, c in segs) + 5, total)
    end = rng.integers(-5, max(c for _, c in segs) + 5, total)
    begin[rng.random(total) < 0.4] = 0
    pos = np.concatenate([np.arange(c - n, c) for n, c in segs])
    keep = rng.random(total) < 0.5
    end[keep] = pos[keep] + 1
    return begin.astype(np.int32), end.astype(np.int32), pos


@pytest.mark.parametrize("seed", range(40))
def test_work_list_covers_what_the_rows_see(seed):
    rng = np.random.default_rng(seed)
    heads = [(4, 2, 64), (8, 8, 128), (40, 8, 128), (16, 1, 64)][seed % 4]
    bs = [16, 32, 64][seed % 3]
    segs = [(int(rng.integers(0, 20)) if rng.random() < 0.6 else int(rng.integers(20, 400)), 0) for _ in range(6)]
    segs = [(n, n + int(rng.integers(0 if n else 1, 2000))) for n, _ in segs]
    begin, end, pos = _masks(rng, segs)
    window = int(rng.choice([0, 0, 1, 100, 700]))
    use = rng.random(2) < 0.6
    kb, ke = (begin if use[0] else None), (end if use[1] else None)
    cu = np.concatenate([[0], np.cumsum([n for n, _ in segs])]).astype(np.int32)
    slots = rng.permutation(9)[:6].astype(np.int32)
    ctx = np.zeros(9, np.int32)
    ctx[slots] = [c for _, c in segs]
    mb = -(-max(c for _, c in segs) // bs)
    work, info = B.pkv_plan_work_mod(cu, slots, ctx, max_slots=9, max_blocks_per_slot=mb, block_size=bs,
                                     num_q_heads=heads[0], num_kv_heads=heads[1], head_dim=heads[2], window=window,
                                     key_begin=kb, key_end=ke)
    assert info.modified == 1
    items = work[:info.work_words].reshape(-1, 4)
    nd, npf, nc, ns = (info.num_decode_items, info.num_prefill_items, info.num_combine_items, info.num_scratch_items)
    dec, pre, comb, scr = np.split(items, np.cumsum([nd, npf, nc]))
    assert len(scr) == ns
    group = heads[0] // heads[1]
    partials = set()
    for s, (n, L) in enumerate(segs):
        rows = slice(cu[s], cu[s + 1])
        lo, hi = SM.bounds(pos[rows], L, window=window, key_begin=None if kb is None else kb[rows],
                           key_end=None if ke is None else ke[rows])
        live = lo < hi
        u = (int(lo[live].min()), int(hi[live].max())) if live.any() else (0, 0)
        mine = dec[dec[:, 0] == s]
        if n == 0:
            assert not len(mine) and not (pre[:, 0] == s).any()
        elif n <= max(1, 16 // group):
            assert (mine[:, 1] == slots[s]).all()
            words = mine[:, 2].astype(np.int64) & 0xFFFFFFFF
            span, first, count = words & 0x7FFFFF, (words >> 23) & 15, words >> 27
            if not live.any():
                assert len(mine) == 1 and count[0] == 0 and mine[0, 3] == -1
                continue
            k0 = span * 256 + first * 16
            order = np.argsort(k0)
            # back to back from the first sub-tile with a visible key to the last, cut at multiples of the span: the
            # shortest that leaves at most 64 spans and 8 x 152 tasks with all nine slots as long, 256 keys at most
            cut = next((k for k in (64, 128) if -(-(u[1] - u[0]) // k) <= min(64, 8 * 152 / (9 * heads[1]))), 256)
            subs = -(-u[1] // 16) - u[0] // 16
            assert (len(mine) == 1) == (subs <= (16 if cut == 256 else 8) or u[0] // cut == (u[1] - 1) // cut)
            assert k0[order][0] == u[0] // 16 * 16
            assert (k0 + count * 16)[order][-1] == -(-u[1] // 16) * 16
            assert ((k0 + count * 16)[order][:-1] == k0[order][1:]).all()
            assert (k0[order][1:] % cut == 0).all() and (count >= 1).all() and (count <= 16).all()
            assert len(mine) == 1 or ((first * 16) % cut + count * 16 <= cut).all()
            merges = comb[comb[:, 0] == s]
            if len(mine) == 1:
                assert mine[0, 3] == -1 and not len(merges)
            else:
                assert len(merges) == n
                base = mine[order][:, 3]
                assert (np.diff(base) == n).all()
                for m in merges:
                    row = (m[2] >> 16) & 255
                    assert m[2] & 0xFFFF == len(mine) and ((m[2] >> 24) & 255) + 1 == n and m[3] == base[0] + row
                got = {int(b) + i for b in base for i in range(n)}
                assert not got & partials
                partials |= got
        else:
            step = 2 if heads[2] == 128 else 1
            tiles = -(-n // (128 // group))
            got = pre[pre[:, 0] == s]
            assert sorted(got[:, 2]) == list(range(0, tiles, step))
            (sc,) = scr[scr[:, 0] == s]
            assert sc[1] == u[0] // bs and sc[1] + sc[3] == -(-u[1] // bs)
    assert partials == set(range(info.num_partials))


def test_causal_list_matches_the_plain_one():
    """Without any bound, in a table too wide for shorter spans, the spans, tiles and merges are pkv_plan_work's."""
    cu, slots, ctx = [0, 1, 4, 204, 205], [0, 1, 2, 3], [700, 5, 900, 256] + [0] * 124
    shape = dict(max_slots=128, max_blocks_per_slot=64, block_size=16, num_q_heads=32, num_kv_heads=8, head_dim=128)
    w0, i0 = B.pkv_plan_work(cu, slots, ctx, **shape)
    w1, i1 = B.pkv_plan_work_mod(cu, slots, ctx, **shape)
    for f in ("num_decode_items", "num_prefill_items", "num_combine_items", "num_partials", "work_words",
              "workspace_bytes", "workspace_bytes_q8", "decode_rows_max", "scratch_blocks"):
        assert getattr(i0, f) == getattr(i1, f), f
    assert i0.modified == 0 and i1.modified == 1
    a, b = w0.reshape(-1, 4), w1.reshape(-1, 4)
    nd = i0.num_decode_items
    assert sorted(map(tuple, a[nd:-1, :].tolist())) == sorted(map(tuple, b[nd:-1, :].tolist()))
    assert sorted((int(s), int(z) & 0x7FFFFF) for s, _, z, _ in b[:nd]) == sorted((int(s), int(z)) for s, _, z, _ in a[:nd])


AT = 1 << 30


def _info(modified=1):
    _, info = (B.pkv_plan_work_mod if modified else B.pkv_plan_work)(
        [0, 1], [0], [40], max_slots=1, max_blocks_per_slot=4, block_size=16, num_q_heads=4, num_kv_heads=2, head_dim=64)
    return info


def _call(fn="pkv_attention_mod", mod=None, info=None, null=False, d=64):
    m = B.ScoreModArgs(*(mod or (0.0, 0, None, None, None)))
    pool = (AT, AT) if fn == "pkv_attention_mod" else (AT,) * 4
    return getattr(B._lib(), fn)(AT, AT, 1, 1, AT, AT, AT, 1, 4, 16, *pool, 8, 4, 2, d, 0.0,
                                 None if null else ctypes.byref(m), AT, ctypes.byref(info or _info()), AT, None, 0, None,
                                 None)


@pytest.mark.parametrize("fn", ["pkv_attention_mod", "pkv_attention_mod_q8"])
@pytest.mark.parametrize("mod", [(-1.0, 0, None, None, None), (math.inf, 0, None, None, None),
                                 (math.nan, 0, None, None, None), (2.0 ** -21, 0, None, None, None),
                                 (4097.0, 0, None, None, None), (1e38, 0, None, None, None), (0.0, -1, None, None, None),
                                 (0.0, 0, AT + 1, None, None), (0.0, 0, None, AT + 2, None), (0.0, 0, None, None, AT + 3)])
def test_refused_modifications(fn, mod):
    assert _call(fn, mod) == 1


def test_refused_lists_and_shapes():
    assert _call(null=True) == 1
    assert _call(info=_info(modified=0)) == 1  # a plain list
    assert _call("pkv_attention_mod_q4") == 3  # head_dim 64
    assert _call(d=96) == 3
    info = _info()
    info.work_words -= 4
    assert _call(info=info) == 1
    # and a modified list is refused by the plain call
    L = B._lib()
    assert L.pkv_attention(AT, AT, 1, 1, AT, AT, AT, 1, 4, 16, AT, AT, 8, 4, 2, 64, 0.0, AT, ctypes.byref(_info()), AT,
                           None, 0, None, None) == 1
    assert L.pkv_attention_q8(AT, AT, 1, 1, AT, AT, AT, 1, 4, 16, AT, AT, AT, AT, 8, 4, 2, 64, 0.0, AT,
                              ctypes.byref(_info()), AT, None, 0, None, None) == 1


def test_plan_refusals():
    shape = dict(max_slots=1, max_blocks_per_slot=4, block_size=16, num_q_heads=4, num_kv_heads=2, head_dim=64)
    with pytest.raises(B.PkvError):
        B.pkv_plan_work_mod([0, 1], [0], [40], window=-1, **shape)
    with pytest.raises(ValueError):
        B.pkv_plan_work_mod([0, 2], [0], [40], key_begin=[0], **shape)
    with pytest.raises(B.PkvError):
        B.pkv_plan_work_mod([0, 2], [0], [1], **shape)
    assert B._lib().pkv_plan_work_mod(None, 0, None, None, 1, 1, 16, 4, 2, 64, None, None, 0, None) == 1


# ---- pins of the oracle -------------------------------------------------------

def _draw(seed, n, L, hq=4, hkv=2, d=64):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((n, hq, d)), rng.standard_normal((L, hkv, d)), rng.standard_normal((L, hkv, d))


def test_oracle_without_modification_is_the_plain_oracle():
    from continuous_batching_paged_pkv_gb300 import workloads as W

    q, k, v = (W.f32_to_bf16_bits(x.astype(np.float32)) for x in _draw(0, 9, 40))
    oracle.build()
    ref = oracle.attention_dense(q, k, v, 0.125)
    pos = np.arange(31, 40)
    got, tol = SM.attention(*(W.bf16_bits_to_f32(x) for x in (q, k, v)), pos, *SM.bounds(pos, 40), 0.125)
    np.testing.assert_allclose(got, ref, rtol=1e-12, atol=1e-12)
    assert (tol > 0).all() and tol.max() < 2e-2


def test_oracle_closed_forms():
    q, k, v = _draw(1, 3, 20)
    pos = np.array([17, 18, 19])
    # a window of one key gives that key's value; no key gives zeros
    out, _ = SM.attention(q, k, v, pos, *SM.bounds(pos, 20, window=1), 0.1)
    np.testing.assert_allclose(out, np.repeat(v[17:20], 2, axis=1))
    out, tol = SM.attention(q, k, v, pos, *SM.bounds(pos, 20, key_end=[0, 5, -3]), 0.1)
    assert (out[[0, 2]] == 0).all() and (tol[[0, 2]] == 0).all() and (out[1] != 0).any()
    # equal scores: the weights are the biases' own, geometric in the distance
    out, _ = SM.attention(np.zeros_like(q), k, v, pos, *SM.bounds(pos, 20), 0.1, slopes=np.full(4, math.log(2)))
    w = 0.5 ** (17 - np.arange(18))
    np.testing.assert_allclose(out[0, 0], (w / w.sum()) @ v[:18, 0])
    # a cap far below the scores' size leaves two levels, a large one nothing
    big = SM.attention(q * 1e4, k, v, pos, *SM.bounds(pos, 20), 1.0, softcap=1e-3)[0]
    np.testing.assert_allclose(big[2, 0], v[:, 0].mean(0), rtol=2e-3, atol=2e-3)
    none, cap = (SM.attention(q, k, v, pos, *SM.bounds(pos, 20), 0.1, softcap=c)[0] for c in (0.0, 1e6))
    np.testing.assert_allclose(cap, none, rtol=1e-9)
    # a prefix is seen from before its end
    lo, hi = SM.bounds([2, 9], 12, key_end=[6, 10], key_begin=[-4, 8])
    assert lo.tolist() == [0, 8] and hi.tolist() == [6, 10]


@pytest.mark.parametrize("head_dim", [64, 128])
def test_a_gap_between_rows_is_covered(head_dim):
    """Rows whose intervals leave a gap: spans and widened blocks run from the first to the last key that one sees."""
    shape = dict(max_slots=2, max_blocks_per_slot=200, block_size=16, num_q_heads=8, num_kv_heads=2, head_dim=head_dim)
    begin = np.concatenate([[33, 1000], np.where(np.arange(60) < 30, 100, 2000)])
    end = np.concatenate([[100, 1100], np.where(np.arange(60) < 30, 150, 2050)])
    work, info = B.pkv_plan_work_mod([0, 2, 62], [0, 1], [1500, 2500], key_begin=begin, key_end=end, **shape)
    items = work[:info.work_words].reshape(-1, 4)
    words = items[:info.num_decode_items, 2].astype(np.int64) & 0xFFFFFFFF
    k0 = (words & 0x7FFFFF) * 256 + ((words >> 23) & 15) * 16
    keys = sorted(zip(k0.tolist(), (k0 + (words >> 27) * 16).tolist()))
    assert keys[0][0] == 32 and keys[-1][1] == 1104
    assert all(a[1] == b[0] for a, b in zip(keys, keys[1:]))
    (scratch,) = items[len(items) - info.num_scratch_items:]
    assert scratch[1] == 100 // 16 and scratch[1] + scratch[3] == -(-2050 // 16)


def test_bounds_and_windows_that_32_bits_do_not_hold_are_refused():
    """ "No bound" written as 2^31 or more must not wrap to a row that sees nothing, nor a huge window to a small one."""
    shape = dict(max_slots=1, max_blocks_per_slot=4, block_size=16, num_q_heads=4, num_kv_heads=2, head_dim=64)
    for value in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 63 - 1):
        for name in ("key_begin", "key_end"):
            for kind in (np.int64, list):
                a = np.full(2, value, np.int64)
                with pytest.raises(ValueError):
                    B.pkv_plan_work_mod([0, 2], [0], [40], **{name: a if kind is np.int64 else a.tolist()}, **shape)
    for value in (2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 2.5):
        with pytest.raises(ValueError):
            B.pkv_plan_work_mod([0, 2], [0], [40], window=value, **shape)
        with pytest.raises(ValueError):
            B.ScoreMod(window=value).marshal(4, 2)
    for a in (np.array([0.0, 1.0]), np.array([np.inf, 0.0]), np.array([True, False])):
        with pytest.raises(ValueError):
            B.pkv_plan_work_mod([0, 2], [0], [40], key_end=a, **shape)
    most, least = 2 ** 31 - 1, -2 ** 31
    wide, _ = B.pkv_plan_work_mod([0, 2], [0], [40], key_begin=[least] * 2, key_end=np.full(2, most), window=most, **shape)
    same, _ = B.pkv_plan_work_mod([0, 2], [0], [40], key_end=[40, 40], **shape)
    assert np.array_equal(wide, same)
    assert B.ScoreMod(window=most).marshal(4, 2).window == most


def test_arrays_shorter_than_their_counts_are_refused():
    """seq_slot has one entry per segment, context_lens one per slot: the planner would read past shorter ones."""
    shape = dict(max_blocks_per_slot=4, block_size=16, num_q_heads=4, num_kv_heads=2, head_dim=64)
    for cu, ss, cl, slots in (([0, 1, 2], [0], [40, 40], 2), ([0, 1], [0], [40], 2), ([0, 1], [3], [40, 40], 4),
                              ([], [], [40], 1)):
        with pytest.raises(ValueError):
            B.pkv_plan_work_mod(cu, ss, cl, max_slots=slots, **shape)
    B.pkv_plan_work_mod([0, 1], [0, 1], [40, 40, 40], max_slots=2, **shape)  # longer ones are not
    for cu, ss in (([], []), ([0, 1], []), ([0, 1], [0, 1])):
        with pytest.raises(ValueError):
            B.pkv_plan_positions(cu, ss, [40, 40])


@pytest.mark.parametrize("fn", ["pkv_plan_work", "pkv_plan_work_mod"])
def test_sizes_without_host_memory_are_refused(fn):
    """A planner that cannot allocate its lists returns a status; an exception through the C entry would end the process."""
    code = f"""
import ctypes, resource
import numpy as np
from continuous_batching_paged_pkv_gb300 import binding as B
L = B._lib()
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (256 << 20), used + (256 << 20)))
cu, ss, cl = (np.array(a, np.int32) for a in ([0, 1], [0], [40]))
mod, info, work = B.ScoreModArgs(), B.WorkInfo(), np.zeros(64, np.int32)
mods = (ctypes.byref(mod),) if {fn!r} == "pkv_plan_work_mod" else ()
call = lambda slots: getattr(L, {fn!r})(B._np_ptr(cu), 1, B._np_ptr(ss), B._np_ptr(cl), slots, 4, 16, 4, 2, 64, *mods,
                                        B._np_ptr(work), 64, ctypes.byref(info))
print(call(2 ** 31 - 1), call(1))
"""
    done = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert (done.returncode, done.stdout.split()) == (0, ["1", "0"]), done
