"""Rotary plan, phases and positions on the host, and the refusals of the rotation calls (no GPU)."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest

from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    libbuild.build()


@pytest.mark.parametrize("rot", [2, 4, 24, 64, 128])
def test_frequencies_of_each_scaling(rot):
    i = np.arange(rot // 2)
    f = 10000.0 ** (-2.0 * i / rot)
    p = B.pkv_rope_plan(rot)
    np.testing.assert_allclose(p.frequencies, f, rtol=1e-14)
    assert p.magnitude == 1.0 and p.phases.dtype == np.uint64
    np.testing.assert_allclose(B.pkv_rope_plan(rot, scaling=B.PKV_ROPE_LINEAR, factor=4.0).frequencies, f / 4,
                               rtol=1e-14)
    if rot > 2:
        g = (10000.0 * 8 ** (rot / (rot - 2))) ** (-2.0 * i / rot)
        np.testing.assert_allclose(B.pkv_rope_plan(rot, scaling=B.PKV_ROPE_NTK, factor=8.0).frequencies, g,
                                   rtol=1e-13)
        # the slowest pair is stretched by the whole factor
        assert g[-1] == pytest.approx(f[-1] / 8, rel=1e-12)
    kept = np.clip((4096 * f / (2 * math.pi) - 1) / 3, 0, 1)
    p = B.pkv_rope_plan(rot, scaling=B.PKV_ROPE_BY_PARTS, factor=8.0, original_len=4096, low=1.0, high=4.0)
    np.testing.assert_allclose(p.frequencies, f * (kept + (1 - kept) / 8), rtol=1e-13)


def test_yarn_by_hand():
    p = B.pkv_rope_plan(128, scaling=B.PKV_ROPE_YARN, factor=16.0, original_len=4096, low=1.0, high=32.0)
    f = 10000.0 ** (-np.arange(64) / 64.0)
    turns = 4096 * f / (2 * math.pi)
    a = math.floor(np.interp(-math.log(32), -np.log(turns), np.arange(64)))  # log(turns) is linear in the index
    b = math.ceil(np.interp(0.0, -np.log(turns), np.arange(64)))
    assert (a, b) == (20, 46)
    g = np.clip((np.arange(64) - a) / (b - a), 0, 1)
    np.testing.assert_allclose(p.frequencies, f * (1 - g) + f / 16 * g, rtol=1e-13)
    assert p.magnitude == pytest.approx(0.1 * math.log(16) + 1)
    assert np.array_equal(p.frequencies[:21], B.pkv_rope_plan(128).frequencies[:21])


@pytest.mark.parametrize("f", [0.0, 1.0, 1e-9, 0.3, 2 * math.pi, 7.5, -1.0, -1e-300, 100.0, 1e-4])
def test_phase_is_the_fraction_of_a_turn(f):
    """The phase equals f / 2 pi modulo a turn to the last bit that a double's quotient holds."""
    (phase,) = B.pkv_rope_phases([f])
    turns = Fraction(math.copysign(math.fmod(abs(f) / 6.283185307179586, 1.0), f)) * 2 ** 64
    assert abs(((int(phase) - turns + 2 ** 63) % 2 ** 64) - 2 ** 63) <= 1


def test_positions_of_a_lowered_step():
    got = B.pkv_plan_positions([0, 3, 3, 4], [2, 0, 1], [9, 5, 7])
    assert got.tolist() == [4, 5, 6, 4] and got.dtype == np.int32
    for cu, ss, cl in (([0, 8], [0], [7]), ([0, -1], [0], [7]), ([1, 2], [0], [7]), ([0, 2, 1], [0, 1], [7, 7])):
        with pytest.raises(B.PkvError):
            B.pkv_plan_positions(cu, ss, cl)
    with pytest.raises(B.PkvError) as e:
        B.pkv_plan_positions([0, 1], [1], [7])
    assert e.value.status == 2


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=-2), dict(rot_dim=64, base=1.0),
                                dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling=9),
                                dict(rot_dim=64, scaling=1, factor=0.0), dict(rot_dim=64, scaling=1, factor=math.nan),
                                dict(rot_dim=2, scaling=2, factor=2.0), dict(rot_dim=64, scaling=3, factor=2.0),
                                dict(rot_dim=64, scaling=4, factor=2.0, original_len=4096, low=4.0, high=4.0)])
def test_plan_refusals(kw):
    with pytest.raises(B.PkvError) as e:
        B.pkv_rope_plan(**kw)
    assert e.value.status == 1


def test_phases_refuse_infinities():
    with pytest.raises(B.PkvError):
        B.pkv_rope_phases([1.0, math.inf])


# Addresses that the calls below refuse, or would refuse, before any launch.
AT = 1 << 30


def _table(**kw):
    t = dict(phases=AT, rot_dim=128, interleaved=0, magnitude=1.0) | kw
    return B.RopeTable(t["phases"], t["rot_dim"], t["interleaved"], t["magnitude"])


def _write(table=None, **kw):
    a = dict(q=AT, qs=512, k=AT + (1 << 20), ks=256, v=AT + (2 << 20), vs=256, pos=AT + (3 << 20), sm=AT + (3 << 20),
             t=4, hq=4, hkv=2, d=128, out=AT + (4 << 20), os=512, kp=AT + (5 << 20), vp=AT + (6 << 20), nb=8, bs=16) | kw
    tb = ctypes.byref(table or _table())
    return B._lib().pkv_rope_cache_write(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["sm"], tb,
                                         a["t"], a["hq"], a["hkv"], a["d"], a["out"], a["os"], a["kp"], a["vp"],
                                         a["nb"], a["bs"], None, None)


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=AT + 8), dict(qs=1 << 60), dict(qs=510), dict(qs=504), dict(ks=128), dict(t=-1),
                                dict(hq=0), dict(hkv=0), dict(nb=0), dict(bs=0), dict(pos=None), dict(pos=AT + 2),
                                dict(sm=AT + 4), dict(kp=None), dict(vp=AT + 4), dict(out=None),
                                dict(out=AT + 16),               # shifted onto the input rows
                                dict(out=AT, os=1024),           # the input rows at another stride
                                dict(out=AT + (1 << 20)),        # onto the keys
                                dict(out=AT + (2 << 20) + 256)])  # onto the values
def test_cache_write_refusals(kw):
    assert _write(**kw) == 1


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=130), dict(rot_dim=5), dict(interleaved=2),
                                dict(phases=None), dict(phases=AT + 4), dict(magnitude=math.inf),
                                dict(magnitude=math.nan)])
def test_table_refusals(kw):
    assert _write(_table(**kw)) == 1
    assert B._lib().pkv_rope(AT, 512, AT, ctypes.byref(_table(**kw)), 4, 4, 128, AT + (1 << 20), 512, None) == 1


def test_unsupported_head_dim_and_empty_steps():
    assert _write(d=96) == 3
    assert _write(t=0) == B.PKV_OK
    assert B._lib().pkv_rope(AT, 512, AT, ctypes.byref(_table()), 0, 4, 128, AT, 512, None) == B.PKV_OK
    assert B._lib().pkv_rope(AT, 512, AT, ctypes.byref(_table()), 4, 4, 128, AT + 32, 512, None) == 1


@pytest.mark.parametrize("kw", [dict(scaling=B.PKV_ROPE_LINEAR, factor=5e-324), dict(scaling=B.PKV_ROPE_LINEAR, factor=1e-309),
                                dict(scaling=B.PKV_ROPE_NTK, factor=1e-200, rot_dim=4),
                                dict(scaling=B.PKV_ROPE_BY_PARTS, factor=5e-324, original_len=4096),
                                dict(scaling=B.PKV_ROPE_YARN, factor=5e-324, original_len=4096)])
def test_frequencies_past_the_largest_double_are_refused(kw):
    kw = dict(rot_dim=64) | kw
    n = kw["rot_dim"] // 2
    cfg = B.RopeConfig(kw["rot_dim"], kw["scaling"], 10000.0, kw["factor"], kw.get("original_len", 0), 1.0, 32.0)
    freqs, phases, mag = np.full(n, 7.0), np.full(n, 7, np.uint64), ctypes.c_float(7)
    assert B._lib().pkv_rope_plan(ctypes.byref(cfg), B._np_ptr(freqs), B._np_ptr(phases), ctypes.byref(mag)) == 1
    assert (freqs == 7).all() and (phases == 7).all() and mag.value == 7
    small = B.pkv_rope_plan(64, scaling=B.PKV_ROPE_LINEAR, factor=1e-300)  # far out, but finite
    assert np.isfinite(small.frequencies).all()


def test_a_bound_call_refuses_another_current_device(monkeypatch):
    """A call is bound on its tensors' device and runs on the current one: they must be the same at every call."""
    torch = pytest.importorskip("torch")
    current = [0]
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    table = _table()
    call = object.__new__(B._BoundCall)
    call._bind("pkv_rope", (AT, 512, AT, ctypes.byref(table), 0, 4, 128, AT + (1 << 20), 512), (table,),
               torch.device("cuda:0"), None)  # no tokens: nothing is launched
    call()
    current[0] = 1
    with pytest.raises(ValueError):
        call()
    current[0] = 0
    call()
