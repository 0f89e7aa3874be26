"""Rotary positions on the GPU against the rotation in 64 bits.

Tolerance of a rotated element m (a cos t - b sin t), derived: half a bf16 step of the result (2^-8 of it), and in
fp32 (|a| + |b|) m times the angle's error (pi 2^-25 from its rounding to 24 bits, 2 pi 2^-33 from the 32 bits kept,
2^-52 |t| for the frequency's and the phase's doubles), sincospi's two units in the last place (2^-23) and three
roundings (2^-24 each): below (|a| + |b|) m (2^-20 + 2^-52 |t|).
"""

import numpy as np
import pytest

from continuous_batching_paged_pkv_gb300 import binding as B
from continuous_batching_paged_pkv_gb300 import build as libbuild

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    libbuild.build()


def _turned(x, positions, plan, interleaved):
    """(rotated rows, tolerance) of bf16 rows x [T, H, D] in float64."""
    x = x.double().cpu().numpy()
    rot = plan.rot_dim
    t = positions.cpu().numpy().astype(np.float64)[:, None, None] * plan.frequencies
    c, s = np.cos(t) * plan.magnitude, np.sin(t) * plan.magnitude
    i = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    a, b = x[..., i[0]], x[..., i[1]]
    out, tol = x.copy(), np.zeros_like(x)
    out[..., i[0]], out[..., i[1]] = a * c - b * s, a * s + b * c
    slack = (np.abs(a) + np.abs(b)) * plan.magnitude * (2.0 ** -20 + 2.0 ** -52 * np.abs(t))
    for j in i:
        tol[..., j] = np.abs(out[..., j]) * 2.0 ** -8 + slack
    return out, tol


def _check(got, x, positions, plan, interleaved, what):
    want, tol = _turned(x, positions, plan, interleaved)
    off = np.abs(got.double().cpu().numpy() - want) - tol
    assert (off <= 0).all(), f"{what}: {off.max():.3e} beyond the tolerance at {np.unravel_index(off.argmax(), off.shape)}"


def _step(seed, t, hq, hkv, d, bs, fused, extra=3, high=1 << 20):
    g = torch.Generator("cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)

    if fused:
        q, k, v = normal(t, hq + 2 * hkv, d).split([hq, hkv, hkv], 1)
    else:
        q, k, v = normal(t, hq, d), normal(t, hkv, d), normal(t, hkv, d)
    blocks = -(-t // bs) + extra
    rows = torch.randperm(blocks * bs, generator=g, device="cuda")[:t]
    pos = torch.randint(0, high, (t,), generator=g, device="cuda", dtype=torch.int32)
    return q, k, v, rows, pos, normal(blocks, hkv, bs, d), normal(blocks, hkv, bs, d)


PLANS = {"plain": {}, "linear": dict(scaling=B.PKV_ROPE_LINEAR, factor=4.0),
         "yarn": dict(scaling=B.PKV_ROPE_YARN, factor=16.0, original_len=4096)}


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("t,hq,hkv,d,rot,bs,fused,plan", [
    (1, 4, 2, 64, 64, 16, False, "plain"), (3, 1, 1, 128, 128, 16, True, "yarn"), (257, 40, 8, 128, 128, 16, True, "linear"),
    (33, 14, 2, 64, 32, 32, False, "plain"), (130, 32, 8, 128, 64, 64, True, "yarn"), (5, 5, 5, 128, 2, 16, False, "plain"),
    (7, 6, 3, 128, 118, 16, True, "plain"), (19, 3, 1, 64, 24, 16, False, "linear"), (9, 2, 1, 64, 8, 16, True, "plain"),
    (66, 7, 7, 128, 40, 16, False, "yarn"), (2111, 16, 1, 64, 48, 16, False, "plain")])
def test_rotation_and_append(t, hq, hkv, d, rot, bs, fused, plan, interleaved):
    q, k, v, rows, pos, kp, vp = _step(t + rot, t, hq, hkv, d, bs, fused)
    rows = rows.clone()
    rows[t // 2::7] = -1  # tokens whose key and value are not kept
    p = B.pkv_rope_plan(rot, **PLANS[plan])
    kp0, vp0, q0 = kp.clone(), vp.clone(), q.clone()
    out = torch.full((t, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(rot_dim=rot, interleaved=interleaved, magnitude=p.magnitude)
    B.pkv_rope_cache_write(q, k, v, pos, p.phase_tensor("cuda"), rows, out, kp, vp, device_status=status, **args)
    assert B.pkv_check_device_status(status) == 0
    assert torch.equal(q, q0)
    _check(out, q, pos, p, interleaved, "queries")
    kept = rows >= 0
    at = rows[kept]
    _check(kp[at // bs, :, at % bs], k[kept], pos[kept], p, interleaved, "keys")
    assert torch.equal(vp[at // bs, :, at % bs], v[kept])
    kp0[at // bs, :, at % bs] = kp[at // bs, :, at % bs]
    vp0[at // bs, :, at % bs] = v[kept]
    assert torch.equal(kp, kp0) and torch.equal(vp, vp0)  # every other row as it was
    # rows to rows gives the same bits, into other rows and in place
    alone = torch.empty_like(out)
    B.pkv_rope(q, pos, p.phase_tensor("cuda"), alone, **args)
    assert torch.equal(alone, out)
    keys = torch.empty(t, hkv, d, dtype=torch.bfloat16, device="cuda")
    B.pkv_rope(k, pos, p.phase_tensor("cuda"), keys, **args)
    assert torch.equal(keys[kept], kp[at // bs, :, at % bs])
    B.pkv_rope_cache_write(q, k, v, pos, p.phase_tensor("cuda"), rows, q, kp, vp, **args)
    assert torch.equal(q, out)


@pytest.mark.parametrize("position", [0, -1, -123457, 131071, 16777217, 2 ** 31 - 1, -2 ** 31])
def test_far_positions(position):
    q, k, v, rows, pos, kp, vp = _step(3, 4, 2, 1, 128, 16, False)
    pos.fill_(position)
    p = B.pkv_rope_plan(128)
    out = torch.empty_like(q)
    B.pkv_rope(q, pos, p.phase_tensor("cuda"), out, rot_dim=128)
    _check(out, q, pos, p, False, f"position {position}")


def test_columns_of_one_buffer():
    """From one column range of a buffer into another of the same rows."""
    g = torch.Generator("cuda").manual_seed(5)
    buf = torch.randn(50, 12, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    keep = buf.clone()
    pos = torch.arange(50, dtype=torch.int32, device="cuda")
    p = B.pkv_rope_plan(64)
    B.pkv_rope(buf[:, 1:5], pos, p.phase_tensor("cuda"), buf[:, 6:10], rot_dim=64)
    _check(buf[:, 6:10], keep[:, 1:5], pos, p, False, "columns")
    for s in (slice(0, 6), slice(10, 12)):
        assert torch.equal(buf[:, s], keep[:, s])
    with pytest.raises(B.PkvError):
        B.pkv_rope(buf[:, 1:5], pos, p.phase_tensor("cuda"), buf[:, 4:8], rot_dim=64)


def test_bad_slots_are_skipped_and_reported():
    q, k, v, rows, pos, kp, vp = _step(9, 20, 4, 2, 128, 16, True)
    rows = rows.clone()
    rows[3] = kp.shape[0] * 16
    rows[11] = 2 ** 40
    p = B.pkv_rope_plan(128)
    kp0 = kp.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.empty(20, 4, 128, dtype=torch.bfloat16, device="cuda")
    B.pkv_rope_cache_write(q, k, v, pos, p.phase_tensor("cuda"), rows, out, kp, vp, rot_dim=128, device_status=status)
    assert B.pkv_check_device_status(status) == 1
    _check(out, q, pos, p, False, "queries")
    changed = (kp != kp0).any(-1).any(1).sum().item()
    assert changed == 18


def test_infinities_stay_in_their_pairs():
    q, k, v, rows, pos, kp, vp = _step(13, 2, 2, 1, 64, 16, False)
    q[0, 0, 3] = float("inf")
    q[1, 1, 40] = float("nan")
    p = B.pkv_rope_plan(64)
    out = torch.empty_like(q)
    B.pkv_rope(q, pos, p.phase_tensor("cuda"), out, rot_dim=64)
    bad = (~torch.isfinite(out)).nonzero().tolist()
    assert bad == [[0, 0, 3], [0, 0, 35], [1, 1, 8], [1, 1, 40]]


def test_another_stream_and_a_replayed_graph():
    q, k, v, rows, pos, kp, vp = _step(21, 64, 8, 2, 128, 16, True)
    p = B.pkv_rope_plan(128, **PLANS["yarn"])
    ph = p.phase_tensor("cuda")
    out, other = torch.zeros(64, 8, 128, dtype=torch.bfloat16, device="cuda"), None
    call = B.RopeCacheWriteCall(q, k, v, pos, ph, rows, out, kp, vp, rot_dim=128, magnitude=p.magnitude)
    call()
    torch.cuda.synchronize()
    want, wk = out.clone(), kp.clone()
    out.zero_()
    kp.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # a bound call runs on the stream that is current at the call
        call()
        other = out.clone()
    side.synchronize()
    assert torch.equal(other, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    q2 = torch.randn_like(q)
    q.copy_(q2)
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q2, pos, p, False, "replayed")
    at = rows
    assert torch.equal(kp[at // 16, :, at % 16], wk[at // 16, :, at % 16])


def test_tensors_are_checked():
    q, k, v, rows, pos, kp, vp = _step(2, 4, 2, 1, 64, 16, False)
    ph = B.pkv_rope_plan(64).phase_tensor("cuda")
    out = torch.empty_like(q)
    for bad in (lambda: B.pkv_rope(q.float(), pos, ph, out, rot_dim=64), lambda: B.pkv_rope(q, pos.long(), ph, out, rot_dim=64),
                lambda: B.pkv_rope(q, pos, ph[:-1].clone(), out, rot_dim=64),
                lambda: B.pkv_rope(q.transpose(1, 2), pos, ph, out.transpose(1, 2), rot_dim=64),
                lambda: B.pkv_rope(q, pos, ph, out[:, :1], rot_dim=64), lambda: B.pkv_rope(q, pos[:2], ph, out, rot_dim=64),
                lambda: B.pkv_rope(q, pos, ph.cpu(), out, rot_dim=64),
                lambda: B.pkv_rope_cache_write(q, k, v[:, :, :32], pos, ph, rows, out, kp, vp, rot_dim=64),
                lambda: B.pkv_rope_cache_write(q, k, v, pos, ph, rows, out, kp, vp[:2], rot_dim=64)):
        with pytest.raises(ValueError):
            bad()
