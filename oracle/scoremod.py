"""Oracle for attention with modified scores -- TEST INFRASTRUCTURE.

Only ``tests/`` may import this module; the CUDA library never calls it and
shares no code with it. Plain float64 attention of one segment over its own
contiguous history, straight from the definition: scaled product, tanh cap,
distance bias, an interval of visible keys per row, softmax, zeros for a row
that sees nothing.

``attention`` also returns how far a kernel may be off at each element. With u
the weights, o = sum u v the result, A = sum u |v|:

* weights rounded to bfloat16 for the second product: 2^-8 each, so 2^-8 A, and
  as much of |o| again where the row sum adds unrounded weights;
* the result's own rounding: 2^-8 |o|;
* a logit off by e changes a weight by the factor 1 + e, and the row sum with
  it: e (A + |o|). e counts the fp32 accumulation of D products (D 2^-23 of
  sum |q k|), the tanh (2^-21 of the cap: two units in its last places) and
  the roundings of the logit and its exponent (2^-22 of its largest
  magnitude, the bias' own included);
* exponentials (2^-22) and sums of n weights in fp32: (n + 16) 2^-24 (A + |o|).

``k_mag`` / ``v_mag`` replace |k| / |v| in the accumulation terms where a pool's
codes enter the products with an offset that fp32 has to cancel (within 16
keys for values: 2^-19 of their magnitude).
"""

from __future__ import annotations

import numpy as np


def bounds(pos, L, *, window=0, key_begin=None, key_end=None):
    """Visible keys [lo, hi) of rows at ``pos`` (arrays); lo = hi = 0 for rows that see none."""
    pos = np.asarray(pos, np.int64)
    lo = np.zeros_like(pos) if key_begin is None else np.maximum(0, np.asarray(key_begin, np.int64))
    if window:
        lo = np.maximum(lo, pos - window + 1)
    hi = pos + 1 if key_end is None else np.minimum(L, np.asarray(key_end, np.int64))
    none = lo >= hi
    return np.where(none, 0, lo), np.where(none, 0, hi)


def attention(q, k, v, pos, lo, hi, scale, *, softcap=0.0, slopes=None, k_mag=None, v_mag=None):
    """(out [n, Hq, D], tolerance) in float64 of q [n, Hq, D] over k, v [L, Hkv, D]."""
    n, hq, d = q.shape
    L, hkv, _ = k.shape
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    j = np.arange(L)
    seen = (j >= np.asarray(lo)[:, None]) & (j < np.asarray(hi)[:, None])
    away = np.abs(np.asarray(pos)[:, None] - j).astype(np.float64)
    keys = j[seen.any(0)]
    if not len(keys):
        return out, tol
    seen, away = seen[:, keys], away[:, keys]
    offset = v_mag is not None
    for h in range(hq):
        g = h // (hq // hkv)
        kg, vg = k[keys, g], v[keys, g]
        x = q[:, h] @ kg.T * scale
        reach = np.abs(q[:, h]) @ (np.abs(kg) if k_mag is None else k_mag[keys, g]).T * scale
        e = reach * d * 2.0 ** -23
        if softcap:
            x = softcap * np.tanh(x / softcap)
            e = e + softcap * 2.0 ** -21
        bias = 0.0 if slopes is None else float(slopes[h]) * away
        e = e + (np.abs(x) + np.abs(bias)) * 2.0 ** -22
        x = np.where(seen, x - bias, -np.inf)
        top = x.max(1, keepdims=True)
        w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = w.sum(1, keepdims=True)
        u = w / np.where(total > 0, total, 1.0)
        o = u @ vg
        size = u @ np.abs(vg)
        off = (u * e).sum(1, keepdims=True) + e.max(1, keepdims=True, where=seen, initial=0.0) \
            + (seen.sum(1, keepdims=True) + 16) * 2.0 ** -24 + 2.0 ** -22
        # the weights' own errors stay with their values; the row sum's reach the whole result
        out[:, h] = o
        tol[:, h] = 1.02 * (2.0 ** -8 * (size + 2 * np.abs(o)) + off * (size + np.abs(o)))
        if offset:
            tol[:, h] += 2.0 ** -19 * (u @ v_mag[keys, g])
    return out, tol
