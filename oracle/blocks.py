"""Oracle for block-sparse steps and trees of drafts -- TEST INFRASTRUCTURE.

Only ``tests/`` may import this module; the CUDA library never calls it and
shares no code with it. Plain float64 numpy, straight from the definitions:
bounds of a block's keys, the choice of blocks by them, and attention of rows
over any set of keys (``seen``), with the element-wise tolerance that
``oracle.scoremod`` derives (a row's visible keys need not be an interval
there: the terms are sums over the keys it sees).
"""

from __future__ import annotations

import numpy as np


def bounds(k):
    """[2, Hkv, D]: smallest and largest value of each channel over the rows of k [rows, Hkv, D]."""
    k = np.asarray(k, np.float64)
    return np.stack([k.min(0), k.max(0)])


def always(L, n, bs, keep_first, keep_last):
    """(blocks, first candidate, end of the candidates) of a slot of L keys whose last n rows are this step's."""
    end = max(0, (L - n) // bs - keep_last)
    return -(-L // bs), min(keep_first, end), end


def choose(q, lo, hi, L, bs, top, keep_first, keep_last):
    """Places of the blocks that one (segment, kv head) reads: q [n, group, D], lo and hi [blocks, D] in logical
    order (those of blocks that are always read are not looked at)."""
    q = np.asarray(q, np.float64)
    blocks, a, b = always(L, q.shape[0], bs, keep_first, keep_last)
    if blocks <= top:
        return list(range(blocks))
    fixed = list(range(a)) + list(range(b, blocks))
    rows = q.reshape(-1, q.shape[-1])
    score = [max(float(np.maximum(r * lo[j], r * hi[j]).sum()) for r in rows) for j in range(a, b)]
    best = sorted(range(b - a), key=lambda j: (-score[j], j))
    return sorted(fixed + [a + j for j in best[: top - len(fixed)]])


def tree_seen(parents, L):
    """[n, L] keys that each node of a tree sees: the history, its ancestors, itself."""
    n = len(parents)
    seen = np.zeros((n, L), bool)
    for i, p in enumerate(parents):
        if p >= 0:
            seen[i] = seen[p]
        else:
            seen[i, : L - n] = True
        seen[i, L - n + i] = True
    return seen


def attention(q, k, v, seen, scale, *, k_mag=None, v_mag=None):
    """(out [n, Hq, D], tolerance) of q over k, v [L, Hkv, D], row i seeing the keys seen[i]. The tolerance is that of
    ``oracle.scoremod.attention`` without a cap or a bias, its sums and maxima taken over the keys that a row sees."""
    n, hq, d = q.shape
    out, tol = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    keys = np.flatnonzero(seen.any(0))
    if not len(keys):
        return out, tol
    seen, k, v = seen[:, keys], k[keys], v[keys]
    k_mag = np.abs(k) if k_mag is None else k_mag[keys]
    for h in range(hq):
        g = h // (hq // k.shape[1])
        x = q[:, h] @ k[:, g].T * scale
        e = np.abs(q[:, h]) @ k_mag[:, g].T * scale * d * 2.0 ** -23 + np.abs(x) * 2.0 ** -22
        x = np.where(seen, x, -np.inf)
        top = x.max(1, keepdims=True)
        w = np.exp(x - np.where(np.isfinite(top), top, 0.0))
        total = w.sum(1, keepdims=True)
        u = w / np.where(total > 0, total, 1.0)
        o, size = u @ v[:, g], u @ np.abs(v[:, g])
        off = (u * e).sum(1, keepdims=True) + e.max(1, keepdims=True, where=seen, initial=0.0) \
            + (seen.sum(1, keepdims=True) + 16) * 2.0 ** -24 + 2.0 ** -22
        out[:, h] = o
        tol[:, h] = 1.02 * (2.0 ** -8 * (size + 2 * np.abs(o)) + off * (size + np.abs(o)))
        if v_mag is not None:
            tol[:, h] += 2.0 ** -19 * (u @ v_mag[keys, g])
    return out, tol
