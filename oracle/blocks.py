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

from oracle import scoremod as SM


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
    """(out [n, Hq, D], tolerance) of q over k, v [L, Hkv, D], row i seeing the keys seen[i]."""
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for i in range(q.shape[0]):
        keys = np.flatnonzero(seen[i])
        if not len(keys):
            continue
        pick = lambda x: None if x is None else x[keys]  # noqa: E731
        o, t = SM.attention(q[i:i + 1], k[keys], v[keys], [len(keys) - 1], [0], [len(keys)], scale, k_mag=pick(k_mag),
                            v_mag=pick(v_mag))
        out[i], tol[i] = o[0], t[0]
    return out, tol
