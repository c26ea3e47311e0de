"""Attention weights and eviction by them in fp64 — the oracle.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``): never imported by the library.

* ``attention_weights``: the softmax weights of one decode step, summed over the query
  heads of each KV group — what the library adds to its running sums.
* ``select``: of a sequence's ``t`` tokens ``n = min(keep, t)`` stay for a KV head: the
  last ``r = min(recent, n)``, the first ``f = min(first, n - r)`` and the rest by their
  sums, larger first, equal ones by the lower position (NaN counts as -infinity).
* ``gather``: rows of the kept positions, in ascending order, into a new block table.
"""
from __future__ import annotations

import numpy as np


def attention_weights(q, keys, scale) -> np.ndarray:
    """``q [Hq, D]``, ``keys [Hkv, t, D]`` -> weights ``[Hkv, t]`` summed over each group."""
    q, keys = np.asarray(q, dtype=np.float64), np.asarray(keys, dtype=np.float64)
    Hkv, t, _ = keys.shape
    G = q.shape[0] // Hkv
    sc = np.float64(np.float32(scale))
    out = np.zeros((Hkv, t))
    for h in range(q.shape[0]):
        x = sc * (keys[h // G] @ q[h])
        w = np.exp(x - x.max())
        out[h // G] += w / w.sum()
    return out


def select(sums, t, keep, first=0, recent=0) -> np.ndarray:
    """Ascending kept positions of one row of sums."""
    n = max(0, min(keep, t))
    r = min(recent, n)
    f = min(first, n - r)
    between = range(f, t - r)
    key = {p: (-np.inf if np.isnan(sums[p]) else float(sums[p])) for p in between}
    best = sorted(between, key=lambda p: (-key[p], p))[:n - r - f]
    return np.array(sorted(list(range(f)) + best + list(range(t - r, t))), dtype=np.int64)


def gather(k_cache, v_cache, table, kept, new_table, head, v_pos=None) -> None:
    """Move one KV head's kept rows in place; ``v_pos``: the byte order of transposed tiles."""
    B = k_cache.shape[2]
    k, v = k_cache.copy(), v_cache.copy()
    for j, p in enumerate(kept):
        src, dst = int(table[p // B]), int(new_table[j // B])
        k_cache[dst, head, j % B] = k[src, head, p % B]
        if v_pos is None:
            v_cache[dst, head, j % B] = v[src, head, p % B]
        else:
            v_cache[dst, head, :, v_pos[j % B]] = v[src, head, :, v_pos[p % B]]
