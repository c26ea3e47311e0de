"""Operators of a speculative step in fp64 — the oracle.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``): never imported by the library.

A sequence's cache ends in ``c`` drafted tokens, a chain or a tree: drafted token ``i``
follows its parent, a drafted token before it, or the end of the context (parent -1).

* ``tree_attention``: every drafted token attends to the context and to the drafted tokens
  that it sees, ``softmax(x) V`` with ``x = scale q . k``, capped (``cap tanh(x / cap)``), with
  a bias ``slope (pos(k) - pos(q))`` and a window ``pos(q) - pos(k) < window``.
* ``norm_rotate``: each head over the root of its mean square, times a weight, then turned
  pair by pair to the position on the pair's axis.
* ``adjust_logits``: penalties for tokens that came before, biases, a mask of allowed tokens.
* ``commit``: the rows of the accepted path moved to the front.
"""
from __future__ import annotations

import numpy as np

from .paged_attention import gather_sequence


def tree_masks(parents):
    """(seen bool [c, c], depths [c]) of one tree: a token sees itself and its ancestors."""
    c = len(parents)
    seen, depth = np.zeros((c, c), dtype=bool), np.zeros(c, dtype=np.int64)
    for i in range(c):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = int(parents[j])
        depth[i] = seen[i].sum() - 1
    return seen, depth


def words(seen, count) -> np.ndarray:
    """int32 words [c, count] of a boolean [c, c]."""
    c = seen.shape[0]
    bits = np.zeros((c, count * 32), dtype=np.uint8)
    bits[:, :seen.shape[1]] = seen
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, scale, seen=None,
                   depths=None, cap=0.0, slopes=None, window=0):
    """fp64 (out [T, Hq, D], spread [T, Hq, D], size [T, Hq]): spread is sum_p w_p |V_p|, size
    the largest sum of |terms| of a visible score (scale |q| . |k| and the bias's parts).
    ``seen``: list of boolean [c, c] per sequence, or None (j <= i)."""
    q = np.asarray(q, dtype=np.float64)
    T, Hq, D = q.shape
    Hkv = np.asarray(k_cache).shape[1]
    G = Hq // Hkv
    sc = np.float64(np.float32(scale))
    qs = np.asarray(query_start, dtype=np.int64)
    out, spread, size = np.zeros((T, Hq, D)), np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for s in range(len(qs) - 1):
        t, c = int(context_lens[s]), int(qs[s + 1] - qs[s])
        if c == 0:
            continue
        base = t - c
        d = np.arange(c) if depths is None else np.maximum(0, np.asarray(depths)[qs[s]:qs[s + 1]])
        pos = np.concatenate([np.arange(base), base + d])
        ok = np.ones((c, t), dtype=bool)
        ok[:, base:] = np.tri(c, dtype=bool) if seen is None else seen[s]
        far = (base + d)[:, None] - pos[None, :]
        if window:
            ok &= far < window
        for g in range(Hkv):
            K = gather_sequence(k_cache, block_tables[s], t, g)
            V = gather_sequence(v_cache, block_tables[s], t, g)
            with np.errstate(invalid="ignore"):
                rough = np.abs(np.nan_to_num(K))
            for h in range(g * G, (g + 1) * G):
                x = np.zeros((c, t))
                big = np.zeros((c, t))
                for i in range(c):
                    v = ok[i]
                    x[i, v] = sc * (K[v] @ q[qs[s] + i, h])
                    big[i, v] = abs(sc) * (rough[v] @ np.abs(q[qs[s] + i, h]))
                if cap:
                    x = cap * np.tanh(x / cap)
                    big = big + cap
                if slopes is not None:
                    m = np.float64(np.float32(slopes[h]))
                    x = x - m * far
                    big = big + np.abs(m * far)
                for i in range(c):
                    v = ok[i]
                    if not v.any():
                        continue
                    w = np.exp(x[i, v] - x[i, v].max())
                    w /= w.sum()
                    out[qs[s] + i, h] = w @ V[v]
                    spread[qs[s] + i, h] = w @ np.abs(V[v])
                    size[qs[s] + i, h] = big[i, v].max()
    return out, spread, size


def norm_rotate(x, weight, eps, positions, pair_axes, inv_freq, interleaved=False) -> np.ndarray:
    """``x [T, H, D]`` normed (``eps`` None: not) and turned; ``positions [A, T]``."""
    y = np.array(x, dtype=np.float64)
    if eps is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + np.float64(np.float32(eps)))
        if weight is not None:
            y = y * np.asarray(weight, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = len(f)
    pos = np.asarray(positions, dtype=np.float64)
    z = np.exp(1j * pos[np.asarray(pair_axes)].T * f)[:, None, :]
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    w = (y[..., one] + 1j * y[..., two]) * z
    y[..., one], y[..., two] = w.real, w.imag
    return y


def adjust_logits(logits, history, history_lens, prompt_lens, rows, repetition=None, frequency=None,
                  presence=None, path=None, bias_tokens=None, bias_values=None, allowed=None):
    """fp64 logits of rows ``rows[r]`` = the request of row r (-1: left alone); ``allowed``:
    boolean [T, V]."""
    y = np.array(logits, dtype=np.float64)
    T, V = y.shape
    for r in range(T):
        s = rows[r]
        if s < 0:
            continue
        n = min(max(int(history_lens[s]), 0), history.shape[1])
        p = 0 if prompt_lens is None else int(prompt_lens[s])
        count, seen = {}, set()
        for at in range(n):
            v = int(history[s, at])
            if not 0 <= v < V:
                continue
            seen.add(v)
            if at >= p:
                count[v] = count.get(v, 0) + 1
        for v in ([] if path is None else path[r]):
            if 0 <= int(v) < V:
                seen.add(int(v))
                count[int(v)] = count.get(int(v), 0) + 1
        rep = 1.0 if repetition is None else float(repetition[s])
        for v in seen:
            y[r, v] = y[r, v] / rep if y[r, v] > 0 else y[r, v] * rep
        for v, k in count.items():
            y[r, v] -= 0.0 if frequency is None else float(frequency[s]) * k
            y[r, v] -= 0.0 if presence is None else float(presence[s])
        if bias_tokens is not None:
            last = {int(v): float(b) for v, b in zip(bias_tokens[s], bias_values[s])}
            for v, b in last.items():
                if 0 <= v < V:
                    y[r, v] += b
        if allowed is not None:
            y[r, ~allowed[r]] = -np.inf
    return y


def commit(cache, block_tables, context_lens, query_start, path, path_lens, move) -> None:
    """Moves the accepted rows of one cache in place; ``move(cache, (block, place), (block,
    place))`` copies one token's row."""
    B = cache.shape[2] if cache.ndim == 4 else 16
    for s in range(len(context_lens)):
        base = int(context_lens[s]) - int(query_start[s + 1] - query_start[s])
        before = cache.copy()
        for j in range(int(path_lens[s])):
            a, b = base + int(path[s, j]), base + j
            move(before, cache, (int(block_tables[s, a // B]), a % B),
                 (int(block_tables[s, b // B]), b % B))
