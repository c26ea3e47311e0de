"""Beam search's selection in fp64 — the oracle.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``): never imported by the library.

Candidate (b, v) of a request scores ``beam_scores[b] + logits[b, v] - lse[b]``; the best
``n`` come out by score, equal scores by beam, within a beam by logit and then by token.
A NaN logit counts as -infinity.  A beam whose score or largest logit is not finite has
candidates of score -infinity only, in token order.
"""
from __future__ import annotations

import numpy as np


def candidate_scores(logits, beam_scores) -> np.ndarray:
    """``[K, V]`` scores of one request."""
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x)] = -np.inf
    out = np.full(x.shape, -np.inf)
    for b in range(x.shape[0]):
        top = x[b].max()
        if np.isfinite(top) and np.isfinite(beam_scores[b]):
            # not x - (top + log sum): a large top would swallow the log
            out[b] = float(beam_scores[b]) + ((x[b] - top) - np.log(np.exp(x[b] - top).sum()))
    return out


def select(logits, beam_scores, n):
    """(scores [n], beams [n], tokens [n]) of one request's best candidates."""
    s = candidate_scores(logits, beam_scores)
    x = np.array(logits, dtype=np.float64)
    x[np.isnan(x) | ~np.isfinite(s)] = -np.inf
    K, V = s.shape
    beam, tok = np.divmod(np.arange(K * V), V)
    order = np.lexsort((tok, -x.ravel(), beam, -s.ravel()))[:n]
    return s.ravel()[order], beam[order], tok[order]
