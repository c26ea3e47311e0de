"""Rotary positions in fp64 — the oracle.

TEST INFRASTRUCTURE (see ``oracle/__init__.py``): never imported by the library.

The first ``rotary_dim`` elements of a head form pairs; pair ``i`` of a token at
position ``p`` is the complex number ``x1 + i x2`` turned by ``p * f_i``:
``y1 = x1 cos - x2 sin``, ``y2 = x2 cos + x1 sin``.  Half layout: pair ``i`` is
elements ``i`` and ``i + rotary_dim / 2``; interleaved: elements ``2i`` and
``2i + 1``.  The rest of the head passes through.

Frequencies: ``f_i = base ** (-2 i / rotary_dim)``, for longer contexts divided by a
factor ("linear"), taken with ``base * factor ** (rotary_dim / (rotary_dim - 2))``
("ntk", which divides the last pair's frequency by the factor and keeps the first's),
or scaled by the pair's turns within the original length ("bands").
"""
from __future__ import annotations

import math

import numpy as np


def frequencies(rotary_dim, base=10000.0, scaling="none", factor=1.0, original_length=0,
                low_turns=1.0, high_turns=4.0) -> np.ndarray:
    out = []
    for i in range(rotary_dim // 2):
        b = base
        if scaling == "ntk" and rotary_dim > 2:
            b = base * factor ** (rotary_dim / (rotary_dim - 2))
        f = b ** (-2.0 * i / rotary_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original_length * f / (2 * math.pi)
            if turns <= low_turns:
                f /= factor
            elif turns < high_turns:
                t = (turns - low_turns) / (high_turns - low_turns)
                f = f * ((1 - t) / factor + t)
        out.append(f)
    return np.array(out)


def rotate(x, positions, inv_freq, interleaved=False, magnitude=1.0) -> np.ndarray:
    """``x [T, H, D]`` turned to ``positions [T]``, fp64."""
    y = np.array(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    half = len(f)
    z = np.exp(1j * np.asarray(positions, dtype=np.float64)[:, None] * f) * magnitude
    one, two = ((slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved
                else (slice(0, half), slice(half, 2 * half)))
    w = (y[..., one] + 1j * y[..., two]) * z[:, None, :]
    y[..., one], y[..., two] = w.real, w.imag
    return y
