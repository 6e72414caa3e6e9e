"""Rotary positions in both pair layouts, over part of a head, scaled (oracle).

Pair i of the first r dimensions of a head turns by ``pos * f_i``; the pair is
(i, i + r/2) ("half") or (2i, 2i + 1) ("interleaved").  Frequencies
``f_i = theta^(-2i/r)``, or with s the scale factor:

    linear   f_i / s
    ntk      theta s^(r/(r-2)) in place of theta: the slowest pair, i = r/2 - 1,
             ends at f / s and the fastest, i = 0, at f
    bands    f_i where a pair turns more than ``high`` times over the original
             context, f_i / s where it turns less than ``low`` times, blended
             linearly in the number of turns between
    yarn     ``oracle.rope.frequencies``

All float64.
"""
from __future__ import annotations

import math

import numpy as np

from . import rope


def frequencies(rd: int, theta: float, scaling=None, factor=1.0, orig_ctx=0, low=0.0, high=0.0, yarn=None):
    if yarn is not None:
        return rope.frequencies(rd, theta, yarn)
    if scaling == "ntk":
        theta = theta * factor ** (rd / (rd - 2))
    f = np.array([float(theta) ** (-2.0 * i / rd) for i in range(rd // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        out = []
        for x in f:
            turns = orig_ctx * x / (2 * math.pi)
            keep = 1.0 if turns >= high else 0.0 if turns <= low else (turns - low) / (high - low)
            out.append(keep * x + (1 - keep) * x / factor)
        return np.array(out)
    return f


def rotate(x, pos, f, interleaved: bool, gain: float = 1.0):
    """``x[n_tok, H, D]`` with the first ``2 len(f)`` dimensions rotated."""
    y = np.array(x, dtype=np.float64)
    rd = 2 * len(f)
    for t, p in enumerate(np.asarray(pos, dtype=np.float64)):
        for i in range(rd // 2):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rd // 2)
            c, s = math.cos(p * f[i]) * gain, math.sin(p * f[i]) * gain
            u, v = y[t, :, a].copy(), y[t, :, b].copy()
            y[t, :, a] = u * c - v * s
            y[t, :, b] = u * s + v * c
    return y
