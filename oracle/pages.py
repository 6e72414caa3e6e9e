"""Whole pages of a paged KV cache (oracle): copies, bounds, selection, attention
over all visible keys or over the selected pages, all from their definitions.

Test infrastructure: only the tests use this module; the library never does.
Pools are float64 values ``[n_pages, Hkv, 128, D]``; a batch is (block table,
block counts, windows, new tokens, lengths) as the library takes it.
"""
from __future__ import annotations

import math

import numpy as np

from . import kv_q4, paged

PAGE = paged.PAGE


def copy(pool, src, dst, keys):
    """``pool[n_pages, Hkv, 128, ...]`` after rows 0 .. keys[i] - 1 of every src have gone to dst."""
    out = pool.copy()
    for a, b, n in zip(src, dst, keys):
        out[b, :, :n] = pool[a, :, :n]
    return out


def copy_q4(pool, d, src, dst, keys):
    """The same of 4-bit blocks ``[n_pages, Hkv, bytes]``."""
    out = pool.copy()
    for a, b, n in zip(src, dst, keys):
        for h in range(pool.shape[1]):
            new, old = kv_q4.unpack_block(pool[a, h], d), kv_q4.unpack_block(out[b, h], d)
            for x, y in zip(old, new):
                x[:n] = y[:n]
            out[b, h] = kv_q4.pack_block(*old)
    return out


def bounds(k, bt, new, lens, before):
    """``before[n_pages, Hkv, 2, D]`` with the bounds of the pages that new tokens lie on."""
    out = before.copy()
    for s, (m, n) in enumerate(zip(new, lens)):
        for i in range((n - m) // PAGE, -(-n // PAGE)) if m else ():
            held = k[bt[s][i], :, :min(PAGE, n - i * PAGE)]
            out[bt[s][i]] = np.stack([held.min(1), held.max(1)], 1)     # NaN where one is
    return out


def _pairwise(terms):
    """float32 sum of a list of float32 arrays, neighbours first, zeros behind."""
    terms = list(terms)
    while len(terms) & (len(terms) - 1):
        terms.append(np.zeros_like(terms[0]))
    while len(terms) > 1:
        terms = [np.add(x, y, dtype=np.float32) for x, y in zip(terms[0::2], terms[1::2])]
    return terms[0]


def scores(q, lo, hi):
    """float32 score of each page: ``q[G, D]``, bounds ``lo, hi[pages, D]``."""
    q = q.astype(np.float32)
    a, b = _pairwise(np.maximum(q, 0)), _pairwise(np.minimum(q, 0))
    lo, hi = lo.astype(np.float32), hi.astype(np.float32)
    terms = np.multiply(a, hi, dtype=np.float32) + np.multiply(b, lo, dtype=np.float32)
    return _pairwise(list(terms.T))


def select(q, bnd, bt, new, lens, n_select, first, last):
    """int32 ``[n_tok, Hkv, n_select]``."""
    hkv = bnd.shape[1]
    group = q.shape[1] // hkv
    at = kv_q4.positions(new, lens)
    out = np.full((len(at), hkv, n_select), -1, np.int32)
    for t, (s, p) in enumerate(at):
        mine = p // PAGE
        pages = [bt[s][i] for i in range(mine + 1)]
        for h in range(hkv):
            sc = scores(q[t, h * group:(h + 1) * group], bnd[pages, h, 0], bnd[pages, h, 1])
            rank = {i: (0 if i < first or i > mine - last else 1 if np.isnan(sc[i]) else 2) for i in range(mine + 1)}
            order = sorted(range(mine + 1), key=lambda i: (rank[i], -float(sc[i]) if rank[i] == 2 else 0.0, i))
            got = sorted(order[:n_select])
            out[t, h, :len(got)] = got
    return out


def attention(q, k, v, bt, n_blocks, window, new, lens, selected=None, weight_step=2.0 ** -20):
    """(out, bound) float64 ``[n_tok, Hq, D]``.  bound is what a float32 evaluation
    may be off by: each score by 2^-20 of the sum of its terms' magnitudes, each
    weight by that and 2^-20 more, the weighted sum by ``weight_step`` of its terms'
    magnitudes (2^-20, or with weights as two bf16, within 2^-18, 2^-18 more), a
    weight by 2^-35 of the largest (two fp16 of values whose largest is 2^10 or
    more)."""
    n_tok, hq, d = q.shape
    group = hq // k.shape[1]
    out, bound = np.zeros((n_tok, hq, d)), np.zeros((n_tok, hq, d))
    for t, (s, p) in enumerate(kv_q4.positions(new, lens)):
        w = int(window[s])
        for h in range(hq):
            if selected is None:
                keys = np.arange(max(0, p - w + 1) if w else 0, p + 1)
            else:
                keys = np.array([i for b in selected[t, h // group] if 0 <= b <= p // PAGE
                                 for i in range(b * PAGE, min(p + 1, (b + 1) * PAGE))], int)
            if len(keys) == 0:
                continue
            block = keys // PAGE % int(n_blocks[s]) if w else keys // PAGE     # as paged.locate
            pages, rows = np.asarray(bt[s])[block], keys % PAGE
            kk, vv = k[pages, h // group, rows], v[pages, h // group, rows]
            x = q[t, h].astype(np.float64)
            score = kk @ x / math.sqrt(d)
            size = (np.abs(kk) @ np.abs(x)).max() / math.sqrt(d)
            e = np.exp(score - score.max())
            e /= e.sum()
            out[t, h] = e @ vv
            bound[t, h] = 2.0 ** -20 * 2 * (size + 1) * (e @ np.abs(vv - out[t, h])) + weight_step * (e @ np.abs(vv))
            bound[t, h] += 2.0 ** -35 * e.max() * np.abs(vv).sum(0)
    return out, bound
