"""The paged 4-bit KV cache (oracle): codec, page blocks, append, attention.

A head vector x of D float32 values is stored as D codes and two fp16 numbers,
every step a single rounding:

    d = fp16((max x - min x) * float32(1/15)),  z = fp16(min x + 8 d)
    code = clamp(round-half-even((x - z) / d) + 8, 0, 15), 8 where d = 0
    value = z + d (code - 8)

A vector with a NaN or an infinity is stored as d = 0, z = NaN.  Page blocks
as in ``pack_block``.  Positions, block tables and windows as in
``oracle.paged``; sequence s brings ``new[s]`` tokens of its ``lens[s]`` keys.
"""
from __future__ import annotations

import math

import numpy as np

from . import paged

PAGE = 128


def quantise(x):
    """``x[..., D]`` float32 -> codes uint8 ``[..., D]``, numbers fp16 ``[..., 2]``."""
    x = np.asarray(x, dtype=np.float32)
    lo, hi = x.min(-1, keepdims=True), x.max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        d16 = ((hi - lo) * np.float32(1 / 15)).astype(np.float16)
        d = d16.astype(np.float32)
        z16 = (lo + np.float32(8) * d).astype(np.float16)
        z = z16.astype(np.float32)
        q = np.rint((x - z) / d) + np.float32(8)
        q = np.where(d == 0, np.float32(8), np.clip(q, 0, 15))
    bad = ~np.isfinite(x).all(-1, keepdims=True)
    d16 = np.where(bad, np.float16(0), d16)
    z16 = np.where(bad, np.float16(np.nan), z16)
    q = np.where(bad, 8, q)
    return q.astype(np.uint8), np.concatenate([d16, z16], -1)


def values(codes, dz):
    """float64 values of codes and numbers."""
    dz = np.asarray(dz).astype(np.float64)
    return dz[..., 1:] + dz[..., :1] * (codes.astype(np.float64) - 8)


def block_bytes(d: int) -> int:
    return PAGE * (d + 8)


def pack_block(kc, kdz, vc, vdz):
    """One (page, head) block of 128 keys: codes ``[128, D]``, numbers ``[128, 2]``."""
    d = kc.shape[1]
    out = bytearray()
    for key in range(PAGE):
        for i in range(d // 2):
            out.append(int(kc[key, 2 * i]) | int(kc[key, 2 * i + 1]) << 4)
    out += np.asarray(kdz, dtype="<f2").tobytes()
    for pair in range(PAGE // 2):
        for w in range(d // 4):
            for key in (2 * pair, 2 * pair + 1):
                n = sum(int(vc[key, 4 * w + i]) << (4 * i) for i in range(4))
                out += bytes((n & 255, n >> 8))
    out += np.asarray(vdz, dtype="<f2").tobytes()
    return np.frombuffer(bytes(out), dtype=np.uint8).copy()


def unpack_block(b, d: int):
    """(kc, kdz, vc, vdz) of one block."""
    c = PAGE * d // 2
    kb = b[:c].reshape(PAGE, d // 2)
    kc = np.stack([kb & 15, kb >> 4], -1).reshape(PAGE, d)
    kdz = b[c:c + 4 * PAGE].copy().view("<f2").reshape(PAGE, 2)
    w = b[c + 4 * PAGE:2 * c + 4 * PAGE].copy().view("<u2").reshape(PAGE // 2, d // 4, 2)
    vc = np.stack([w >> (4 * i) & 15 for i in range(4)], -1)  # pair, word, key, nibble
    vc = vc.transpose(0, 2, 1, 3).reshape(PAGE, d).astype(np.uint8)
    vdz = b[2 * c + 4 * PAGE:].copy().view("<f2").reshape(PAGE, 2)
    return kc, kdz, vc, vdz


def positions(new, lens):
    """(sequence, position) of every token row."""
    return [(s, int(n) - int(m) + j) for s, (m, n) in enumerate(zip(new, lens)) for j in range(int(m))]


def append(pool, bt, n_blocks, window, new, lens, k, v):
    """Copy of ``pool[n_pages, Hkv, bytes]`` with the token rows' 4-bit rows;
    ``k, v`` float32 ``[n_tok, Hkv, D]`` as they are stored (rotated already)."""
    out, d = pool.copy(), k.shape[-1]
    for t, (s, p) in enumerate(positions(new, lens)):
        page, row = paged.locate(p, bt[s], int(n_blocks[s]), int(window[s]))
        for h in range(k.shape[1]):
            kc, kdz, vc, vdz = unpack_block(out[page, h], d)
            kc[row], kdz[row] = quantise(k[t, h])
            vc[row], vdz[row] = quantise(v[t, h])
            out[page, h] = pack_block(kc, kdz, vc, vdz)
    return out


def pool_values(pool, d: int):
    """float64 K and V ``[n_pages, Hkv, 128, D]`` of every page."""
    return _pool_map(pool, d, values)


def pool_sizes(pool, d: int):
    """|z| + d |code - 8| of every K and V value: the magnitudes of the two
    terms that make it, which a float32 evaluation rounds apart."""
    def size(codes, dz):
        dz = np.abs(np.asarray(dz).astype(np.float64))
        return dz[..., 1:] + dz[..., :1] * np.abs(codes.astype(np.float64) - 8)
    return _pool_map(pool, d, size)


def _pool_map(pool, d: int, fn):
    n, hkv = pool.shape[:2]
    k, v = np.empty((n, hkv, PAGE, d)), np.empty((n, hkv, PAGE, d))
    for i in range(n):
        for h in range(hkv):
            kc, kdz, vc, vdz = unpack_block(pool[i, h], d)
            k[i, h], v[i, h] = fn(kc, kdz), fn(vc, vdz)
    return k, v


def attention(q, kvals, vvals, bt, n_blocks, window, new, lens, sizes=None):
    """(out, bound) float64 ``[n_tok, Hq, D]`` of ``q[n_tok, Hq, D]``; bound is
    what a float32 evaluation may be off by, from the roundings it makes: each
    score by 2^-20 of the sum of its terms' magnitudes, each weight by that
    and 2^-20 more, the weighted sum by 2^-20 of its terms' magnitudes, and a
    weight times its scale by 2^-35 of the largest such product (a split into
    two fp16 of values whose largest is 2^10 or more), for each of the up to 8
    steps of its code.  ``sizes``: magnitudes of the terms of each value
    (``pool_sizes``)."""
    n_tok, hq, d = q.shape
    group = hq // kvals.shape[1]
    ksize, vsize = (np.abs(kvals), np.abs(vvals)) if sizes is None else sizes
    out, bound = np.empty((n_tok, hq, d)), np.empty((n_tok, hq, d))
    for t, (s, p) in enumerate(positions(new, lens)):
        w = int(window[s])
        lo = max(0, p - w + 1) if w else 0
        at = [paged.locate(i, bt[s], int(n_blocks[s]), w) for i in range(lo, p + 1)]
        pages, rows = np.array([a[0] for a in at]), np.array([a[1] for a in at])
        for h in range(hq):
            k, v = kvals[pages, h // group, rows], vvals[pages, h // group, rows]
            score = k @ q[t, h].astype(np.float64) / math.sqrt(d)
            size = (ksize[pages, h // group, rows] @ np.abs(q[t, h].astype(np.float64))).max() / math.sqrt(d)
            e = np.exp(score - score.max())
            e /= e.sum()
            out[t, h] = e @ v
            bound[t, h] = 2.0 ** -20 * (2 * (size + 1) * (e @ np.abs(v - out[t, h])) +
                                        e @ vsize[pages, h // group, rows])
            step = (v.max(-1) - v.min(-1)) / 8                     # above d
            bound[t, h] += 2.0 ** -35 * (e * step).max() * 8 * len(e)
    return out, bound
