"""Pins of the 4-bit KV and rotary oracles (no GPU)."""
import math

import numpy as np
import pytest

from oracle import attention as oatt
from oracle import kv_q4 as oq4
from oracle import rope as orope
from oracle import rotary as orot


def test_codec_on_hand_values():
    x = np.arange(16, dtype=np.float32) - 4          # -4 .. 11: d = 1, z = 4, codes 0..15
    q, dz = oq4.quantise(x)
    assert dz.tolist() == [1.0, 4.0] and q.tolist() == list(range(16))
    assert np.array_equal(oq4.values(q, dz), x)
    q, dz = oq4.quantise(np.full(64, 2.5, np.float32))   # no spread: d = 0, the value is z
    assert dz.tolist() == [0.0, 2.5] and set(q.tolist()) == {8}
    # halves go to the even code: -0.5 and 0.5 below and above z = 8 both give code 8
    x = np.array([0, 15, 7.5, 8.5, 6.5, 9.5], np.float32)
    q, dz = oq4.quantise(x)
    assert dz.tolist() == [1.0, 8.0] and q.tolist() == [0, 15, 8, 8, 6, 10]
    for bad in (np.nan, np.inf, -np.inf):
        x = np.zeros(64, np.float32)
        x[3] = bad
        assert np.isnan(oq4.values(*oq4.quantise(x))).all()


def test_codec_error_is_half_a_step():
    rng = np.random.default_rng(0)
    for scale, shift in ((1.0, 0.0), (1e-3, 0.0), (5.0, 40.0), (100.0, -3.0)):
        x = (rng.standard_normal((200, 128)) * scale + shift).astype(np.float32)
        q, dz = oq4.quantise(x)
        d, z = dz[:, :1].astype(np.float64), dz[:, 1:].astype(np.float64)
        # d and z are rounded to fp16: the ends may fall outside the codes by what that
        # moves them, 8 d 2^-11 and |z| 2^-11 (z is a half step of fp16 away at most)
        slack = 8 * d * 2.0 ** -10 + np.abs(z) * 2.0 ** -11 + 1e-7
        assert (np.abs(oq4.values(q, dz) - x) <= d / 2 + slack).all()


@pytest.mark.parametrize("d", [64, 128])
def test_block_layout(d):
    rng = np.random.default_rng(d)
    kc, vc = rng.integers(0, 16, (2, 128, d)).astype(np.uint8)
    kdz, vdz = rng.standard_normal((2, 128, 2)).astype(np.float16)
    b = oq4.pack_block(kc, kdz, vc, vdz)
    assert b.nbytes == oq4.block_bytes(d)
    for got, want in zip(oq4.unpack_block(b, d), (kc, kdz, vc, vdz)):
        assert np.array_equal(got, want)
    # single places, from the description
    assert b[5 * d // 2 + 3] == kc[5, 6] | kc[5, 7] << 4
    v0 = 64 * d + 512
    assert b[v0 + 3 * d + 4 * 2 + 2] == vc[7, 8] | vc[7, 9] << 4      # pair 3, word 2, its odd key
    assert b[v0 - 512 + 4 * 9:v0 - 512 + 4 * 9 + 4].view("<f2").tolist() == kdz[9].tolist()


def test_append_touches_its_rows_only():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (4, 2, oq4.block_bytes(64))).astype(np.uint8)
    bt = np.array([[2, 0], [3, 1]])
    k, v = rng.standard_normal((2, 3, 2, 64)).astype(np.float32)
    got = oq4.append(pool, bt, [2, 2], [0, 100], [2, 1], [130, 260], k, v)   # keys 128, 129 and key 259 (ring)
    kc, kdz, vc, vdz = oq4.unpack_block(got[0, 1], 64)
    q, dz = oq4.quantise(k[1, 1])
    assert np.array_equal(kc[1], q) and np.array_equal(kdz[1], dz)
    assert np.array_equal(oq4.values(*oq4.quantise(v[2, 0])), oq4.pool_values(got, 64)[1][3, 0, 259 % 128])
    changed = {(p, h) for p in range(4) for h in range(2) if not np.array_equal(got[p, h], pool[p, h])}
    assert changed == {(0, 0), (0, 1), (3, 0), (3, 1)}
    old = oq4.unpack_block(pool[0, 0], 64)
    for a, b in zip(oq4.unpack_block(got[0, 0], 64), old):
        assert np.array_equal(a[2:].view(np.uint8), b[2:].view(np.uint8))


def test_attention_matches_the_plain_oracle():
    rng = np.random.default_rng(2)
    kv = rng.standard_normal((2, 1, 2, 128, 64))
    q = rng.standard_normal((1, 4, 64)).astype(np.float32)
    out, bound = oq4.attention(q, kv[0], kv[1], [[0]], [1], [0], [1], [37])
    for h in range(4):
        w = oatt.weights(q[0, h], kv[0][0, h // 2, :37])
        assert np.allclose(out[0, h], w @ kv[1][0, h // 2, :37], rtol=1e-13)
    assert (bound > 0).all() and bound.max() < 1e-3
    one, _ = oq4.attention(q, kv[0], kv[1], [[0]], [1], [1], [1], [37])      # a window of one key returns V
    assert np.array_equal(one[0, 3], kv[1][0, 1, 36])


def test_rotary_layouts():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((3, 2, 16))
    pos = [0, 5, 12345]
    f = orot.frequencies(16, 10000.0)
    assert np.allclose(orot.rotate(x, pos, f, False), orope.rope_posvec(x, pos, 10000.0), atol=1e-12)
    # the two layouts are the same rotation of permuted dimensions
    perm = np.array([i // 2 + 8 * (i % 2) for i in range(16)])
    assert np.allclose(orot.rotate(x[..., perm], pos, f, True), orot.rotate(x, pos, f, False)[..., perm], atol=1e-12)
    # part of the head: the rest passes, the rotated part is a head of its own
    f6 = orot.frequencies(6, 100.0)
    y = orot.rotate(x, pos, f6, False)
    assert np.array_equal(y[..., 6:], x[..., 6:])
    assert np.allclose(y[..., :6], orope.rope_posvec(x[..., :6], pos, 100.0), atol=1e-12)
    assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))


def test_scalings():
    f = orot.frequencies(64, 10000.0)
    assert np.allclose(orot.frequencies(64, 10000.0, "linear", 8.0) * 8, f)
    ntk = orot.frequencies(64, 10000.0, "ntk", 8.0)
    assert math.isclose(ntk[0], f[0]) and math.isclose(ntk[-1], f[-1] / 8, rel_tol=1e-12)
    b = orot.frequencies(64, 10000.0, "bands", 8.0, 8192, 1.0, 4.0)
    turns = 8192 * f / (2 * math.pi)
    assert np.array_equal(b[turns >= 4], f[turns >= 4]) and np.allclose(b[turns <= 1], f[turns <= 1] / 8, rtol=1e-15)
    mid = (turns > 1) & (turns < 4)
    assert mid.any() and (b[mid] < f[mid]).all() and (b[mid] > f[mid] / 8).all()
