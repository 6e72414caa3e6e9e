"""Pins of the page oracle: hand values, closed forms and agreement with the other
oracles where their domains meet."""
import numpy as np
import pytest

from oracle import kv_q4 as oq4
from oracle import paged as opg
from oracle import pages as op

P = 128


def _one(lens, new, rng, hkv=2, d=8, extra=1):
    blocks = [-(-n // P) for n in lens]
    total = sum(blocks) + extra
    order = rng.permutation(total)
    bt, at = np.zeros((len(lens), max(blocks)), int), 0
    for s, b in enumerate(blocks):
        bt[s, :b] = order[at:at + b]
        at += b
    k, v = rng.standard_normal((2, total, hkv, P, d))
    return bt, blocks, k, v


def test_copy_moves_rows_and_leaves_the_others():
    rng = np.random.default_rng(0)
    pool = rng.standard_normal((4, 2, P, 3))
    out = op.copy(pool, [0, 0], [2, 3], [5, 128])
    assert np.array_equal(out[:2], pool[:2]) and np.array_equal(out[3], pool[0])
    assert np.array_equal(out[2, :, :5], pool[0, :, :5]) and np.array_equal(out[2, :, 5:], pool[2, :, 5:])


def test_copy_q4_equals_a_copy_of_the_values():
    rng = np.random.default_rng(1)
    pool = rng.integers(0, 256, (3, 1, P * 72), dtype=np.uint8)
    pool.view("<u2")[:] &= 0xBFFF                            # numbers stay finite
    out = op.copy_q4(pool, 64, [1], [2], [77])
    for got, was in zip(oq4.pool_values(out, 64), oq4.pool_values(pool, 64)):
        assert np.array_equal(got, op.copy(was, [1], [2], [77]))


def test_pairwise_is_neighbours_first():
    big, one = np.float32(2 ** 24), np.float32(1)
    assert op._pairwise([big, one, one, one]) == 2 ** 24 + 2          # (2^24 + 1 -> 2^24) + 2
    assert op._pairwise([one, one, big]) == 2 ** 24 + 2
    assert op._pairwise([big, one, one]) == 2 ** 24                   # 2^24 + (1 + 0): a tie, to even


def test_score_bounds_every_key():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((5, 8)), rng.standard_normal((3, P, 8))
    s = op.scores(q, k.min(1), k.max(1))
    assert np.all(s >= (k @ q.sum(0)).max(1) - 1e-5)
    # a page of equal keys: the score is the sum of the products
    one = np.repeat(k[:1, :1], 1, 1)[:, 0]
    assert np.allclose(op.scores(q, one, one), one @ q.sum(0), atol=1e-5)


def test_select_ties_forced_pages_and_short_sequences():
    bnd = np.zeros((6, 1, 2, 4))
    bnd[3, 0, 1] = 1.0                                       # page 3: hi = 1
    q = np.ones((1, 1, 4))
    bt = np.arange(6)[None]
    got = op.select(q, bnd, bt, [1], [6 * P], 3, 0, 1)
    assert got.tolist() == [[[0, 3, 5]]]                     # its own, the largest, the tie's first
    assert op.select(q, bnd, bt, [1], [6 * P], 3, 1, 2).tolist() == [[[0, 4, 5]]]
    assert op.select(q, bnd, bt, [1], [2 * P], 3, 0, 1).tolist() == [[[0, 1, -1]]]
    bnd[1, 0, 0, 2] = np.nan
    assert op.select(-q, bnd, bt, [1], [6 * P], 2, 0, 1).tolist() == [[[1, 5]]]


def test_bounds_of_touched_pages_only():
    rng = np.random.default_rng(3)
    bt, blocks, k, _ = _one([300, 5], [3, 0], rng)
    before = np.full((k.shape[0], 2, 2, 8), 7.0)
    out = op.bounds(k, bt, [3, 0], [300, 5], before)
    page = bt[0, 2]
    assert np.array_equal(out[page, 1, 0], k[page, 1, :44].min(0))
    out[page] = 7.0
    assert np.array_equal(out, before)


@pytest.mark.parametrize("window", [0, 50])
def test_attention_equals_the_paged_oracle(window):
    rng = np.random.default_rng(4)
    lens, new = [200, 131], [2, 2]
    bt, blocks, k, v = _one(lens, new, rng)
    q = rng.standard_normal((4, 4, 8))
    w = [window, window]
    got, _ = op.attention(q, k, v, bt, blocks, w, new, lens)
    want = opg.attention_paged(q, k, v, bt, blocks, w, 2, lens)
    assert np.allclose(got, want, rtol=1e-12)


def test_attention_over_every_page_is_the_dense_one_and_an_empty_row_is_zero():
    rng = np.random.default_rng(5)
    bt, blocks, k, v = _one([300], [2], rng)
    q = rng.standard_normal((2, 2, 8))
    dense, _ = op.attention(q, k, v, bt, blocks, [0], [2], [300])
    sel = np.tile(np.array([0, 1, 2, -1]), (2, 2, 1))
    got, _ = op.attention(q, k, v, bt, blocks, [0], [2], [300], sel)
    assert np.allclose(got, dense, rtol=1e-12)
    sel[:] = -1
    assert not op.attention(q, k, v, bt, blocks, [0], [2], [300], sel)[0].any()
