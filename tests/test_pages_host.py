"""Refusals of the calls on whole pages (no GPU): every bad argument is named before
any device work, and the binding checks buffers before a pointer reaches the
library."""
import ctypes
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")

FAKE = ctypes.c_void_p(1 << 20)          # never dereferenced: validation fails first
FAR = ctypes.c_void_p(1 << 30)
ODD = ctypes.c_void_p((1 << 20) + 4)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def d():
    from session_decode_step_dsb_gb300 import build, dsb
    if not os.path.exists(dsb.LIB_PATH):
        build.build()
    dsb.lib()
    return dsb


def _kv(d, k=FAKE, v=FAR, dtype=0, n_pages=8, heads=2, dim=64):
    return d.KVPages(k, v, dtype, n_pages, heads, dim)


def _batch(d, **kw):
    a = dict(block_table=[[0, 1], [2, 3]], n_blocks=[2, 2], window=[0, 0], new_tokens=[1, 2], seq_lens=[130, 2])
    a.update(kw)
    return d.PagedBatch(**a)


def _refused(d, status, want, word):
    assert status == want, (status, d.lib().dsb_last_error())
    assert word in d.lib().dsb_last_error().decode(), d.lib().dsb_last_error()


def _i32(*x):
    a = np.array(x, np.int32)
    return a, a.ctypes.data


# --------------------------------------------------------------------- copies
def _copy(d, src, dst, keys, pools=None, n=None, q4=False):
    lib = d.lib()
    pools = [_kv(d)] if pools is None else pools
    arr = (type(pools[0]) * len(pools))(*pools)
    (s, ps), (t, pt), (k, pk) = _i32(*src), _i32(*dst), _i32(*keys)
    fn = lib.dsb_kv_copy_pages_q4 if q4 else lib.dsb_kv_copy_pages
    return fn(arr, len(pools) if n is None else n, ps, pt, pk, len(src), None)


@pytest.mark.parametrize("src,dst,keys,word", [
    ([0], [8], [1], "out of [0, 8)"), ([-1], [1], [1], "out of [0, 8)"), ([0], [1], [129], "keys[0]"),
    ([0], [1], [-1], "keys[0]"), ([0, 1], [2, 2], [1, 1], "another one"), ([0, 2], [2, 3], [1, 1], "read by the same"),
    ([4], [4], [128], "read by the same"), ([0, 1], [1, 0], [5, 5], "read by the same")])
@pytest.mark.parametrize("q4", [False, True])
def test_copies_that_race_or_leave_the_pool(d, src, dst, keys, word, q4):
    pools = [d.KVQ4Pages(FAKE, 8, 2, 64)] if q4 else None
    _refused(d, _copy(d, src, dst, keys, pools, q4=q4), INVALID, word)


def test_copies_of_nothing_are_no_work(d):
    assert _copy(d, [], [], []) == 0
    assert _copy(d, [0, 1], [1, 1], [0, 0]) == 0             # no row: no conflict, no launch


@pytest.mark.parametrize("pools,status,word", [
    (lambda d: [_kv(d), _kv(d, k=ctypes.c_void_p((1 << 20) + 4096))], INVALID, "overlap"),
    (lambda d: [_kv(d, v=FAKE)], INVALID, "overlap"),
    (lambda d: [_kv(d), _kv(d, k=ctypes.c_void_p(1 << 31), v=ctypes.c_void_p(1 << 32), n_pages=9)], INVALID, "differs"),
    (lambda d: [_kv(d, k=ODD)], INVALID, "aligned"), (lambda d: [_kv(d, k=None)], INVALID, "NULL"),
    (lambda d: [_kv(d, dtype=2)], INVALID, "dtype"), (lambda d: [_kv(d, dim=96)], UNSUPPORTED, "head_dim"),
    (lambda d: [_kv(d, n_pages=0)], INVALID, "n_pages"), (lambda d: [_kv(d, n_pages=1 << 23, heads=2)], UNSUPPORTED, "pool")])
def test_pools_that_copies_refuse(d, pools, status, word):
    _refused(d, _copy(d, [0], [1], [5], pools(d)), status, word)


def test_the_number_of_pools(d):
    _refused(d, _copy(d, [0], [1], [5], n=0), INVALID, "n_pools")
    _refused(d, _copy(d, [0], [1], [5], n=513), INVALID, "n_pools")
    _refused(d, d.lib().dsb_kv_copy_pages(None, 1, None, None, None, 0, None), INVALID, "pools is NULL")
    arr = (d.KVPages * 1)(_kv(d))
    _refused(d, d.lib().dsb_kv_copy_pages(arr, 1, None, None, None, 1, None), INVALID, "src / dst / keys")
    _refused(d, d.lib().dsb_kv_copy_pages(arr, 1, None, None, None, -1, None), INVALID, "n_copies")


# ------------------------------------------------------------------ attention
def _shared(d, kv=None, b=None, q=ctypes.c_void_p(1 << 33), stride=256, hq=4, out=ctypes.c_void_p(1 << 34), ws=FAKE):
    kv, b = kv or _kv(d), b or _batch(d)
    return d.lib().dsb_attention_decode_shared(q, stride, hq, ctypes.byref(kv), b.ref, out, ws, None)


def _selected(d, kv=None, b=None, q=ctypes.c_void_p(1 << 33), stride=256, hq=4, sel=ctypes.c_void_p(1 << 35), n=2,
              out=ctypes.c_void_p(1 << 34), ws=FAKE):
    kv, b = kv or _kv(d), b or _batch(d)
    return d.lib().dsb_attention_decode_selected(q, stride, hq, ctypes.byref(kv), b.ref, sel, n, out, ws, None)


def _select(d, kv=None, b=None, q=ctypes.c_void_p(1 << 33), stride=256, hq=4, bounds=ctypes.c_void_p(1 << 34), n=3,
            first=1, last=1, sel=ctypes.c_void_p(1 << 35), ws=FAKE):
    kv, b = kv or _kv(d), b or _batch(d)
    return d.lib().dsb_kv_select_pages(q, stride, hq, ctypes.byref(kv), bounds, b.ref, n, first, last, sel, ws, None)


def _bounds(d, kv=None, b=None, bounds=ctypes.c_void_p(1 << 34)):
    kv, b = kv or _kv(d), b or _batch(d)
    return d.lib().dsb_kv_page_bounds(ctypes.byref(kv), b.ref, bounds, None)


@pytest.mark.parametrize("call", [_shared, _selected, _select])
@pytest.mark.parametrize("change,status,word", [
    (dict(hq=0), INVALID, "n_q_heads"), (dict(hq=3), INVALID, "n_q_heads"), (dict(stride=252), INVALID, "q_stride"),
    (dict(stride=258), INVALID, "q_stride"), (dict(q=None), INVALID, "NULL"), (dict(q=ODD), INVALID, "aligned"),
    (dict(ws=None), WORKSPACE, "workspace")])
def test_bad_rows_are_named(d, call, change, status, word):
    _refused(d, call(d, **change), status, word)


@pytest.mark.parametrize("call", [_shared, _selected, _select, _bounds])
@pytest.mark.parametrize("change,word", [
    (dict(seq_lens=[257, 2]), "do not cover"), (dict(seq_lens=[130, 1]), "new_tokens"), (dict(seq_lens=[-1, 2]), "seq_lens"),
    (dict(new_tokens=[-1, 2]), "new_tokens"), (dict(block_table=[[0, 8], [2, 3]]), "block_table"),
    (dict(block_table=[[0, 1], [-1, 3]]), "block_table"), (dict(n_blocks=[3, 2]), "n_blocks"),
    (dict(window=[-1, 0]), "window"),
    (dict(new_tokens=[8000, 8000], seq_lens=[8000, 8000], n_blocks=[63, 63], block_table=[[0] * 63] * 2), "exceed")])
def test_bad_batches_are_named(d, call, change, word):
    _refused(d, call(d, b=_batch(d, **change)), INVALID, word)


@pytest.mark.parametrize("call", [_selected, _select, _bounds])
def test_rings_have_no_selection(d, call):
    _refused(d, call(d, b=_batch(d, window=[0, 100])), UNSUPPORTED, "rings")


@pytest.mark.parametrize("call", [_shared, _selected, _select, _bounds])
@pytest.mark.parametrize("kv,status,word", [
    (dict(k=None), INVALID, "NULL"), (dict(v=ODD), INVALID, "aligned"), (dict(dtype=5), INVALID, "dtype"),
    (dict(dim=80), UNSUPPORTED, "head_dim"), (dict(n_pages=1 << 23), UNSUPPORTED, "pool")])
def test_bad_pools_are_named(d, call, kv, status, word):
    _refused(d, call(d, kv=_kv(d, **kv)), status, word)


def test_outputs_apart_from_inputs(d):
    _refused(d, _shared(d, out=ctypes.c_void_p((1 << 33) + 64)), INVALID, "rows of q")
    _refused(d, _shared(d, out=FAKE), INVALID, "page pools")
    _refused(d, _selected(d, out=ctypes.c_void_p((1 << 30) + 64)), INVALID, "page pools")
    _refused(d, _selected(d, sel=ctypes.c_void_p(1 << 34)), INVALID, "selected")
    _refused(d, _select(d, sel=ctypes.c_void_p(1 << 33)), INVALID, "selected")
    _refused(d, _select(d, sel=ctypes.c_void_p((1 << 34) + 16)), INVALID, "selected")
    _refused(d, _bounds(d, bounds=FAKE), INVALID, "bounds")
    _refused(d, _shared(d, out=ODD), INVALID, "aligned")
    _refused(d, _select(d, bounds=ODD), INVALID, "aligned")
    _refused(d, _selected(d, sel=None), INVALID, "NULL")
    _refused(d, _bounds(d, bounds=None), INVALID, "bounds")


@pytest.mark.parametrize("n,first,last", [(0, 0, 1), (2, 1, 2), (3, -1, 1), (3, 1, 0), (1, 1, 1), (-5, 0, 1)])
def test_selections_that_do_not_fit(d, n, first, last):
    _refused(d, _select(d, n=n, first=first, last=last), INVALID, "keep_")


def test_lists_without_entries(d):
    _refused(d, _selected(d, n=0), INVALID, "n_select")
    _refused(d, _selected(d, n=1 << 30), INVALID, "n_select")


def test_two_sequences_on_one_page_have_no_bounds(d):
    _refused(d, _bounds(d, b=_batch(d, block_table=[[0, 1], [1, 3]])), INVALID, "twice on page 1")


def test_calls_without_new_tokens_do_nothing(d):
    b = _batch(d, new_tokens=[0, 0])
    assert _shared(d, b=b) == 0 and _selected(d, b=b) == 0 and _select(d, b=b) == 0 and _bounds(d, b=b) == 0


# -------------------------------------------------------------------- binding
def test_the_binding_checks_shapes_and_types(d):
    z = torch.zeros
    kv, b = _kv(d), _batch(d)
    kv._tensors, kv._device = (z(1), z(1)), 0
    with pytest.raises(ValueError, match="head_dim"):
        d.attention_decode_shared(z(3, 4, 32), kv, b, None)
    with pytest.raises(ValueError, match="3 rows"):
        d.attention_decode_shared(z(2, 4, 64), kv, b, None)
    with pytest.raises(ValueError, match="float32"):
        d.attention_decode_shared(z(3, 4, 64).half(), kv, b, None)
    with pytest.raises(ValueError, match="CUDA device"):
        d.attention_decode_shared(z(3, 4, 64), kv, b, None)
    with pytest.raises(ValueError, match="sequence of KVPages"):
        d.kv_copy_pages([], [0], [1], [1])
    with pytest.raises(ValueError, match="sequence of KVPages"):
        d.kv_copy_pages([d.KVQ4Pages(FAKE, 8, 2, 64)], [0], [1], [1])
    with pytest.raises(ValueError, match="dst has 2 entries"):
        d.kv_copy_pages([kv], [0], [1, 2], [1])
    with pytest.raises(ValueError, match="int32 can hold"):
        d.kv_copy_pages([kv], [0.5], [1], [1])
    with pytest.raises(ValueError, match="CUDA device"):
        d.kv_page_bounds(kv, b, z(8, 2, 2, 64))
