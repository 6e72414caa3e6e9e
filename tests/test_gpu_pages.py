"""GPU parity of the calls on whole pages -- copies, bounds, selection, attention over
shared and over selected pages -- against the float64 oracle, through the C ABI.

Copies, bounds and selections are exact.  The attention's bound is the oracle's: every
rounding of a float32 evaluation, and for bf16 caches 2^-18 more of the weighted
values' magnitudes, which leaves room for weights of two bf16 (each rounding 2^-9 of
what is left; the kernels take three)."""
import numpy as np
import pytest

from oracle import pages as op
from tests.gpu_util import to_dev, to_host

pytestmark = pytest.mark.gpu

P = 128


def _dsb():
    from session_decode_step_dsb_gb300 import dsb
    return dsb


def _torch():
    import torch
    return torch


def _type(kind):
    d, t = _dsb(), _torch()
    return (d.DSB_F16, t.float16) if kind == "f16" else (d.DSB_BF16, t.bfloat16)


def _pools(rng, n_pages, hkv, D, kind, scale=1.0):
    """Device K and V pools and their float64 values."""
    t = _torch()
    dev = [t.from_numpy(rng.standard_normal((n_pages, hkv, P, D)) * scale).to(_type(kind)[1]).cuda() for _ in "kv"]
    return dev, [x.double().cpu().numpy() for x in dev]


def _tree(rng, groups, per, common, branch, tails, spare=2):
    """Block table of groups * per sequences over a shuffled pool, its block counts, lengths, page count."""
    lens = [(common + branch) * P + int(n) for n in tails]
    blocks = [max(1, -(-n // P)) for n in lens]
    own = [b - common - branch for b in blocks]
    total = common + groups * branch + sum(own) + spare
    order = rng.permutation(total)
    table, at = np.zeros((len(lens), max(blocks)), np.int32), common + groups * branch
    for s, b in enumerate(blocks):
        g = s // per
        table[s, :b] = np.concatenate([order[:common], order[common + g * branch:common + (g + 1) * branch],
                                       order[at:at + own[s]]])
        at += own[s]
    return table, blocks, lens, total


def _attend(q, dev, kind, table, blocks, window, new, lens, **kw):
    d = _dsb()
    kv = d.kv_pages(dev[0], dev[1], _type(kind)[0])
    batch = d.PagedBatch(table, blocks, window, new, lens)
    ws = d.Workspace(max(batch.n_tok, 1), q.shape[1], q.shape[2], max(lens))
    if "selected" in kw:
        return d.attention_decode_selected(q, kv, batch, kw["selected"], ws)
    return d.attention_decode_shared(q, kv, batch, ws)


def _check(got, want, bound, what=""):
    got = to_host(got).astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: not finite"
    bad = np.abs(got - want) > bound
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} outside the bound, worst "
                           f"{(np.abs(got - want) / np.maximum(bound, 1e-300)).max():.2f} times it at "
                           f"{np.unravel_index((np.abs(got - want) / np.maximum(bound, 1e-300)).argmax(), bad.shape)}")


def _step(kind):
    return 2.0 ** -20 + (2.0 ** -18 if kind == "bf16" else 0)


# --------------------------------------------------------------------- copies
@pytest.mark.parametrize("kind,D,hkv,layers,keys", [
    ("f16", 64, 1, 1, [1]), ("bf16", 128, 3, 3, [128, 77, 0, 1]), ("f16", 128, 8, 2, [128] * 5),
    ("q4", 64, 1, 1, [1]), ("q4", 64, 3, 2, [128, 127, 2, 3, 0]), ("q4", 128, 2, 3, [1, 5, 64, 126, 128, 33]),
    ("q4", 128, 8, 40, [4, 7]), ("bf16", 64, 2, 512, [9])])
def test_copies_move_the_keys_and_nothing_else(kind, D, hkv, layers, keys):
    d, t, rng = _dsb(), _torch(), np.random.default_rng(len(keys) * D + layers)
    n = 2 * len(keys) + 1
    order = rng.permutation(n)
    src, dst = order[:len(keys)].copy(), order[len(keys):2 * len(keys)]
    if len(keys) > 1:
        src[1] = src[0]
    if kind == "q4":
        host = rng.integers(0, 256, (layers, n, hkv, P * (D + 8)), dtype=np.uint8)
        dev = to_dev(host)
        d.kv_copy_pages_q4([d.kv_q4_pages(p, D) for p in dev], src, dst, keys)
        want = np.stack([op.copy_q4(p, D, src, dst, keys) for p in host]) if layers < 9 else None
        if want is None:                                     # the first and the last layer
            want = host.copy()
            for i in (0, layers - 1):
                want[i] = op.copy_q4(host[i], D, src, dst, keys)
                assert np.array_equal(to_host(dev[i]), want[i])
            return
    else:
        host = rng.integers(0, 1 << 16, (layers, 2, n, hkv, P, D), dtype=np.uint16)
        dev = to_dev(host.view(np.int16))
        d.kv_copy_pages([d.kv_pages(p[0], p[1], _type(kind)[0]) for p in dev], src, dst, keys)
        want = np.stack([[op.copy(x, src, dst, keys) for x in p] for p in host]).view(np.int16)
    assert np.array_equal(to_host(dev), want)


def test_more_copies_than_a_launch_holds():
    d, rng = _dsb(), np.random.default_rng(3)
    n = 1500
    host = rng.integers(0, 1 << 16, (2, 2 * n, 1, P, 64), dtype=np.uint16)
    dev = to_dev(host.view(np.int16))
    order, keys = rng.permutation(2 * n), rng.integers(0, 4, n)
    d.kv_copy_pages([d.kv_pages(dev[0], dev[1], d.DSB_F16)], order[:n], order[n:], keys)
    want = np.stack([op.copy(x, order[:n], order[n:], keys) for x in host]).view(np.int16)
    assert np.array_equal(to_host(dev), want)


# ------------------------------------------------------ attention, shared pages
SHARED = [
    # kind, hq, hkv, D, groups, per, common, branch, tails, new
    ("f16", 1, 1, 64, 1, 1, 0, 0, [1], [1]),
    ("bf16", 2, 1, 128, 1, 1, 0, 0, [128], [1]),
    ("f16", 12, 12, 64, 1, 4, 2, 0, [20, 200, 1, 129], [1, 1, 1, 1]),
    ("bf16", 10, 2, 128, 1, 5, 3, 0, [1, 130, 300, 7, 128], [1, 1, 1, 1, 1]),
    ("f16", 10, 2, 128, 2, 3, 1, 2, [50, 3, 140, 1, 1, 260], [3, 0, 2, 1, 1, 4]),
    ("bf16", 8, 1, 64, 3, 2, 0, 2, [5, 6, 7, 8, 9, 300], [5, 6, 1, 2, 0, 40]),
    ("f16", 3, 3, 128, 1, 9, 5, 0, [11] * 9, [1] * 9),
    ("bf16", 16, 2, 128, 1, 2, 0, 0, [700, 650], [1, 2]),
    ("f16", 40, 8, 128, 1, 3, 2, 0, [100, 90, 80], [1, 1, 1]),
    ("f16", 5, 1, 64, 1, 1, 9, 0, [77], [77]),
    ("bf16", 5, 1, 128, 1, 1, 0, 0, [300], [300]),
    ("f16", 64, 1, 128, 1, 2, 3, 0, [3, 2], [1, 1]),
    ("bf16", 4, 2, 64, 1, 40, 2, 0, list(range(1, 41)), [1] * 40),
    ("f16", 2, 2, 128, 1, 3, 30, 0, [64, 1, 2], [1, 1, 1]),
]


@pytest.mark.parametrize("kind,hq,hkv,D,groups,per,common,branch,tails,new", SHARED)
def test_shared_attention_matches_the_oracle(kind, hq, hkv, D, groups, per, common, branch, tails, new):
    rng = np.random.default_rng(sum(tails) + hq + D)
    table, blocks, lens, total = _tree(rng, groups, per, common, branch, tails)
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32) * 2
    window = [0] * len(lens)
    got = _attend(to_dev(q), dev, kind, table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step(kind))
    _check(got, want, bound)


def test_windows_beside_shared_pages():
    rng = np.random.default_rng(11)
    table, blocks, lens, total = _tree(rng, 1, 5, 3, 0, [40, 300, 90, 200, 10])
    window, new = [0, 130, 0, 1, 500], [2, 3, 1, 2, 1]
    # rings: as many pages as the window needs
    for s in (1, 3, 4):
        blocks[s] = (window[s] + new[s] - 2) // P + 2
    table = np.pad(table, ((0, 0), (0, 3)))
    extra = total + 30
    for s in (1, 3, 4):
        table[s, :blocks[s]] = np.arange(total + 6 * (s - 1), total + 6 * (s - 1) + blocks[s])
    dev, (k, v) = _pools(rng, extra, 2, 64, "f16")
    q = rng.standard_normal((sum(new), 6, 64)).astype(np.float32)
    got = _attend(to_dev(q), dev, "f16", table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens)
    _check(got, want, bound)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("new", [[1, 1, 1], [4, 3, 5], [70, 2, 30]])
def test_what_is_hidden_reaches_no_row(kind, new):
    t, rng = _torch(), np.random.default_rng(5)
    table, blocks, lens, total = _tree(rng, 1, 3, 2, 0, [100, 200, 33])
    dev, (k, v) = _pools(rng, total, 2, 64, kind)
    q = rng.standard_normal((sum(new), 4, 64)).astype(np.float32)
    window = [0, 0, 0]
    clean = to_host(_attend(to_dev(q), dev, kind, table, blocks, window, new, lens))
    # rows behind the last keys and pages of nobody hold anything
    used = set()
    for s, n in enumerate(lens):
        for p in range(n):
            used.add((int(table[s, p // P]), p % P))
    mask = np.array([[(p, r) not in used for r in range(P)] for p in range(total)])
    for x in dev:
        x[t.from_numpy(mask).cuda()[:, None].expand(-1, 2, -1)] = float("nan")
    got = to_host(_attend(to_dev(q), dev, kind, table, blocks, window, new, lens))
    assert np.array_equal(got, clean)
    # a draft's key and value seen by the later drafts only
    last, page, row = lens[0] - 1, int(table[0, (lens[0] - 1) // P]), (lens[0] - 1) % P
    dev[0][page, :, row] = float("nan")
    dev[1][page, :, row] = float("inf")
    got = to_host(_attend(to_dev(q), dev, kind, table, blocks, window, new, lens))
    row0 = new[0] - 1
    keep = np.arange(sum(new)) != row0
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step(kind))
    assert (np.abs(got - want)[keep] <= bound[keep]).all()
    assert not np.isfinite(got[row0]).any()


@pytest.mark.parametrize("size", [1e-30, 1e30, 3e38])
def test_queries_of_any_size(size):
    rng = np.random.default_rng(8)
    table, blocks, lens, total = _tree(rng, 1, 2, 1, 0, [30, 90])
    dev, (k, v) = _pools(rng, total, 1, 64, "bf16", 1.0 / size if size > 1 else 1.0)
    q = rng.uniform(-1, 1, (2, 2, 64)).astype(np.float32) * np.float32(size)
    got = _attend(to_dev(q), dev, "bf16", table, blocks, [0, 0], [1, 1], lens)
    want, bound = op.attention(q, k, v, table, blocks, [0, 0], [1, 1], lens, weight_step=_step("bf16"))
    _check(got, want, bound + 2e-40)


def test_strided_rows_other_streams_and_replays():
    d, t, rng = _dsb(), _torch(), np.random.default_rng(9)
    table, blocks, lens, total = _tree(rng, 2, 3, 2, 1, [5, 100, 200, 1, 64, 31])
    new = [1, 2, 1, 1, 3, 1]
    dev, _ = _pools(rng, total, 2, 128, "f16")
    rows = to_dev(rng.standard_normal((sum(new), 10 + 4, 128)).astype(np.float32))
    q = rows[:, :10]
    want = _attend(q.contiguous(), dev, "f16", table, blocks, [0] * 6, new, lens)
    assert t.equal(_attend(q, dev, "f16", table, blocks, [0] * 6, new, lens), want)
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table, blocks, [0] * 6, new, lens)
    ws = d.Workspace(sum(new), 10, 128, max(lens))
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    got = d.attention_decode_shared(q, kv, batch, ws, stream=side)
    side.synchronize()
    assert t.equal(got, want)
    out, graph = t.zeros_like(want), t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        d.attention_decode_shared(q, kv, batch, ws, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(out, want)


# ------------------------------------------------------------ bounds, selection
@pytest.mark.parametrize("kind,D,hkv,new,lens", [
    ("f16", 64, 1, [1], [1]), ("bf16", 128, 3, [1, 0, 200], [700, 30, 200]), ("f16", 128, 8, [5, 128, 1], [130, 128, 257]),
    ("bf16", 64, 2, [1000], [5000])])
def test_bounds_are_the_least_and_largest_keys(kind, D, hkv, new, lens):
    d, t, rng = _dsb(), _torch(), np.random.default_rng(D + len(new))
    table, blocks, lens, total = _tree(rng, 1, len(lens), 0, 0, lens)
    dev, (k, _) = _pools(rng, total, hkv, D, kind)
    dev[0][table[0, 0], 0, 0, 3] = float("nan")
    k = dev[0].double().cpu().numpy()
    before = t.full((total, hkv, 2, D), 7.0, dtype=_type(kind)[1], device="cuda")
    kv, batch = d.kv_pages(dev[0], dev[1], _type(kind)[0]), d.PagedBatch(table, blocks, [0] * len(lens), new, lens)
    got = d.kv_page_bounds(kv, batch, before)
    want = op.bounds(k, table, new, lens, np.full((total, hkv, 2, D), 7.0))
    assert np.array_equal(to_host(got.double()), want, equal_nan=True)


SELECT = [
    # kind, hq, hkv, D, new, lens, n_select, first, last
    ("f16", 1, 1, 64, [1], [1], 1, 0, 1),
    ("bf16", 12, 12, 64, [1], [5000], 8, 1, 1),
    ("f16", 10, 2, 128, [3, 0, 1], [4000, 300, 129], 5, 1, 2),
    ("bf16", 8, 1, 128, [1, 200], [20000, 900], 3, 0, 1),
    ("f16", 7, 1, 64, [2], [2000], 15, 1, 2),
    ("bf16", 40, 8, 128, [1] * 16, [700 + 100 * i for i in range(16)], 6, 1, 1),
    ("f16", 24, 1, 64, [1], [70000], 500, 1, 2),
    ("f16", 17, 1, 128, [1], [3000], 20, 10, 10),
]


@pytest.mark.parametrize("kind,hq,hkv,D,new,lens,n_select,first,last", SELECT)
@pytest.mark.parametrize("ties", [False, True])
def test_selection_matches_the_oracle(kind, hq, hkv, D, new, lens, n_select, first, last, ties):
    d, t, rng = _dsb(), _torch(), np.random.default_rng(n_select + hq + D)
    table, blocks, lens, total = _tree(rng, 1, len(lens), 0, 0, lens)
    bnd = rng.standard_normal((total, hkv, 2, D))
    if ties:
        bnd = np.round(bnd * 0.7) * (rng.random((total, hkv, 1, 1)) < 0.3)
    bnd.sort(axis=2)
    bnd = t.from_numpy(bnd).to(_type(kind)[1])
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32)
    if ties:
        q = np.round(q)
    pool = t.zeros((total, hkv, P, D), dtype=_type(kind)[1], device="cuda")
    kv, batch = d.kv_pages(pool, t.zeros_like(pool), _type(kind)[0]), d.PagedBatch(table, blocks, [0] * len(lens), new, lens)
    ws = d.Workspace(sum(new), hq, D, max(lens))
    got = d.kv_select_pages(to_dev(q), kv, bnd.cuda(), batch, n_select, ws, keep_first=first, keep_last=last)
    want = op.select(q, bnd.double().numpy(), table, new, lens, n_select, first, last)
    assert np.array_equal(to_host(got), want)


def test_a_page_with_a_nan_is_selected():
    d, t, rng = _dsb(), _torch(), np.random.default_rng(2)
    bnd = t.from_numpy(np.sort(rng.standard_normal((40, 1, 2, 64)), 2)).half().cuda()
    bnd[17] = float("nan")
    pool = t.zeros((40, 1, P, 64), dtype=t.float16, device="cuda")
    batch = d.PagedBatch(np.arange(40)[None], [40], [0], [1], [40 * P])
    got = d.kv_select_pages(t.randn((1, 1, 64), device="cuda"), d.kv_pages(pool, t.zeros_like(pool), d.DSB_F16), bnd,
                            batch, 2, d.Workspace(1, 1, 64, 40 * P), keep_first=0)
    assert to_host(got).tolist() == [[[17, 39]]]


# ------------------------------------------------------ attention, selected pages
@pytest.mark.parametrize("kind,hq,hkv,D,new,lens,n", [
    ("f16", 1, 1, 64, [1], [1], 1), ("bf16", 12, 12, 64, [1], [2000], 4), ("f16", 10, 2, 128, [3, 0, 1], [1500, 300, 129], 3),
    ("bf16", 18, 2, 128, [1, 2], [900, 640], 40), ("f16", 40, 8, 128, [1, 1], [1000, 130], 2)])
def test_selected_attention_matches_the_oracle(kind, hq, hkv, D, new, lens, n):
    rng = np.random.default_rng(hq + n + D)
    table, blocks, lens, total = _tree(rng, 1, len(lens), 0, 0, lens)
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32)
    sel = np.full((sum(new), hkv, n), -1, np.int32)
    row = 0
    for m, length in zip(new, lens):
        for j in range(m):
            mine = (length - m + j) // P
            for h in range(hkv):
                pick = np.sort(rng.permutation(mine + 1)[:n])
                sel[row, h, :len(pick)] = pick
            row += 1
    got = _attend(to_dev(q), dev, kind, table, blocks, [0] * len(lens), new, lens, selected=to_dev(sel))
    want, bound = op.attention(q, k, v, table, blocks, [0] * len(lens), new, lens, sel, weight_step=_step(kind))
    _check(got, want, bound)


def test_lists_of_any_content_stay_within_the_cache():
    """No block, blocks behind the token's own, the same twice, and nothing at all."""
    rng = np.random.default_rng(6)
    table, blocks, lens, total = _tree(rng, 1, 2, 0, 0, [500, 400])
    dev, (k, v) = _pools(rng, total, 1, 64, "f16")
    q = rng.standard_normal((3, 2, 64)).astype(np.float32)
    sel = np.array([[[2, -1, 2, 99]], [[-1, -1, -1, -1]], [[2 ** 31 - 1, -2 ** 31, 1, 3]]], np.int32)
    got = _attend(to_dev(q), dev, "f16", table, blocks, [0, 0], [2, 1], lens, selected=to_dev(sel))
    want, bound = op.attention(q, k, v, table, blocks, [0, 0], [2, 1], lens, sel)
    assert not to_host(got)[1].any()
    _check(got, want, bound)


# ------------------------------------------------------------------- together
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_a_forked_session_goes_on_like_its_parent(kind):
    """Append a prompt, fork it twice (pages shared, the last copied), append other
    tokens to each, attend over the shared pages, then select pages and attend over
    those: every result as the oracle's on the pages that are there."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(12)
    hq, hkv, D, n0 = 6, 2, 64, 1000
    dt, tt = _type(kind)
    pools = [t.zeros((40, hkv, P, D), dtype=tt, device="cuda") for _ in "kv"]
    kv, bounds = d.kv_pages(pools[0], pools[1], dt), t.zeros((40, hkv, 2, D), dtype=tt, device="cuda")
    rot, ws = d.Rotary(10000.0), d.Workspace(2000, hq, D, 4096)
    def step(table, blocks, new, lens, n_select=3):
        batch = d.PagedBatch(table, blocks, [0] * len(lens), new, lens)
        qkv = to_dev(rng.standard_normal((sum(new), (hq + 2 * hkv) * D)).astype(np.float32))
        d.kv_append_paged(qkv, hq, kv, batch, rot, ws)
        d.kv_page_bounds(kv, batch, bounds)
        q = qkv.view(sum(new), hq + 2 * hkv, D)[:, :hq]
        dense = d.attention_decode_shared(q, kv, batch, ws)
        sel = d.kv_select_pages(q, kv, bounds, batch, n_select, ws)
        return q, dense, sel, d.attention_decode_selected(q, kv, batch, sel, ws)
    table = np.zeros((3, 10), np.int32)
    table[0, :8] = [31, 2, 17, 5, 8, 21, 13, 39]
    step(table[:1], [8], [n0], [n0])
    # forks: 7 full pages shared, 104 keys of the eighth copied
    table[1:, :8] = table[0, :8]
    table[1:, 7] = [4, 6]
    d.kv_copy_pages([kv], [39, 39], [4, 6], [n0 % P] * 2)
    table[0, 8], table[1, 8] = 9, 10
    lens, new = [n0 + 30, n0 + 25, n0 + 1], [30, 25, 1]
    q, dense, sel, sparse = step(table, [9, 9, 8], new, lens)
    k, v = (x.double().cpu().numpy() for x in pools)
    host = to_host(q).astype(np.float64)
    want, bound = op.attention(host, k, v, table, [9, 9, 8], [0] * 3, new, lens, weight_step=_step(kind))
    _check(dense, want, bound, "dense")
    bnd = np.zeros((40, hkv, 2, D))
    bnd = op.bounds(k, table, lens, lens, bnd)               # of every page that a sequence has
    used = sorted({int(x) for s, n in enumerate(lens) for x in table[s, :-(-n // P)]})
    assert np.array_equal(to_host(bounds.double())[used], bnd[used])
    want_sel = op.select(to_host(q), bnd, table, new, lens, 3, 1, 1)
    assert np.array_equal(to_host(sel), want_sel)
    want, bound = op.attention(host, k, v, table, [9, 9, 8], [0] * 3, new, lens, want_sel, weight_step=_step(kind))
    _check(sparse, want, bound, "sparse")


# --------------------------- rows enough for the tcgen05 kernel (128 of them to a tile)
WIDE = [
    # a prompt on nothing; drafts of 16 sessions behind a prompt; many tiles on pages that are cut by CTAs' shares;
    # prompts behind a shared prefix, one of a single token
    ("f16", 10, 2, 128, 1, 1, 0, 0, [600], [600]),
    ("bf16", 40, 8, 64, 1, 16, 16, 0, [5 + 9 * i for i in range(16)], [4] * 14 + [1, 3]),
    ("f16", 32, 4, 128, 1, 30, 40, 0, [1 + i for i in range(30)], [1] * 30),
    ("bf16", 20, 2, 128, 1, 3, 2, 0, [300, 129, 1], [300, 129, 1]),
    ("f16", 64, 1, 64, 2, 2, 3, 1, [200, 100, 128, 257], [200, 7, 128, 30]),
]


@pytest.mark.parametrize("kind,hq,hkv,D,groups,per,common,branch,tails,new", WIDE)
def test_wide_tiles_match_the_oracle(kind, hq, hkv, D, groups, per, common, branch, tails, new):
    d, rng = _dsb(), np.random.default_rng(sum(tails) + hq + D)
    table, blocks, lens, total = _tree(rng, groups, per, common, branch, tails)
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32) * 2
    window = [0] * len(lens)
    got = _attend(to_dev(q), dev, kind, table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step(kind))
    _check(got, want, bound)
    again = _attend(to_dev(q), dev, kind, table, blocks, window, new, lens)
    assert _torch().equal(got, again)
    d.device_error()


def test_wide_tiles_on_rings():
    """Prompts under a window, and a long one whose tiles see other pages each."""
    rng = np.random.default_rng(21)
    new, window, lens = [400, 300, 250], [200, 0, 1], [1500, 700, 250]
    blocks = [(200 + 400 - 2) // P + 2, 6, 3]
    table = np.zeros((3, 8), np.int32)
    order = rng.permutation(20)
    for s, b in enumerate(blocks):
        table[s, :b] = order[6 * s:6 * s + b]
    dev, (k, v) = _pools(rng, 20, 1, 64, "bf16")
    q = rng.standard_normal((sum(new), 12, 64)).astype(np.float32)
    got = _attend(to_dev(q), dev, "bf16", table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step("bf16"))
    _check(got, want, bound)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_wide_tiles_leave_hidden_values_out(kind):
    """Infinite and NaN values of keys that only later tokens see, several to a page, and of no
    token's: rows that do not see them are as without."""
    t, rng = _torch(), np.random.default_rng(22)
    n, hq, hkv, D = 600, 10, 2, 128
    table, blocks, lens, total = _tree(rng, 1, 2, 1, 0, [n, n])
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    q = rng.standard_normal((2 * n, hq, D)).astype(np.float32)
    args = (kind, table, blocks, [0, 0], [n, n], lens)
    clean = to_host(_attend(to_dev(q), dev, *args))
    for s in (0, 1):                                         # behind the last keys
        dev[0][int(table[s, -1]), :, lens[s] % P:] = float("nan")
        dev[1][int(table[s, -1]), :, lens[s] % P:] = float("-inf")
    assert np.array_equal(to_host(_attend(to_dev(q), dev, *args)), clean)
    first = P + 300                                          # sequence 0's keys from position 428 on
    for p, value in ((first, "inf"), (first + 1, "nan"), (first + 57, "-inf"), (first + 200, "nan"), (lens[0] - 1, "inf")):
        dev[1][int(table[0, p // P]), :, p % P] = float(value)
    got = to_host(_attend(to_dev(q), dev, *args))
    want, bound = op.attention(q, k, v, table, blocks, [0, 0], [n, n], lens, weight_step=_step(kind))
    keep = np.ones(2 * n, bool)
    keep[300:n] = False
    assert (np.abs(got - want)[keep] <= bound[keep]).all()
    assert not np.isfinite(got[300:n]).any()


def test_wide_tiles_on_streams_and_in_graphs():
    """Calls of both kernels on two streams at once, each with a workspace of its own, and two
    graphs that share one."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(23)
    kind, hq, hkv, D = "bf16", 40, 8, 64
    table, blocks, lens, total = _tree(rng, 1, 16, 16, 0, [5 + 9 * i for i in range(16)])
    new = [4] * 16
    dev, _ = _pools(rng, total, hkv, D, kind)
    qs = [to_dev(rng.standard_normal((64, hq, D)).astype(np.float32)) for _ in range(2)]
    want = [_attend(q, dev, kind, table, blocks, [0] * 16, new, lens) for q in qs]
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_BF16), d.PagedBatch(table, blocks, [0] * 16, new, lens)
    spaces = [d.Workspace(64, hq, D, max(lens)) for _ in range(2)]
    streams = [t.cuda.Stream() for _ in range(2)]
    t.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i in (0, 1):
            got[i].append(d.attention_decode_shared(qs[i], kv, batch, spaces[i], stream=streams[i]))
    t.cuda.synchronize()
    assert all(t.equal(x, want[i]) for i in (0, 1) for x in got[i])
    outs, graphs = [t.zeros_like(w) for w in want], [t.cuda.CUDAGraph() for _ in want]
    for q, o, g in zip(qs, outs, graphs):
        with t.cuda.graph(g):
            d.attention_decode_shared(q, kv, batch, spaces[0], out=o)
    for _ in range(3):
        for o, g in zip(outs, graphs):
            o.zero_()
            g.replay()
        t.cuda.synchronize()
        assert all(t.equal(o, w) for o, w in zip(outs, want))


# ----------------------------------------------------- long contexts, large pools
@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_many_calls_give_the_same_bits(kind):
    """Samples of eight prompts: both kernels beside each other, short runs of tiles of 128 rows.
    A wait that could miss what it waits for would, in one of so many calls, run out."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(31)
    table, blocks, lens, total = _tree(rng, 8, 8, 8, 9, rng.integers(1, 700, 64))
    dev, _ = _pools(rng, total, 8, 128, kind)
    kv, batch = d.kv_pages(dev[0], dev[1], _type(kind)[0]), d.PagedBatch(table, blocks, [0] * 64, [1] * 64, lens)
    q, ws = to_dev(rng.standard_normal((64, 40, 128)).astype(np.float32)), d.Workspace(64, 40, 128, max(lens))
    want, out = d.attention_decode_shared(q, kv, batch, ws), t.empty_like(q)
    wrong = t.zeros((), dtype=t.int64, device="cuda")
    for i in range(20_000):
        d.attention_decode_shared(q, kv, batch, ws, out=out)
        if i % 20 == 0:
            wrong += (out != want).sum()
    assert int(wrong) == 0
    d.device_error()


def test_a_context_of_more_pages_than_a_segment_holds():
    rng = np.random.default_rng(24)
    n = 300_000
    table, blocks, lens, total = _tree(rng, 1, 1, 0, 0, [n])
    dev, (k, v) = _pools(rng, total, 1, 64, "f16")
    q = rng.standard_normal((1, 2, 64)).astype(np.float32)
    got = _attend(to_dev(q), dev, "f16", table, blocks, [0], [1], lens)
    want, bound = op.attention(q, k, v, table, blocks, [0], [1], lens)
    _check(got, want, bound)


def test_page_numbers_past_16_bits():
    """A pool of 70000 pages: numbers of 32 bits in every call, and byte offsets past 2^30."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(25)
    n_pages, hq, D, lens, new = 70_000, 6, 64, [1000, 700], [2, 1]
    used = np.sort(rng.permutation(2000)[:16]) + 68_000
    pools = [t.zeros((n_pages, 1, P, D), dtype=t.float16, device="cuda") for _ in "kv"]
    small = [t.from_numpy(rng.standard_normal((16, 1, P, D))).half() for _ in "kv"]
    for x, y in zip(pools, small):
        x[used] = y.cuda()
    bt = np.array([[3, 7, 1, 0, 9, 12, 4, 15], [3, 7, 5, 6, 2, 8, 0, 0]])
    table, blocks = used[bt].astype(np.int32), [8, 6]
    q = rng.standard_normal((3, hq, D)).astype(np.float32)
    kv, batch = d.kv_pages(*pools, d.DSB_F16), d.PagedBatch(table, blocks, [0, 0], new, lens)
    ws, qd = d.Workspace(3, hq, D, 1000), to_dev(q)
    k, v = (x.double().numpy() for x in small)
    want, bound = op.attention(q, k, v, bt, blocks, [0, 0], new, lens)
    _check(d.attention_decode_shared(qd, kv, batch, ws), want, bound)
    bnd = t.zeros((n_pages, 1, 2, D), dtype=t.float16, device="cuda")
    d.kv_page_bounds(kv, d.PagedBatch(table[:1], blocks[:1], [0], lens[:1], lens[:1]), bnd)
    d.kv_page_bounds(kv, d.PagedBatch(table[1:, 2:6], [4], [0], [700 - 2 * P], [700 - 2 * P]), bnd)
    host = op.bounds(k, bt, [1000, 0], lens, np.zeros((16, 1, 2, D)))
    host = op.bounds(k, bt[1:, 2:], [700 - 2 * P], [700 - 2 * P], host)
    assert np.array_equal(to_host(bnd[used].double()), host)
    sel = d.kv_select_pages(qd, kv, bnd, batch, 3, ws)
    pick = op.select(q, host, bt, new, lens, 3, 1, 1)
    assert np.array_equal(to_host(sel), pick)
    want, bound = op.attention(q, k, v, bt, blocks, [0, 0], new, lens, pick)
    _check(d.attention_decode_selected(qd, kv, batch, sel, ws), want, bound)
    d.kv_copy_pages([kv], [int(used[3])], [69_999 if 69_999 not in used else 67_000], [77])
    at = 69_999 if 69_999 not in used else 67_000
    assert t.equal(pools[0][at, :, :77].cpu(), small[0][3, :, :77]) and not pools[0][at, :, 77:].any()


def test_selection_among_more_pages_than_shared_memory_has_without_asking():
    d, t, rng = _dsb(), _torch(), np.random.default_rng(26)
    n = 14_000
    bnd = np.sort(rng.standard_normal((n, 1, 2, 64)), 2)
    bnd = t.from_numpy(bnd).half()
    pool = t.zeros((n, 1, P, 64), dtype=t.float16, device="cuda")
    batch = d.PagedBatch(rng.permutation(n)[None].astype(np.int32), [n], [0], [1], [n * P - 3])
    q = rng.standard_normal((1, 3, 64)).astype(np.float32)
    got = d.kv_select_pages(to_dev(q), d.kv_pages(pool, pool.clone(), d.DSB_F16), bnd.cuda(), batch, 100,
                            d.Workspace(1, 3, 64, n * P), keep_first=2, keep_last=3)
    want = op.select(q, bnd.double().numpy(), batch._arrays[0], [1], [n * P - 3], 100, 2, 3)
    assert np.array_equal(to_host(got), want)


def test_more_rows_than_the_gpu_holds_warps():
    """Prompts beside single tokens: rows in one part and in several, several to a warp of the join."""
    rng = np.random.default_rng(30)
    kind, hq, hkv, D = "f16", 40, 2, 64
    table, blocks, lens, total = _tree(rng, 1, 5, 1, 0, [260, 5, 131, 400, 60])
    new = [250, 1, 128, 90, 0]
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32)
    assert len(q) * hq > 16384
    got = _attend(to_dev(q), dev, kind, table, blocks, [0] * 5, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, [0] * 5, new, lens)
    _check(got, want, bound)


def test_more_metadata_than_places_for_it():
    """1024 sequences of 340 pages each: 18 launches, and 16 places for staged metadata.  Tables
    repeat the pages of a small pool, so that a key's weight is its own times how often its
    page is listed."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(28)
    n_seq, n, total, hq, D = 1024, 340, 64, 2, 64
    table = rng.integers(0, total, (n_seq, n)).astype(np.int32)
    dev, _ = _pools(rng, total, 1, D, "f16")
    q = to_dev(rng.standard_normal((n_seq, hq, D)).astype(np.float32))
    got = _attend(q, dev, "f16", table, [n] * n_seq, [0] * n_seq, [1] * n_seq, [n * P] * n_seq).double()
    k, v = (x.double().reshape(total * P, D) for x in dev)
    often = np.stack([np.bincount(row, minlength=total) for row in table])
    often = t.from_numpy(np.repeat(often, P, 1)).double().cuda()
    for s in range(0, n_seq, 32):
        x, times = q[s:s + 32].double(), often[s:s + 32, None, :]
        score = x @ k.T / 8
        size = (x.abs() @ k.abs().T).amax(-1)[..., None] / 8
        e = t.exp(score - score.amax(-1, keepdim=True))
        total_e = (e * times).sum(-1, keepdim=True)
        e, one = e * times / total_e, (e / total_e).amax(-1)[..., None]
        want = e @ v
        apart = t.stack([(e[i, :, :, None] * (v[None] - want[i, :, None, :]).abs()).sum(1) for i in range(len(x))])
        bound = 2.0 ** -20 * 2 * (size + 1) * apart + 2.0 ** -20 * (e @ v.abs())      # the oracle's
        bound += 2.0 ** -35 * one * (times @ v.abs())
        assert bool(((got[s:s + 32] - want).abs() <= bound).all()), f"sequences {s} on"


def test_selections_of_two_threads():
    """Lists that need more shared memory than a launch has without asking, beside short ones."""
    import threading
    d, t, rng = _dsb(), _torch(), np.random.default_rng(29)
    n = 14_000
    bnd = t.from_numpy(np.sort(rng.standard_normal((n, 1, 2, 64)), 2)).half().cuda()
    pool = t.zeros((n, 1, P, 64), dtype=t.float16, device="cuda")
    kv = d.kv_pages(pool, pool.clone(), d.DSB_F16)
    order = rng.permutation(n)[None].astype(np.int32)
    q = to_dev(rng.standard_normal((1, 3, 64)).astype(np.float32))
    lens = [n * P - 3, 10_400 * P]
    want = [None, None]
    got, errors = [[], []], []

    def run(i, times):
        try:
            ws, st = d.Workspace(1, 3, 64, lens[i]), t.cuda.Stream()
            batch = d.PagedBatch(order, [n], [0], [1], [lens[i]])
            for _ in range(times):
                got[i].append(d.kv_select_pages(q, kv, bnd, batch, 100, ws, stream=st))
            st.synchronize()
        except Exception as e:  # told by the test's own thread
            errors.append(e)

    t.cuda.synchronize()
    for i in (0, 1):
        run(i, 1)
        want[i] = got[i].pop()
    threads = [threading.Thread(target=run, args=(i, 200)) for i in (0, 1)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not errors
    assert all(len(got[i]) == 200 and all(t.equal(x, want[i]) for x in got[i]) for i in (0, 1))


# ------------------------------------------------------- memory around the outputs
def _banded(shape, dtype):
    """A tensor between two bands of a pattern in one allocation, and the bands."""
    t = _torch()
    n = int(np.prod(shape)) * t.empty(0, dtype=dtype).element_size()
    raw = t.full((n + 16384,), 0xA5, dtype=t.uint8, device="cuda")
    return raw[8192:8192 + n].view(dtype).view(shape), (raw[:8192], raw[8192 + n:])


def test_calls_write_their_outputs_and_nothing_around():
    d, t, rng = _dsb(), _torch(), np.random.default_rng(27)
    table, blocks, lens, total = _tree(rng, 1, 3, 2, 0, [5, 131, 70])
    new, hq, hkv, D = [1, 3, 2], 6, 2, 64
    bands = []
    def banded(shape, dtype):
        x, b = _banded(shape, dtype)
        bands.extend(b)
        return x
    pools = [banded((total, hkv, P, D), t.float16) for _ in "kv"]
    for x in pools:
        x.copy_(t.from_numpy(rng.standard_normal(x.shape)))
    kv, batch = d.kv_pages(*pools, d.DSB_F16), d.PagedBatch(table, blocks, [0] * 3, new, lens)
    ws, q = d.Workspace(6, hq, D, max(lens)), to_dev(rng.standard_normal((6, hq, D)).astype(np.float32))
    bnd, sel = banded((total, hkv, 2, D), t.float16), banded((6, hkv, 2), t.int32)
    outs = [banded((6, hq, D), t.float32) for _ in range(2)]
    bnd.zero_()
    d.kv_page_bounds(kv, batch, bnd)
    d.kv_select_pages(q, kv, bnd, batch, 2, ws, selected=sel)
    d.attention_decode_shared(q, kv, batch, ws, out=outs[0])
    d.attention_decode_selected(q, kv, batch, sel, ws, out=outs[1])
    was = [x.clone() for x in pools]
    free = [p for p in range(total) if p not in set(table.ravel().tolist())]
    d.kv_copy_pages([kv], [int(table[0, 0])], free[:1], [33])
    for x, y in zip(pools, was):
        y[free[0], :, :33] = y[int(table[0, 0]), :, :33]
        assert t.equal(x, y)
    assert t.equal(outs[0], d.attention_decode_shared(q, kv, batch, ws))
    assert t.equal(outs[1], d.attention_decode_selected(q, kv, batch, sel, ws))
    assert all(bool((b == 0xA5).all()) for b in bands)
