"""GPU tests of the calls on whole pages at their edges: calls of several launches,
captured and not, lists of any length, large groups and batches, caches near their
type's ends.  Helpers, readings and bounds as in test_gpu_pages."""
import numpy as np
import pytest

from oracle import pages as op
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_pages import P, _attend, _check, _dsb, _pools, _step, _torch, _tree, _type

pytestmark = pytest.mark.gpu


def _captured(call):
    """call(), captured into a graph and replayed; its result."""
    t = _torch()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        out = call()
    out.fill_(7)                                             # its own memory: written by the replay
    graph.replay()
    t.cuda.synchronize()
    return out


# ------------------------------------------------------- calls of several launches
@pytest.mark.parametrize("long,short", [(7, 300), (8, 300)])
def test_lists_are_read_alike_in_every_launch(long, short):
    """Some long sequences, then short ones: cut into launches of which the last holds short ones
    alone (the first case uncaptured, the second captured).  Lists of the short ones begin with
    entries that are no block."""
    d, rng = _dsb(), np.random.default_rng(long)
    hq, D, n, total = 2, 64, 3000, 64
    lens = [n * P - 5 * i for i in range(long)] + [1 + int(x) for x in rng.integers(0, 2 * P, short)]
    new = [1] * len(lens)
    table = rng.integers(0, total, (len(lens), n)).astype(np.int32)
    dev, (k, v) = _pools(rng, total, 1, D, "f16")
    q = rng.standard_normal((len(lens), hq, D)).astype(np.float32)
    sel = np.full((len(lens), 1, 5), -1, np.int32)
    for s in range(len(lens)):
        blocks = -(-lens[s] // P)
        if s < long:
            sel[s, 0] = np.sort(rng.permutation(blocks)[:5])
        else:
            sel[s, 0, 3] = blocks - 1
            sel[s, 0, 4] = 0                                  # the first page, of some the only one: twice
    blocks, window = [n] * len(lens), [0] * len(lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, sel)
    qd, sd = to_dev(q), to_dev(sel)
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table, blocks, window, new, lens)
    ws = d.Workspace(len(lens), hq, D, max(lens))
    call = lambda: d.attention_decode_selected(qd, kv, batch, sd, ws)
    _check(call(), want, bound, "called")
    _check(_captured(call), want, bound, "captured")


def test_selected_pages_of_long_prompts_and_many_heads():
    """More rows times listed pages than a launch counts: a prompt of 8192 tokens, 64 heads, 2100 pages
    of a small pool."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(41)
    new, h, D, n, total = 8192, 64, 64, 2100, 8
    table = rng.integers(0, total, (1, n)).astype(np.int32)
    dev, (k, v) = _pools(rng, total, h, D, "f16")
    q = t.from_numpy(rng.standard_normal((1, h, D)).astype(np.float32)).cuda().expand(new, h, D).contiguous()
    sel = t.full((new, h, n), -1, dtype=t.int32, device="cuda")
    sel[:, :, n - 2] = t.arange(new, device="cuda")[:, None] % (n - new // P)       # a page that every token sees
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table, [n], [0], [new], [n * P])
    got = d.attention_decode_selected(q, kv, batch, sel, d.Workspace(64, h, D, n * P))
    one = q[:1].double().cpu().numpy()
    for b in range(total):                                   # the rows of a page are all alike
        at = np.flatnonzero(table[0, np.arange(new) % (n - new // P)] == b)
        want, bound = op.attention(one, k, v, np.array([[b]]), [1], [0], [1], [P])
        x = to_host(got[t.from_numpy(at).cuda()]).astype(np.float64)
        assert (np.abs(x - want) <= bound).all(), f"page {b}"


# ------------------------------------------------- many sessions, large groups
@pytest.mark.parametrize("groups,per,branch,most", [(1, 1024, 0, 1), (128, 8, 3, 1), (1, 1024, 0, 4), (4, 256, 1, 3)])
def test_a_thousand_sessions_behind_one_prompt(groups, per, branch, most):
    """More sessions on the same pages than one launch's metadata holds, of one or of up to `most` new
    tokens each, called and captured."""
    d, rng = _dsb(), np.random.default_rng(per + most)
    n, hq, D = 1024, 2, 64
    table, blocks, lens, total = _tree(rng, groups, per, 2, branch, rng.integers(most, 200, n))
    new = [1] * n if most == 1 else rng.integers(0, most + 1, n).tolist()
    dev, (k, v) = _pools(rng, total, 1, D, "f16")
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32)
    want, bound = op.attention(q, k, v, table, blocks, [0] * n, new, lens)
    qd, kv, batch = to_dev(q), d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table, blocks, [0] * n, new, lens)
    ws = d.Workspace(sum(new), hq, D, max(lens))
    call = lambda: d.attention_decode_shared(qd, kv, batch, ws)
    _check(call(), want, bound, "called")
    _check(_captured(call), want, bound, "captured")


def _prompt_errors(got, q, k, v, pages, len_, window=0):
    """Largest error of a prompt's rows over the oracle's bound, in which |v - out| is no more than
    |v| + |out|: got, q [tokens, hq, D] of the last tokens of len_ keys, one kv head, device tensors."""
    t = _torch()
    n, hq, D = got.shape
    key, val = (x[pages, 0].double().reshape(-1, D)[:len_] for x in (k, v))
    at, worst = t.arange(len_, device="cuda"), 0.0
    p = t.arange(len_ - n, len_, device="cuda")[:, None]
    hidden = (at > p) | (at <= p - window if window else at < 0)
    for h in range(hq):
        x = q[:, h].double()
        score = (x @ key.T / D ** 0.5).masked_fill_(hidden, -np.inf)
        size = (x.abs() @ key.abs().T).masked_fill_(hidden, 0).amax(-1, keepdim=True) / D ** 0.5
        e = t.softmax(score, -1)
        want, mag = e @ val, e @ val.abs()
        bound = 2.0 ** -20 * 2 * (size + 1) * (mag + want.abs()) + 2.0 ** -20 * mag
        bound += 2.0 ** -35 * e.amax(-1, keepdim=True) * ((~hidden).double() @ val.abs())
        worst = max(worst, float(((got[:, h].double() - want).abs() / bound).max()))
    return worst


@pytest.mark.parametrize("hq,new,before,window,captured", [
    (64, 4096, 0, 0, True), (128, 8192, 0, 0, False), (128, 8192, 0, 0, True), (80, 4000, 500, 300, True), (5, 8192, 300, 0, True)])
def test_prompts_of_many_rows(hq, new, before, window, captured):
    """More tiles of rows than one launch's metadata has places for what each sees."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(hq)
    D, len_ = 64, new + before
    n = -(-len_ // P)
    nb = -(-(window + new - 1) // P) + 1 if window else n
    order = rng.permutation(n + 2)
    dev = [t.randn((n + 2, 1, P, D), device="cuda", generator=t.Generator("cuda").manual_seed(i)).half() for i in (1, 2)]
    table = order[:nb] if window else order[:n]
    pages = [int(table[i % nb]) for i in range(n)]           # (what a ring's older blocks held, no row sees)
    q = t.randn((new, hq, D), device="cuda", generator=t.Generator("cuda").manual_seed(3))
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table[None].astype(np.int32), [nb], [window], [new], [len_])
    ws = d.Workspace(new, hq, D, len_)
    call = lambda: d.attention_decode_shared(q, kv, batch, ws)
    got = _captured(call) if captured else call()
    assert _prompt_errors(got, q, dev[0], dev[1], pages, len_, window) <= 1
    d.device_error()


# ------------------------------------------------------ the ends of a type's range
FORMS = [
    # hq, hkv, tails, new: rows for the warp-level kernel, and for the tcgen05 one
    (4, 2, [30, 500], [1, 2]), (2, 1, [40_000], [1]), (20, 2, [600, 300], [600, 2])]


def _far(rng, hq, hkv, tails, new, ksize, vsize, qsize, D=64):
    table, blocks, lens, total = _tree(rng, 1, len(tails), 1, 0, tails)
    t = _torch()
    host = [np.clip(rng.standard_normal((total, hkv, P, D)), -3, 3) * x for x in (ksize, vsize)]
    dev = [t.from_numpy(x).bfloat16().cuda() for x in host]
    q = (rng.standard_normal((sum(new), hq, D)) * qsize).astype(np.float32)
    return dev, [x.double().cpu().numpy() for x in dev], q, table, blocks, [0] * len(lens), lens


@pytest.mark.parametrize("hq,hkv,tails,new", FORMS)
@pytest.mark.parametrize("ksize,qsize", [(2.0 ** 100, 2.0 ** -100), (2.0 ** 118, 2.0 ** -117), (2.0 ** 126, 2.0 ** -124),
                                         (2.0 ** -100, 2.0 ** 100)])
def test_bf16_keys_of_any_size(hq, hkv, tails, new, ksize, qsize):
    rng = np.random.default_rng(hq)
    dev, (k, v), q, table, blocks, window, lens = _far(rng, hq, hkv, tails, new, ksize, 1.0, qsize)
    got = _attend(to_dev(q), dev, "bf16", table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step("bf16"))
    _check(got, want, bound)


@pytest.mark.parametrize("hq,hkv,tails,new", FORMS)
@pytest.mark.parametrize("vsize", [2.0 ** 100, 2.0 ** 118, 2.0 ** 126, 2.0 ** -90])
def test_bf16_values_of_any_size(hq, hkv, tails, new, vsize):
    rng = np.random.default_rng(hq)
    dev, (k, v), q, table, blocks, window, lens = _far(rng, hq, hkv, tails, new, 1.0, vsize, 1.0)
    got = _attend(to_dev(q), dev, "bf16", table, blocks, window, new, lens)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, weight_step=_step("bf16"))
    _check(got, want, bound)


@pytest.mark.parametrize("hq,hkv,tails,new", FORMS)
def test_the_largest_bf16_values(hq, hkv, tails, new):
    """Every value the type's largest, every score alike: a row's result is that value, to the rounding
    of a sum of weights and of one quotient."""
    rng, t = np.random.default_rng(hq), _torch()
    dev, _, q, table, blocks, window, lens = _far(rng, hq, hkv, tails, new, 0.0, 0.0, 1.0)
    most = t.finfo(t.bfloat16).max
    dev[1].fill_(most)
    got = to_host(_attend(to_dev(q), dev, "bf16", table, blocks, window, new, lens)).astype(np.float64)
    assert (np.abs(got - most) <= most * 2.0 ** -20).all()


@pytest.mark.parametrize("ksize,qsize,vsize", [(2.0 ** 118, 2.0 ** -117, 1.0), (1.0, 1.0, 2.0 ** 126)])
def test_selected_pages_of_any_size(ksize, qsize, vsize):
    rng = np.random.default_rng(51)
    hkv, new = 2, [1, 3]
    dev, (k, v), q, table, blocks, window, lens = _far(rng, 10, hkv, [3000, 5000], new, ksize, vsize, qsize)
    sel = np.full((4, hkv, 45), -1, np.int32)
    for i, (s, p) in enumerate([(0, lens[0] - 1)] + [(1, lens[1] - 3 + j) for j in range(3)]):
        sel[i, :, :p // P + 1] = np.arange(p // P + 1)
    got = _attend(to_dev(q), dev, "bf16", table, blocks, window, new, lens, selected=to_dev(sel))
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, sel, weight_step=_step("bf16"))
    _check(got, want, bound)


# ----------------------------------------------- lists and calls of every length
@pytest.mark.parametrize("kind,hq,hkv,D,n", [("f16", 5, 1, 64, 33), ("bf16", 16, 2, 128, 32), ("f16", 8, 1, 128, 97),
                                             ("bf16", 3, 3, 64, 200)])
def test_lists_of_any_length(kind, hq, hkv, D, n):
    """Lists past the 32 entries that a warp's lanes hold, NaN behind the last keys and on pages of nobody."""
    t, rng = _torch(), np.random.default_rng(n)
    lens, new = [29_000, 9_000, 200], [2, 1, 3]
    table, blocks, _, total = _tree(rng, 1, 3, 0, 0, lens)
    dev, (k, v) = _pools(rng, total, hkv, D, kind)
    for x in dev:
        for s, m in enumerate(lens):
            x[int(table[s, blocks[s] - 1]), :, (m - 1) % P + 1:] = float("nan")
        x[t.tensor(sorted(set(range(total)) - {int(b) for s in range(3) for b in table[s, :blocks[s]]})).cuda()] = float("inf")
    q = rng.standard_normal((6, hq, D)).astype(np.float32)
    sel = np.full((6, hkv, n), -1, np.int32)
    for row, (s, p) in enumerate([(0, 28_998), (0, 28_999), (1, 8_999), (2, 197), (2, 198), (2, 199)]):
        for h in range(hkv):
            pick = np.sort(np.append(rng.permutation(p // P)[:n - 1 - row % 2], p // P))
            sel[row, h, :len(pick)] = pick
    sel[1] = sel[1, :, ::-1]                                 # in another order, behind what is no block
    got = _attend(to_dev(q), dev, kind, table, blocks, [0] * 3, new, lens, selected=to_dev(sel))
    want, bound = op.attention(q, k, v, table, blocks, [0] * 3, new, lens, sel, weight_step=_step(kind))
    _check(got, want, bound)


@pytest.mark.parametrize("n_seq,pages", [(3, 3500), (90, 500), (1000, 8)])
def test_selections_of_several_launches(n_seq, pages):
    """Metadata beyond a launch's parameters and beyond a place for staged words, called and captured: the
    selection, and the attention over what it selects."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(n_seq)
    hq, hkv, D, total, n_select = 4, 2, 64, 48, 6
    table = rng.integers(0, total, (n_seq, pages)).astype(np.int32)
    lens = [int(x) for x in rng.integers(pages * P // 2, pages * P, n_seq)]
    new = [int(x) for x in rng.integers(0, 3, n_seq)]
    blocks, window = [pages] * n_seq, [0] * n_seq
    dev, (k, v) = _pools(rng, total, hkv, D, "f16")
    bnd = np.sort(rng.standard_normal((total, hkv, 2, D)), 2)
    bnd = t.from_numpy(bnd).half()
    q = rng.standard_normal((sum(new), hq, D)).astype(np.float32)
    qd, bd = to_dev(q), bnd.cuda()
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_F16), d.PagedBatch(table, blocks, window, new, lens)
    ws = d.Workspace(sum(new), hq, D, max(lens))
    pick = lambda: d.kv_select_pages(qd, kv, bd, batch, n_select, ws, keep_first=1, keep_last=2)
    want_sel = op.select(q, bnd.double().numpy(), table, new, lens, n_select, 1, 2)
    sel = pick()
    assert np.array_equal(to_host(sel), want_sel)
    assert np.array_equal(to_host(_captured(pick)), want_sel)
    want, bound = op.attention(q, k, v, table, blocks, window, new, lens, want_sel)
    call = lambda: d.attention_decode_selected(qd, kv, batch, sel, ws)
    _check(call(), want, bound, "called")
    _check(_captured(call), want, bound, "captured")


def test_copies_and_bounds_in_a_graph():
    """A fork's copy and the bounds of the pages that new tokens lie on, captured and replayed on other
    contents."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(43)
    table, blocks, lens, total = _tree(rng, 1, 3, 2, 0, [5, 131, 70], spare=4)
    new, hkv, D = [1, 140, 2], 2, 64
    dev, _ = _pools(rng, total, hkv, D, "bf16")
    q4 = to_dev(rng.integers(0, 256, (total, hkv, P * (D + 8)), dtype=np.uint8))
    bnd = t.zeros((total, hkv, 2, D), dtype=t.bfloat16, device="cuda")
    kv, batch = d.kv_pages(dev[0], dev[1], d.DSB_BF16), d.PagedBatch(table, blocks, [0] * 3, new, lens)
    free = [p for p in range(total) if p not in set(table.ravel().tolist())]
    src, dst, keys = [int(table[0, 2]), int(table[1, 0])], free[:2], [5, 128]
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        d.kv_copy_pages([kv], src, dst, keys)
        d.kv_copy_pages_q4([d.kv_q4_pages(q4, D)], src, dst, keys)
        d.kv_page_bounds(kv, batch, bnd)
    for seed in (1, 2):
        for x in dev:
            x.copy_(t.from_numpy(np.random.default_rng(seed).standard_normal(x.shape)))
        q4.copy_(to_dev(np.random.default_rng(seed).integers(0, 256, q4.shape, dtype=np.uint8)))
        was = [x.view(t.int16).cpu().numpy() for x in dev] + [to_host(q4)]
        graph.replay()
        t.cuda.synchronize()
        for x, y in zip(dev, was):
            assert np.array_equal(to_host(x.view(t.int16)), op.copy(y, src, dst, keys))
        assert np.array_equal(to_host(q4), op.copy_q4(was[2], D, src, dst, keys))
        want = op.bounds(dev[0].double().cpu().numpy(), table, new, lens, np.zeros((total, hkv, 2, D)))
        assert np.array_equal(to_host(bnd.double()), want)


def test_4bit_copies_in_every_layer():
    """All 40 layers' pools, whole: of the keys that are copied the source's bytes, of the others their own."""
    d, rng = _dsb(), np.random.default_rng(44)
    layers, n, hkv, D = 40, 5, 8, 128
    host = rng.integers(0, 256, (layers, n, hkv, P * (D + 8)), dtype=np.uint8)
    dev = to_dev(host)
    src, dst, keys = [3, 3], [0, 4], [4, 7]
    d.kv_copy_pages_q4([d.kv_q4_pages(p, D) for p in dev], src, dst, keys)
    # which key a byte belongs to: the oracle's copy of one key's bytes onto zeros, key by key
    owner = np.full(P * (D + 8), -1)
    for key in range(P):
        ones = np.full((2, 1, P * (D + 8)), 255, np.uint8)
        ones[1] = 0
        whole, less = (op.copy_q4(ones, D, [0], [1], [m])[1, 0] for m in (key + 1, key))
        owner[whole != less] = key
    assert (owner >= 0).all()
    want = host.copy()
    for a, b, m in zip(src, dst, keys):
        want[:, b] = np.where(owner < m, host[:, a], host[:, b])
    assert np.array_equal(to_host(dev), want)


@pytest.mark.parametrize("hq,new,D", [(20, 7, 64), (20, 7, 128), (20, 600, 64), (20, 600, 128)])
def test_bf16_weights_keep_float32s_bits(hq, new, D):
    """A prompt whose first key is the only one with a value (1) and a score: token p's result is w / (w + p)
    with w = exp(score) in (1/2, 1].  Off by: the score (below 1 in powers of two; the factor, q's product and
    parts, the products' sum, the reference) 2^-22, exp2 2^-22, the sum of the weight's parts 2^-22, the sum of
    up to 64 weights, the quotient and a join 2^-22; together 2^-20, half of the bound.  A weight as two
    bf16 is up to 2^-18 off."""
    d, t, rng = _dsb(), _torch(), np.random.default_rng(new + D)
    n, rows = -(-new // P), min(new, 64)
    k, v = (t.zeros((n, 1, P, D), dtype=t.bfloat16, device="cuda") for _ in "kv")
    k[0, 0, 0, 0], v[0, 0, 0] = 1, 1
    q = np.zeros((new, hq, D), np.float32)
    q[..., 0] = rng.uniform(-np.log(2), 0, (new, hq)) * D ** 0.5
    got = to_host(_attend(to_dev(q), [k, v], "bf16", np.arange(n, dtype=np.int32)[None], [n], [0], [new], [new]))[:rows]
    w = np.exp(q[:rows, :, 0].astype(np.float64) / D ** 0.5)
    want = w / (w + np.arange(rows)[:, None])
    off = np.abs(got - want[..., None]) / want[..., None]
    assert off.max() <= 2.0 ** -19, off.max() * 2 ** 19
    # the same with a mistake: weights of two bf16 leave the bound
    def bf16(x):
        return t.from_numpy(x).bfloat16().double().numpy()
    wrong = (bf16(w) + bf16(w - bf16(w))) / (w + np.arange(rows)[:, None])
    assert (np.abs(wrong - want) / want).max() > 2.0 ** -19
