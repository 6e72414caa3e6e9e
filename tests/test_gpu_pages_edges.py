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
