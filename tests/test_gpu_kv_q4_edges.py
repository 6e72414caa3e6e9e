"""GPU tests of the rotary, paged-append and 4-bit KV calls at their edges: what
a key that a row does not see may hold, scales far apart, many sessions, long
prompts, and the hand-overs inside a CTA.  Helpers, readings and bounds as in
test_gpu_kv_q4."""
import numpy as np
import pytest

from tests.gpu_util import to_dev
from tests.test_gpu_kv_q4 import _dsb, _pool

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,group,new", [(64, 1, 1), (64, 2, 3), (128, 1, 2), (128, 8, 1)])
def test_one_cta_after_many_units(cuda_device, D, group, new):
    """More units than the GPU has room for, so that every CTA joins several one
    after the other, with one to four threads' worth of live rows: the same bits
    as a few sequences at a time, call after call."""
    import torch
    d = _dsb()
    n, hkv = 96, 12
    rng = np.random.default_rng(D + group)
    lens = rng.integers(600, 1000, n)
    pool = to_dev(_pool(rng, 20, 1, D)).expand(20, hkv, -1).contiguous()
    bt = rng.integers(0, 20, (n, 8)).astype(np.int32)
    q = torch.from_numpy(rng.standard_normal((n * new, hkv * group, D)).astype(np.float32)).cuda()
    kv, ws = d.kv_q4_pages(pool, D), d.Workspace(n * new, hkv * group, D, 1024)
    part = [d.attention_decode_q4(q[s * new:(s + 4) * new], kv,
                                  d.PagedBatch(bt[s:s + 4], [8] * 4, [0] * 4, [new] * 4, lens[s:s + 4]), ws)
            for s in range(0, n, 4)]
    want = torch.cat(part)
    batch = d.PagedBatch(bt, [8] * n, [0] * n, [new] * n, lens)
    for _ in range(20):
        assert torch.equal(d.attention_decode_q4(q, kv, batch, ws), want)
    d.device_error()
