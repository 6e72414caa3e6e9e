"""GPU tests of the rotary, paged-append and 4-bit KV calls at their edges: what
a key that a row does not see may hold, scales far apart, many sessions, long
prompts, and the hand-overs inside a CTA.  Helpers, readings and bounds as in
test_gpu_kv_q4."""
import numpy as np
import pytest

from oracle import kv_q4 as oq4
from oracle import rotary as orot
from tests.gpu_util import to_dev, to_host
from tests.test_gpu_kv_q4 import P, _dsb, _geometry, _partner, _pool, _rot

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


def _hidden_case(D, T, L, rng, vsize):
    """A pool whose V vectors are of size ``vsize``, the last T keys new."""
    n = -(-L // P)
    return _pool(rng, n, 1, D, vsize), [list(range(n))]


def _numbers(pool, key, D, which, d=None, z=None):
    """Copy of the pool with key ``key``'s (d, z) of K (0) or V (1) replaced."""
    out = pool.copy()
    at = P * D // 2 + which * (P * D // 2 + 4 * P) + 4 * (key % P)
    for i, x in ((0, d), (2, z)):
        if x is not None:
            out[key // P, :, at + i:at + i + 2] = np.frombuffer(np.float16(x).tobytes(), np.uint8)
    return out


FORMS = [(64, 1, 3, 200), (64, 4, 2, 135), (128, 2, 2, 129), (128, 3, 4, 300), (128, 8, 3, 2400)]  # D, hq, T, L


@pytest.mark.parametrize("D,hq,T,L", FORMS)
def test_a_row_does_not_depend_on_keys_it_does_not_see(cuda_device, D, hq, T, L):
    """Whatever the numbers of a later draft's key are, the rows before it keep
    their bits (both kernels, 4 and 8 rows a product)."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(D + L)
    pool, bt = _hidden_case(D, T, L, rng, 1e-3)
    q = to_dev(rng.standard_normal((T, hq, D)).astype(np.float32))
    b, ws = d.PagedBatch(bt, [len(bt[0])], [0], [T], [L]), d.Workspace(T, hq, D, L)
    clean = d.attention_decode_q4(q, d.kv_q4_pages(to_dev(pool), D), b, ws)
    assert torch.isfinite(clean).all()
    nan, inf = float("nan"), float("inf")
    for key in (L - 1, L - T + 1):
        first = key - (L - T)                # the row that is the first to see it
        for which, dd, z in ((0, nan, nan), (0, 60000.0, 0.0), (1, nan, nan), (1, nan, 0.0), (1, inf, None), (1, 60000.0, 0.0),
                             (1, 2.0 ** -24, 0.0), (1, 0.0, 0.0)):
            got = d.attention_decode_q4(q, d.kv_q4_pages(to_dev(_numbers(pool, key, D, which, dd, z)), D), b, ws)
            assert torch.equal(got[:first], clean[:first]), (key, which, dd)
            if not np.isfinite(dd):
                assert not torch.isfinite(got[first:]).any()
    d.device_error()


@pytest.mark.parametrize("D,hq,T,L", FORMS)
@pytest.mark.parametrize("ratio", [16, 20, 25])
def test_scales_far_apart(cuda_device, D, hq, T, L, ratio):
    """Every 20th key has V vectors 2^ratio times the others' and a score 2^-(ratio
    + 24) of theirs in weight, so that it does not count: the keys that do keep
    their bits."""
    d = _dsb()
    rng = np.random.default_rng(ratio)
    n = -(-L // P)
    k = rng.standard_normal((n * P, D)) * 0.02
    k[:, 0] = 0.0
    v = rng.standard_normal((n * P, D)) * 2.0 ** -11
    k[::20, 0], v[::20] = -20.0, v[::20] * 2.0 ** ratio
    pool = np.stack([oq4.pack_block(*oq4.quantise(k[a:a + P]), *oq4.quantise(v[a:a + P])) for a in range(0, n * P, P)])[:, None]
    q = (rng.standard_normal((T, hq, D)) * 0.1).astype(np.float32)
    q[..., 0] = (ratio + 24) * np.log(2) * np.sqrt(D) / 20
    kvals, vvals = oq4.pool_values(pool, D)
    bt = [list(range(n))]
    want, bound = oq4.attention(q, kvals, vvals, bt, [n], [0], [T], [L], oq4.pool_sizes(pool, D))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, [n], [0], [T], [L]),
                                        d.Workspace(T, hq, D, L)))
    worst = (np.abs(got - want) / bound).max()
    assert worst <= 1, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("D,hq,T,L", FORMS)
def test_a_key_without_values_that_carries_the_weight(cuda_device, D, hq, T, L):
    """A first key whose V vector is zero (its scale is 0) takes all but 2^-50 of
    the weight: the output is that small, and as exact as ever."""
    d = _dsb()
    rng = np.random.default_rng(L)
    n = -(-L // P)
    k, v = rng.standard_normal((2, n * P, D)) * 0.02, rng.standard_normal((n * P, D))
    k = k[0]
    k[:, 0] = 0.0
    k[0, 0], v[0] = 20.0, 0.0
    pool = np.stack([oq4.pack_block(*oq4.quantise(k[a:a + P]), *oq4.quantise(v[a:a + P])) for a in range(0, n * P, P)])[:, None]
    q = (rng.standard_normal((T, hq, D)) * 0.1).astype(np.float32)
    q[..., 0] = 50 * np.log(2) * np.sqrt(D) / 20
    kvals, vvals = oq4.pool_values(pool, D)
    bt = [list(range(n))]
    want, bound = oq4.attention(q, kvals, vvals, bt, [n], [0], [T], [L], oq4.pool_sizes(pool, D))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, [n], [0], [T], [L]),
                                        d.Workspace(T, hq, D, L)))
    assert 0 < np.abs(want).max() < 2.0 ** -40
    worst = (np.abs(got - want) / bound).max()
    assert worst <= 1, f"{worst:.2f} of the bound"


@pytest.mark.parametrize("D,hq,T,L", FORMS)
@pytest.mark.parametrize("size", [1e36, 1e37, 3e38])
def test_query_rows_up_to_the_largest_float(cuda_device, D, hq, T, L, size):
    """Scores that float32 holds: all keys alike (2^-20 in each dimension), the
    output is the mean of the values that a row sees.  A weight is 1 up to the
    exponential's 2^-22, each of up to L sums and the two-part products within
    2^-22 of the terms' magnitudes: 2^-20 of the mean magnitude with room."""
    d = _dsb()
    rng = np.random.default_rng(L)
    n = -(-L // P)
    v = rng.standard_normal((n * P, D))
    k = np.full((P, D), 2.0 ** -20)
    pool = np.stack([oq4.pack_block(*oq4.quantise(k), *oq4.quantise(v[a:a + P])) for a in range(0, n * P, P)])[:, None]
    q = np.zeros((T, hq, D), np.float32)
    q[..., 3] = size
    q[..., 5] = -size / 4
    _, vvals = oq4.pool_values(pool, D)
    _, vsize = oq4.pool_sizes(pool, D)
    vvals, vsize = vvals.reshape(-1, D), vsize.reshape(-1, D)
    bt = [list(range(n))]
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, [n], [0], [T], [L]),
                                        d.Workspace(T, hq, D, L)))
    for j in range(T):
        seen = L - T + j + 1
        assert (np.abs(got[j] - vvals[:seen].mean(0)) <= 2.0 ** -20 * vsize[:seen].mean(0)).all()
    d.device_error()


PI = 314159265358979323846264338327950288419716939937510582097494459230781640628620899


def _turned(pos, f):
    """float32 nearest to cos(pos f) and sin(pos f), f the float64 given: the angle
    modulo a turn in integers (2^-160), its cosine in float64."""
    one = 1 << 160
    turn = 2 * PI * one // 10 ** 80
    m, e = f.as_integer_ratio()
    r = int(pos) * m * one // e % turn / one
    return np.float32(np.cos(r)), np.float32(np.sin(r))


@pytest.mark.parametrize("pos0", [0, 100000, 1 << 20, (1 << 24) - 300])
def test_cosines_and_sines_are_the_nearest(cuda_device, pos0):
    """Pairs (1, 0) turn to the factors themselves.  A turn's fraction is within
    2^-65 for each position, 2^-38 radians at 2^24, and the sums within 2^-44: of
    values spread over the circle less than one in a thousand lies as near to a
    border between two float32 (some 13 octaves below 1, each with 2^-13.3 of its
    share of about a third)."""
    d = _dsb()
    n, D = 300, 128
    f = orot.frequencies(D, 10000.0)
    x = np.zeros((n, 1, D), np.float32)
    x[..., :D // 2] = 1.0
    t = to_dev(x)
    d.rope_rotary(t, None, np.arange(pos0, pos0 + n), d.Rotary(10000.0), d.Workspace(n, 1, D, P))
    got = to_host(t)[:, 0]
    want = np.array([np.array([_turned(pos0 + i, v) for v in f.tolist()]).T.reshape(-1) for i in range(n)], np.float32)
    assert (np.abs(got.astype(np.float64) - want) <= np.spacing(np.abs(want)) + 2.0 ** -38).all()
    off = int((got != want).sum())
    assert off * 1000 <= want.size, f"{off} of {want.size}"


@pytest.mark.parametrize("rd,inter,scale,pos0", [(128, False, "none", 0), (64, True, "bands", 131000), (48, False, "ntk", 77),
                                                 (128, True, "yarn", 8000), (34, False, "linear", (1 << 24) - 400)])
def test_rotated_values_keep_their_roundings(cuda_device, rd, inter, scale, pos0):
    """x c + p s with c and s the nearest float32 (2^-24 of the gain's octave) and
    three more roundings of at most 2^-24: 2^-24 for the factors, one for the two
    products together and one for the sum, of (|x| + |p|) gain; and 4e-9 rad, what
    float64 leaves of the oracle's own angle at 2^24."""
    d = _dsb()
    n, D = 400, 128
    rng = np.random.default_rng(rd)
    x = rng.standard_normal((n, 3, D)).astype(np.float32)
    pos = pos0 + np.arange(n)
    rot, f, gain = _rot(scale, rd, inter)
    t = to_dev(x)
    d.rope_rotary(t, None, pos, rot, d.Workspace(n, 3, D, P))
    want = orot.rotate(x, pos, f, inter, gain)
    tol = (3 * 2.0 ** -24 + 4e-9) * gain
    assert (np.abs(to_host(t) - want) <= tol * _partner(x.astype(np.float64), rd, inter)).all()


def test_results_on_the_default_stream_by_its_handle(cuda_device):
    """Handle 0 given as the stream: the results come from the default stream's
    memory, which a side stream still at work on freed memory cannot hold."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(3)
    pool = to_dev(_pool(rng, 3, 2, 64))
    q = to_dev(rng.standard_normal((1, 4, 64)).astype(np.float32))
    kv, b, ws = d.kv_q4_pages(pool, 64), d.PagedBatch([[2, 0, 1]], [3], [0], [1], [333]), d.Workspace(1, 4, 64, 384)
    assert torch.cuda.default_stream().cuda_stream == 0
    want, (wk, wv) = d.attention_decode_q4(q, kv, b, ws), d.kv_gather_q4(kv, b, [5], [300], d.DSB_F16, ws)
    torch.cuda.synchronize()
    for _ in range(40):                     # every stream of torch's pool has freed memory that it is yet to write
        with torch.cuda.stream(torch.cuda.Stream()):
            busy = [torch.full_like(t, 7.0) for t in (want, wk, wv)]
            torch.cuda._sleep(10_000_000)
            for t in busy:
                t.fill_(9.0)
            del busy, t
    out = d.attention_decode_q4(q, kv, b, ws, stream=0)
    k, v = d.kv_gather_q4(kv, b, [5], [300], d.DSB_F16, ws, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(k, wk) and torch.equal(v, wv)


@pytest.mark.parametrize("n", [70, 1024])
@pytest.mark.parametrize("store", ["q4", "f16", "bf16"])
def test_appends_of_many_sessions(cuda_device, n, store):
    """Metadata of some hundred words in the launch (70 sessions) and staged (1024):
    the same bits as the sessions a few at a time, whose words are few."""
    import torch
    d = _dsb()
    D, hq, hkv = 64, 3, 2
    rng = np.random.default_rng(n)
    lens = rng.integers(1, 400, n)
    new = np.minimum(np.where(rng.random(n) < 0.05, 0, rng.integers(1, 6, n)), lens)
    window = np.where(rng.random(n) < 0.3, 100, 0)
    bt, blocks, n_pages = _geometry(lens, new, window, rng)
    rot = d.Rotary(rotary_dim=48)
    w = [to_dev((rng.standard_normal(D) * 0.1 + 1).astype(np.float32)) for _ in range(2)]
    qkv = to_dev(rng.standard_normal((int(new.sum()), (hq + 2 * hkv) * D)).astype(np.float32))
    ws = d.Workspace(len(qkv), hq, D, 512)

    def run(cuts):
        if store == "q4":
            pools = [torch.full((n_pages, hkv, P * (D + 8)), 7, dtype=torch.uint8, device="cuda")]
            kv, call = d.kv_q4_pages(pools[0], D), d.kv_append_q4
        else:
            pools = [torch.full((n_pages, hkv, P, D), 7, dtype=torch.int16, device="cuda") for _ in range(2)]
            kv, call = d.kv_pages(*pools, d.DSB_F16 if store == "f16" else d.DSB_BF16), d.kv_append_paged
        rows, at = qkv.clone(), 0
        for a, b in cuts:
            m = int(new[a:b].sum())
            if m:
                call(rows[at:at + m], hq, kv, d.PagedBatch(bt[a:b], blocks[a:b], window[a:b], new[a:b], lens[a:b]), rot, ws,
                     q_norm=w[0], k_norm=w[1], eps=1e-6)
            at += m
        return [rows, *pools]

    together, apart = run([(0, n)]), run([(a, min(a + 8, n)) for a in range(0, n, 8)])
    for a, b in zip(together, apart):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,hq,hkv,lens,new,window", [
    (128, 2, 1, [2300], [300], [0]), (128, 6, 2, [2500, 40, 2400], [90, 1, 130], [0, 0, 2200]), (64, 3, 1, [700], [260], [0])])
def test_attention_of_a_prompts_rows(cuda_device, D, hq, hkv, lens, new, window):
    """Hundreds of rows on a kv head, beside a single token's, on caches long enough
    for the tcgen05 kernel and on a short one."""
    d = _dsb()
    rng = np.random.default_rng(sum(lens))
    bt, blocks, n_pages = _geometry(lens, new, window, rng)
    pool = _pool(rng, n_pages, hkv, D)
    q = (rng.standard_normal((sum(new), hq, D)) * 2).astype(np.float32)
    kvals, vvals = oq4.pool_values(pool, D)
    want, bound = oq4.attention(q, kvals, vvals, bt, blocks, window, new, lens, oq4.pool_sizes(pool, D))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, blocks, window, new, lens),
                                        d.Workspace(sum(new), hq, D, max(lens))))
    assert (np.abs(got - want) <= bound).all()
    d.device_error()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D,rd,inter,scale", [(128, 128, False, "yarn"), (64, 64, True, "none")])
def test_a_long_prompt_into_16_bit_pages(cuda_device, dtype, D, rd, inter, scale):
    """3000 rows at once: k as the rotary call turns it and v as it is, rounded once."""
    import torch
    d = _dsb()
    n, past, hq, hkv = 3000, 90, 5, 2
    rng = np.random.default_rng(D)
    x = to_dev(rng.standard_normal((n, hq + 2 * hkv, D)).astype(np.float32))
    rot, ws = _rot(scale, rd, inter)[0], d.Workspace(n, hq, D, 4096)
    turned = x.clone()
    d.rope_rotary(turned[:, :hq], turned[:, hq:hq + hkv], np.arange(past, past + n), rot, ws)
    blocks = -(-(past + n) // P)
    table = rng.permutation(blocks).astype(np.int32)
    kind = torch.float16 if dtype == "f16" else torch.bfloat16
    k, v = (torch.full((blocks, hkv, P, D), 7.0, device="cuda", dtype=kind) for _ in range(2))
    got = x.clone()
    d.kv_append_paged(got.view(n, -1), hq, d.kv_pages(k, v, d.DSB_F16 if dtype == "f16" else d.DSB_BF16),
                      d.PagedBatch(table[None], [blocks], [0], [n], [past + n]), rot, ws)
    assert torch.equal(got[:, :hq], turned[:, :hq]) and torch.equal(got[:, hq:], x[:, hq:])
    order = torch.from_numpy(table).cuda().long()
    for pages, rows in ((k, turned[:, hq:hq + hkv]), (v, x[:, hq + hkv:])):
        flat = pages[order].permute(0, 2, 1, 3).reshape(-1, hkv, D)
        assert torch.equal(flat[past:past + n], rows.to(kind))
        assert (flat[:past] == 7.0).all() and (flat[past + n:] == 7.0).all()


@pytest.mark.parametrize("D,hq,T,L", FORMS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -3e38])
def test_a_bad_query_row_is_its_own(cuda_device, D, hq, T, L, bad):
    """A NaN, an infinity or a huge value in one row changes no bit of the others."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(L)
    pool, bt = _hidden_case(D, T, L, rng, 1.0)
    q = to_dev(rng.standard_normal((T, hq, D)).astype(np.float32))
    kv, b, ws = d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, [len(bt[0])], [0], [T], [L]), d.Workspace(T, hq, D, L)
    want = d.attention_decode_q4(q, kv, b, ws)
    for j, h in ((0, 0), (T - 1, hq - 1)):
        x = q.clone()
        x[j, h, 17] = bad
        got = d.attention_decode_q4(x, kv, b, ws)
        keep = torch.ones((T, hq), dtype=torch.bool, device="cuda")
        keep[j, h] = False
        assert torch.equal(got[keep], want[keep])
        if not np.isfinite(bad):
            assert torch.isnan(got[j, h]).all()


@pytest.mark.parametrize("D,hq,T,L", FORMS)
@pytest.mark.parametrize("size", [3e38, -1e36, -3e38])
def test_windows_whose_first_page_only_some_rows_see(cuda_device, D, hq, T, L, size):
    """The first row's window starts at the last key of a page, the others' on the
    next; scores of any size that float32 holds.  Bound as above."""
    d = _dsb()
    rng = np.random.default_rng(L)
    n, w = -(-L // P) + 1, L - T + 1 - 127
    v = rng.standard_normal((n * P, D))
    k = np.full((P, D), 2.0 ** -20)
    pool = np.stack([oq4.pack_block(*oq4.quantise(k), *oq4.quantise(v[a:a + P])) for a in range(0, n * P, P)])[:, None]
    q = np.zeros((T, hq, D), np.float32)
    q[..., 3] = size
    q[..., 5] = -size / 4
    _, vvals = oq4.pool_values(pool, D)
    _, vsize = oq4.pool_sizes(pool, D)
    vvals, vsize = vvals.reshape(-1, D), vsize.reshape(-1, D)
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D),
                                        d.PagedBatch([list(range(n))], [n], [w], [T], [L]), d.Workspace(T, hq, D, L)))
    for j in range(T):
        seen = slice(127 + j, L - T + j + 1)
        assert (np.abs(got[j] - vvals[seen].mean(0)) <= 2.0 ** -20 * vsize[seen].mean(0)).all()
    d.device_error()
