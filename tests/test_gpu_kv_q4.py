"""GPU parity of the rotary layouts, the paged appends, the attention over the
4-bit cache and its read-back, against the float64 oracle, through the C ABI.

Tolerances.  A rotated value x c + p s is off by the errors of c and s times
|x| + |p| and by three float32 roundings.  c and s: the angle modulo an eighth
of a turn rounded to float32 (2^-24 pi/4), the frequency's 2^-53 turns times a
position below 2^24 (1.2e-8 rad), a sincospif of at most one unit in the last
place (2^-23) and, with a gain, one rounding: below 2^-22 in all; so the value
within (|x| + |p|) gain (2^-22 + 3 * 2^-24) < 4.2e-7 (|x| + |p|) gain.  A head
norm before it: sum of squares of D float32 terms and four roundings, below
2e-6 of the value at D = 128.  A stored row is within half a step of what it
was given, plus the roundings of d and z to fp16 at the ends.  The attention's
bound is the oracle's (every rounding of a float32 evaluation), over the
magnitudes of the two terms z and d (code - 8) that make a value: the kernel sums
them apart, and where they cancel each keeps the rounding of its own size."""
import ctypes

import numpy as np
import pytest

from oracle import kv as okv
from oracle import kv_q4 as oq4
from oracle import paged as opg
from oracle import rotary as orot
from oracle.rope import Yarn
from tests.gpu_util import to_dev, to_host

pytestmark = pytest.mark.gpu

P = 128
TURN = 4.2e-7
SCALES = {"none": {}, "linear": dict(scaling="linear", factor=8.0), "ntk": dict(scaling="ntk", factor=4.0),
          "bands": dict(scaling="bands", factor=8.0, orig_ctx=8192, low=1.0, high=4.0), "yarn": dict(yarn=Yarn(4.0, 4096))}


def _dsb():
    from session_decode_step_dsb_gb300 import dsb
    return dsb


def _rot(scale, rd, inter):
    kw = SCALES[scale]
    d = _dsb()
    return (d.Rotary(10000.0, rotary_dim=rd, interleaved=inter, **kw), orot.frequencies(rd, 10000.0, **kw),
            0.1 * np.log(4.0) + 1 if scale == "yarn" else 1.0)


def _partner(x, rd, inter):
    p = np.zeros_like(x)
    i = np.arange(rd)
    p[..., :rd] = x[..., (i ^ 1) if inter else (i + rd // 2) % rd]
    return np.abs(x) + np.abs(p)


# ------------------------------------------------------------------- rotary
@pytest.mark.parametrize("n,hq,hkv,D,rd,inter,scale,pos0", [
    (1, 1, 0, 64, 64, False, "none", 0), (1, 12, 12, 64, 64, False, "none", 1999), (3, 5, 1, 128, 128, True, "yarn", 8000),
    (17, 8, 2, 128, 48, False, "bands", 131000), (5, 3, 3, 64, 18, False, "ntk", 77), (5, 3, 3, 64, 18, True, "ntk", 77),
    (2, 3, 1, 34, 10, False, "linear", 5), (2, 2, 2, 6, 6, True, "none", 4), (1, 2, 1, 1024, 1024, False, "none", 4096),
    (1000, 4, 1, 64, 32, True, "none", (1 << 24) - 1000), (1, 64, 64, 128, 2, False, "none", 9)])
def test_rope_rotary(cuda_device, n, hq, hkv, D, rd, inter, scale, pos0):
    import torch
    d = _dsb()
    rng = np.random.default_rng(n + rd)
    rows = rng.standard_normal((n, hq + 2 * hkv + 1, D)).astype(np.float32)      # parts of wider rows
    pos = pos0 + (np.arange(n)[::-1] if n % 2 else (np.arange(n) + n // 4) % n)   # backwards, or in two runs
    rot, f, gain = _rot(scale, rd, inter)
    t = to_dev(rows)
    q, k = t[:, :hq], t[:, hq:hq + hkv] if hkv else None
    if (hq * D) % 4:          # k would not start on 16 bytes: apart
        k = to_dev(rows[:, hq:hq + hkv])
    d.rope_rotary(q, k, pos, rot, d.Workspace(n, hq, D, P))
    # the oracle on every 97th row of a long call
    at = np.arange(n) if n < 100 else np.arange(0, n, 97)
    for part, lo, hi in ((q, 0, hq), (k, hq, hq + hkv)):
        if part is None:
            continue
        x = rows[at, lo:hi]
        want = orot.rotate(x, pos[at], f, inter, gain)
        got = to_host(part.contiguous())[at].astype(np.float64)
        assert (np.abs(got - want) <= TURN * gain * _partner(x.astype(np.float64), rd, inter)).all()
        assert np.array_equal(got[..., rd:], x[..., rd:])
    rest = to_host(t)[:, hq + hkv:] if (hq * D) % 4 == 0 else to_host(t)[:, hq:]
    assert np.array_equal(rest, rows[:, hq + hkv:] if (hq * D) % 4 == 0 else rows[:, hq:])
    one = to_dev(rows[-1:])
    d.rope_rotary(one[:, :hq], None, pos[-1:], rot, d.Workspace(1, hq, D, P))
    assert torch.equal(one[0, :hq], t[-1, :hq])


# ------------------------------------------------------------------- append
def _geometry(lens, new, window, rng, spare=2):
    """Shuffled block tables (a ring one page wider than it has to be)."""
    blocks = [max(1, -(-(w + n - 1) // P) + 1 if w else -(-L // P)) for L, n, w in zip(lens, new, window)]
    n_pages = sum(blocks) + spare
    perm, at = rng.permutation(n_pages), 0
    bt = np.zeros((len(lens), max(blocks)), np.int32)
    for s, b in enumerate(blocks):
        bt[s, :b] = perm[at:at + b]
        at += b
    return bt, np.array(blocks), n_pages


APPENDS = [  # D, hq, hkv, lens, new, window, rd, inter, scale, norm
    (64, 2, 1, [1], [1], [0], 64, False, "none", False),
    (128, 5, 1, [130, 7], [3, 7], [0, 0], 128, False, "yarn", True),
    (64, 12, 3, [128, 0, 300, 129], [128, 0, 5, 1], [0, 0, 200, 0], 18, False, "ntk", True),
    (128, 8, 2, [1000, 256, 5], [1, 256, 0], [100, 0, 0], 64, True, "bands", False),
    (64, 0, 2, [77], [70], [0], 2, True, "linear", False)]


@pytest.mark.parametrize("case", APPENDS)
@pytest.mark.parametrize("store", ["q4", "f16", "bf16"])
def test_append(cuda_device, case, store):
    import torch
    D, hq, hkv, lens, new, window, rd, inter, scale, norm = case
    d = _dsb()
    rng = np.random.default_rng(len(lens) * 1000 + D + rd)
    bt, blocks, n_pages = _geometry(lens, new, window, rng)
    n_tok, H = sum(new), hq + 2 * hkv
    qkv = rng.standard_normal((n_tok, H * D + 8)).astype(np.float32) * np.exp(rng.standard_normal((n_tok, 1))).astype(np.float32)
    qkv[0, hq * D:(hq + 1) * D] = 3.25                       # a vector without spread
    qn, kn = (rng.standard_normal((2, D)) * 0.1 + 1).astype(np.float32)
    rot, f, gain = _rot(scale, rd, inter)
    batch = d.PagedBatch(bt, blocks, window, new, lens)
    t = to_dev(qkv)
    ws = d.Workspace(max(n_tok, 1), max(hq, 1), D, max(lens))
    kw = dict(q_norm=to_dev(qn), k_norm=to_dev(kn), eps=1e-6) if norm else {}
    if store == "q4":
        pool = rng.integers(0, 256, (n_pages, hkv, P * (D + 8))).astype(np.uint8)
        pools = [to_dev(pool)]
        d.kv_append_q4(t[:, :H * D], hq, d.kv_q4_pages(pools[0], D), batch, rot, ws, **kw)
    else:
        pool = rng.integers(0, 1 << 16, (2, n_pages, hkv, P, D)).astype(np.uint16)
        pools = [to_dev(x.view(np.int16)) for x in pool]
        d.kv_append_paged(t[:, :H * D], hq, d.kv_pages(*pools, 0 if store == "f16" else 1), batch, rot, ws, **kw)
    torch.cuda.synchronize()
    where = oq4.positions(new, lens)
    pos = np.array([p for _, p in where])
    x = qkv[:, :H * D].reshape(n_tok, H, D).astype(np.float64)
    if norm:
        for lo, hi, w in ((0, hq, qn), (hq, hq + hkv, kn)):
            x[:, lo:hi] = x[:, lo:hi] / np.sqrt((x[:, lo:hi] ** 2).mean(-1, keepdims=True) + 1e-6) * w
    slack = (TURN * gain + (2e-6 * gain if norm else 0)) * _partner(x, rd, inter)
    y = orot.rotate(x[:, :hq + hkv], pos, f, inter, gain)
    got = to_host(t)
    assert (np.abs(got[:, :hq * D].reshape(n_tok, hq, D) - y[:, :hq]) <= slack[:, :hq]).all()
    assert np.array_equal(got[:, hq * D:], qkv[:, hq * D:])   # k, v and what lies behind the row
    k, v = y[:, hq:], qkv[:, (hq + hkv) * D:H * D].reshape(n_tok, hkv, D)
    ks = slack[:, hq:hq + hkv]
    rows = {opg.locate(p, bt[s], int(blocks[s]), int(window[s])): i for i, (s, p) in enumerate(where)}
    if store != "q4":
        for which, p in enumerate(pools):
            h = to_host(p).view(np.uint16)
            for page in range(n_pages):
                for r in range(P):
                    if (page, r) not in rows:
                        assert np.array_equal(h[page, :, r], pool[which, page, :, r])
            for (page, r), i in rows.items():
                if which:
                    assert np.array_equal(h[page, :, r], okv.convert(v[i], store))
                else:
                    val = okv.bits_to_f64(h[page, :, r], store)
                    half = 2.0 ** (-11 if store == "f16" else -8)
                    assert (np.abs(val - k[i]) <= ks[i] + half * (np.abs(k[i]) + ks[i]) + 2.0 ** -25).all()
        return
    h = to_host(pools[0])
    flips = 0
    for page in range(n_pages):
        for g in range(hkv):
            now, old = oq4.unpack_block(h[page, g], D), oq4.unpack_block(pool[page, g], D)
            for r in range(P):
                i = rows.get((page, r))
                if i is None:      # rows that are not the call's
                    for a, b in zip(now, old):
                        assert np.array_equal(a[r].view(np.uint8), b[r].view(np.uint8))
                    continue
                vc, vdz = oq4.quantise(v[i, g])
                assert np.array_equal(now[2][r], vc) and np.array_equal(now[3][r].view(np.uint16), vdz.view(np.uint16))
                kd, kz = now[1][r].astype(np.float64)
                ends = 8 * kd * 2.0 ** -10 + abs(kz) * 2.0 ** -11 + 1e-7
                assert (np.abs(oq4.values(now[0][r], now[1][r]) - k[i, g]) <= kd / 2 + ends + 2 * ks[i, g].max()).all()
                kc, kdz = oq4.quantise(k[i, g].astype(np.float32))
                # The numbers are fp16 roundings (2^-10 of the result between two of them, 2^-24
                # below fp16's normal range) of values that differ: (max - min) / 15 by 2/15 of
                # the rotation's error, and min + 8 d, where the two may cancel, by that error,
                # 8 times d's difference and the float32 rounding of the sum.
                ours, err = kdz.astype(np.float64), ks[i, g].max()
                far = np.abs(now[1][r].astype(np.float64) - ours)
                assert far[0] <= ours[0] * 2.0 ** -10 + 2.0 ** -24 + err * 2 / 15
                assert far[1] <= abs(ours[1]) * 2.0 ** -10 + 2.0 ** -24 + err + 8 * far[0] + 2.0 ** -23 * 8 * ours[0]
                if np.array_equal(now[1][r], kdz):
                    assert np.abs(now[0][r].astype(int) - kc.astype(int)).max() <= 1
                    flips += int((now[0][r] != kc).sum())
    # a code flips where its value lies within the rotation's error of a border: 2 slack / d of them
    assert flips <= 3 + 1e-3 * n_tok * hkv * D


@pytest.mark.parametrize("D,rd,inter,scale,n", [(128, 128, False, "yarn", 300), (64, 48, True, "linear", 5),
                                               (128, 34, True, "none", 70), (64, 18, False, "ntk", 40)])
def test_the_append_turns_as_the_rotary_call_does(cuda_device, D, rd, inter, scale, n):
    """The same steps, each rounded once: the same bits on both paths."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(D + rd)
    hq, hkv = 6, 2
    x = to_dev(rng.standard_normal((n, hq + 2 * hkv, D)).astype(np.float32))
    rot = _rot(scale, rd, inter)[0]
    turned = x.clone()
    ws = d.Workspace(n, hq, D, 4096)
    d.rope_rotary(turned[:, :hq], turned[:, hq:hq + hkv], np.arange(700, 700 + n), rot, ws)
    blocks = -(-(700 + n) // P)
    batch = d.PagedBatch(np.arange(blocks, dtype=np.int32)[None], [blocks], [0], [n], [700 + n])
    k = torch.zeros((blocks, hkv, P, D), device="cuda", dtype=torch.float16)
    got = x.clone()
    d.kv_append_paged(got.view(n, -1), hq, d.kv_pages(k, torch.zeros_like(k), d.DSB_F16), batch, rot, ws)
    assert torch.equal(got[:, :hq], turned[:, :hq]) and torch.equal(got[:, hq:], x[:, hq:])
    rows = k.permute(0, 2, 1, 3).reshape(-1, hkv, D)[700:700 + n]
    assert torch.equal(rows, turned[:, hq:hq + hkv].half())


def test_append_stores_bad_vectors_as_nan(cuda_device):
    d = _dsb()
    x = np.random.default_rng(0).standard_normal((4, 3 * 64)).astype(np.float32)
    x[0, 64 + 5], x[1, 128 + 63], x[2, 64] = np.nan, np.inf, -np.inf
    pool = to_dev(np.zeros((1, 1, P * 72), np.uint8))
    b = d.PagedBatch([[0]], [1], [0], [4], [4])
    kv, ws = d.kv_q4_pages(pool, 64), d.Workspace(4, 1, 64, P)
    d.kv_append_q4(to_dev(x), 1, kv, b, d.Rotary(), ws)
    k, v = (to_host(a.float()) for a in d.kv_gather_q4(kv, b, [0], [4], 0, ws))
    assert np.isnan(k[[0, 2]]).all() and np.isfinite(k[[1, 3]]).all()
    assert np.isnan(v[1]).all() and np.isfinite(v[[0, 2, 3]]).all()


# ---------------------------------------------------------- attention, gather
def _pool(rng, n_pages, hkv, D, vsize=1.0, pairs=None):
    """Bytes of a pool of random rows; codes and numbers of every block."""
    pool = np.empty((n_pages, hkv, P * (D + 8)), np.uint8)
    for p in range(n_pages):
        for h in range(hkv):
            k = rng.standard_normal((P, D)) * np.exp(0.5 * rng.standard_normal((P, 1)))
            v = rng.standard_normal((P, D)) * np.exp(0.5 * rng.standard_normal((P, 1))) * vsize + 0.3 * vsize
            pool[p, h] = oq4.pack_block(*oq4.quantise(k), *oq4.quantise(v))
    return pool


def _spoil(pool, bt, blocks, window, lens, D):
    """NaN numbers (and full codes) in every row that no key of a sequence holds."""
    held = {opg.locate(p, bt[s], int(blocks[s]), int(window[s]))
            for s, L in enumerate(lens) for p in range(max(0, L - int(blocks[s]) * P) if window[s] else 0, L)}
    out, c = pool.copy(), P * D // 2
    for p in range(pool.shape[0]):
        for r in range(P):
            if (p, r) not in held:
                out[p, :, r * D // 2:(r + 1) * D // 2] = 255
                out[p, :, c + 4 * r:c + 4 * r + 4] = 255
                out[p, :, 2 * c + 4 * P + 4 * r:2 * c + 4 * P + 4 * r + 4] = 255
    return out


ATTN = [  # D, hq, hkv, lens, new, window
    (64, 1, 1, [1], [1], [0]),
    (64, 8, 2, [200], [1], [0]),
    (128, 5, 1, [128, 129, 255, 0], [1, 1, 1, 0], [0] * 4),
    (128, 40, 8, [700], [1], [0]),
    (64, 12, 12, [900, 33, 5], [4, 0, 5], [200, 0, 0]),
    (128, 3, 3, [1, 2, 31, 32, 33, 95, 97], [1, 2, 1, 1, 3, 1, 2], [0, 1, 7, 0, 32, 0, 96]),
    (64, 10, 1, [2600], [7], [0]),                       # 70 query rows
    (128, 2, 1, [5000, 260], [1, 64], [0, 130]),
    (64, 16, 2, [300], [130], [0]),                       # a prompt: 1040 rows
    (128, 16, 1, [1, 127, 128, 700], [1, 1, 1, 1], [0, 0, 60, 300]),    # 16 rows
    (128, 10, 2, [400, 8, 1500, 513], [8, 8, 1, 2], [0, 0, 0, 333]),     # 40, 5 and 10 rows in one call
    (64, 9, 1, [1000, 260], [1, 3], [129, 0]),            # 9 and 27 rows
    (128, 20, 2, [2300, 40, 2177, 2500, 0], [2, 2, 3, 1, 0], [0, 0, 2100, 0, 0]),   # 20 and 30 rows on long caches, 20 on a short
    (128, 40, 1, [4100, 2500], [2, 1], [0, 0]),           # 80 and 40 rows
    (128, 2, 2, [3000, 2049], [49, 17], [2200, 0]),       # 49 rows in a window; the shortest of the kind, 17 rows
    (128, 4, 1, [2300, 700, 900, 2500], [5, 1, 2, 1], [0, 0, 300, 0])]    # 20, 4, 8 and 4 rows in one call


@pytest.mark.parametrize("case", ATTN)
def test_attention_q4(cuda_device, case):
    D, hq, hkv, lens, new, window = case
    d = _dsb()
    rng = np.random.default_rng(D + hq + sum(lens))
    bt, blocks, n_pages = _geometry(lens, new, window, rng, spare=1)
    pool = _pool(rng, n_pages, hkv, D)
    q = (rng.standard_normal((sum(new), hq, D)) * 2).astype(np.float32)
    kvals, vvals = oq4.pool_values(pool, D)
    want, bound = oq4.attention(q, kvals, vvals, bt, blocks, window, new, lens,
                                oq4.pool_sizes(pool, D))
    batch = d.PagedBatch(bt, blocks, window, new, lens)
    ws = d.Workspace(sum(new), hq, D, max(lens))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), batch, ws))
    assert np.isfinite(got).all()
    worst = (np.abs(got - want) / bound).max()
    assert worst <= 1, f"{worst:.2f} of the bound"
    # what rows of a page past a sequence's keys hold changes no bit
    bad = to_dev(_spoil(pool, bt, blocks, window, lens, D))
    again = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(bad, D), batch, ws))
    assert np.array_equal(again.view(np.uint32), got.view(np.uint32))
    # every sequence alone, from query rows that lie apart, bitwise the same
    row = 0
    for s, n in enumerate(new):
        if n == 0:
            continue
        one = d.PagedBatch(bt[s:s + 1], blocks[s:s + 1], window[s:s + 1], [n], [lens[s]])
        wide = to_dev(np.concatenate([q[row:row + n], np.full((n, 1, D), np.nan, np.float32)], 1))
        alone = to_host(d.attention_decode_q4(wide[:, :hq], d.kv_q4_pages(bad, D), one, d.Workspace(n, hq, D, lens[s])))
        assert np.array_equal(alone.view(np.uint32), got[row:row + n].view(np.uint32))
        row += n
    d.device_error()


@pytest.mark.parametrize("vsize,qsize", [(1e-4, 1.0), (3e3, 1.0), (1.0, 1e-6), (1.0, 50.0), (1e-7, 0.0)])
def test_attention_q4_at_odd_sizes_of_values(cuda_device, vsize, qsize):
    """Small and large scales: the fp16 split keeps its bits; q = 0 is the mean."""
    d = _dsb()
    rng = np.random.default_rng(5)
    pool = _pool(rng, 3, 1, 64, vsize)
    q = (rng.standard_normal((1, 4, 64)) * qsize).astype(np.float32)
    kvals, vvals = oq4.pool_values(pool, 64)
    bt = [[2, 0, 1]]
    want, bound = oq4.attention(q, kvals, vvals, bt, [3], [0], [1], [333], oq4.pool_sizes(pool, 64))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), 64), d.PagedBatch(bt, [3], [0], [1], [333]),
                                        d.Workspace(1, 4, 64, 384)))
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("hq,T,L", [(4, 1, 3000), (10, 4, 700), (2, 8, 200), (10, 4, 2200)])
def test_attention_q4_as_exact_as_float32(cuda_device, hq, T, L):
    """Vectors with a few wide dimensions, as a trained model's.  Every operand and
    sum of the kernel keeps 22 bits or more, so its error may be twice that of a
    float32 evaluation with numpy's blocked sums, and 2^-22 for the split."""
    d = _dsb()
    rng = np.random.default_rng(hq + T)
    D, n_pages = 128, -(-L // P)
    wide = np.where(rng.random((2, D)) < 0.05, 7.0, 1.0)
    pool = np.stack([oq4.pack_block(*oq4.quantise(rng.standard_normal((P, D)) * wide[0]),
                                    *oq4.quantise(rng.standard_normal((P, D)) * wide[1])) for _ in range(n_pages)])[:, None]
    q = (rng.standard_normal((T, hq, D)) * wide[0]).astype(np.float32)
    kvals, vvals = oq4.pool_values(pool, D)
    bt = np.arange(n_pages)[None]
    want, _ = oq4.attention(q, kvals, vvals, bt, [n_pages], [0], [T], [L], oq4.pool_sizes(pool, D))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D),
                                        d.PagedBatch(bt, [n_pages], [0], [T], [L]), d.Workspace(T, hq, D, L)))
    k32, v32 = (np.asarray(x).reshape(-1, D).astype(np.float32)[:L] for x in (kvals, vvals))
    plain = np.empty_like(q)
    for j in range(T):
        seen = L - T + j + 1
        s = (q[j] @ k32[:seen].T) * np.float32(D ** -0.5)
        w = np.exp(s - s.max(-1, keepdims=True))
        plain[j] = (w @ v32[:seen]) / w.sum(-1, keepdims=True)
    size = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= 2 * np.linalg.norm(plain - want) + 2.0 ** -22 * size


def test_attention_q4_scales_far_apart(cuda_device):
    """The keys that carry the weight have values 2^-13 of the others': the
    reference is kept over weight times scale, so they lose no bits."""
    d = _dsb()
    rng = np.random.default_rng(6)
    k = rng.standard_normal((P, 64)) * 0.01
    v = rng.standard_normal((P, 64)) * 1000
    k[40:, 0], v[40:] = 60.0, v[40:] * 2.0 ** -13
    k[:40, 0] = -60.0
    pool = oq4.pack_block(*oq4.quantise(k), *oq4.quantise(v))[None, None]
    q = np.zeros((1, 1, 64), np.float32)
    q[..., 0] = 2.0
    kvals, vvals = oq4.pool_values(pool, 64)
    want, bound = oq4.attention(q, kvals, vvals, [[0]], [1], [0], [1], [100], oq4.pool_sizes(pool, 64))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), 64), d.PagedBatch([[0]], [1], [0], [1], [100]),
                                        d.Workspace(1, 1, 64, P)))
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("pages", [9, 19])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,T", [(2, 2), (12, 1), (6, 5)])
def test_attention_q4_references_move(cuda_device, D, hq, T, pages):
    """Keys that grow from page to page: each page's largest weight is far above
    the last one's, for all rows or for some (rows of the other sign shrink)."""
    d = _dsb()
    rng = np.random.default_rng(13)
    pool = np.empty((pages, 1, P * (D + 8)), np.uint8)
    for p in range(pages):
        k = rng.standard_normal((P, D)) * 0.1
        k[:, 0] += 4.0 * p
        pool[p, 0] = oq4.pack_block(*oq4.quantise(k), *oq4.quantise(rng.standard_normal((P, D)) * 2.0 ** (p % 3)))
    q = rng.standard_normal((T, hq, D)).astype(np.float32) * 0.2
    q[..., 0] = np.sqrt(D) * np.where(rng.random((T, hq)) < 0.5, 3.5, -1.0)
    L = pages * P - 52
    bt = [list(range(pages))]
    kvals, vvals = oq4.pool_values(pool, D)
    want, bound = oq4.attention(q, kvals, vvals, bt, [pages], [0], [T], [L], oq4.pool_sizes(pool, D))
    got = to_host(d.attention_decode_q4(to_dev(q), d.kv_q4_pages(to_dev(pool), D), d.PagedBatch(bt, [pages], [0], [T], [L]),
                                        d.Workspace(T, hq, D, pages * P)))
    assert (np.abs(got - want) <= bound).all()


def test_a_nan_key_reaches_the_rows_that_see_it(cuda_device):
    d = _dsb()
    rng = np.random.default_rng(7)
    pool = _pool(rng, 2, 1, 64)
    pool[0, 0, 64 * 64 + 4 * 70:64 * 64 + 4 * 70 + 4] = 255            # K numbers of key 70
    q = to_dev(rng.standard_normal((3, 1, 64)).astype(np.float32))
    b = d.PagedBatch([[0, 1]], [2], [60], [3], [132])                  # rows at 129, 130, 131 see keys 70, 71, 72 on
    got = to_host(d.attention_decode_q4(q, d.kv_q4_pages(to_dev(pool), 64), b, d.Workspace(3, 1, 64, 256)))
    assert np.isnan(got[0]).all() and np.isfinite(got[1:]).all()


@pytest.mark.parametrize("D,hkv,dtype", [(64, 2, "f16"), (128, 1, "bf16"), (128, 3, "f16"), (64, 1, "bf16")])
def test_gather_q4(cuda_device, D, hkv, dtype):
    import torch
    d = _dsb()
    rng = np.random.default_rng(D + hkv)
    lens, window = [300, 1, 0, 1000, 128], [0, 0, 0, 150, 0]
    first, count = [5, 0, 0, 1000 - 3 * P, 127], [290, 1, 0, 3 * P, 1]
    bt, blocks, n_pages = _geometry(lens, [0] * 5, window, rng)
    assert blocks[3] == 3                    # its oldest and newest keys share a page of the ring
    pool = _pool(rng, n_pages, hkv, D)
    b = d.PagedBatch(bt, blocks, window, [0] * 5, lens)
    ws = d.Workspace(1, 1, D, P)
    k, v = d.kv_gather_q4(d.kv_q4_pages(to_dev(pool), D), b, first, count, 0 if dtype == "f16" else 1, ws)
    kvals, vvals = oq4.pool_values(pool, D)
    at = [opg.locate(p, bt[s], int(blocks[s]), int(window[s])) for s in range(5) for p in range(first[s], first[s] + count[s])]
    pages, rows = np.array([a[0] for a in at]), np.array([a[1] for a in at])
    for got, vals in ((k, kvals), (v, vvals)):
        want = okv.convert(vals[pages, :, rows].astype(np.float32), dtype)
        assert got.shape == want.shape and got.dtype == (torch.float16 if dtype == "f16" else torch.bfloat16)
        assert np.array_equal(to_host(got.view(torch.int16)).view(np.uint16), want)


# ------------------------------------------------------- together, and in use
def test_prompt_then_steps_together(cuda_device):
    """Three sessions: prompts appended, then steps of one and three tokens
    (append, attention, the next), against the oracle on the pool's own bytes;
    the attention over the rows read back into a 16-bit cache agrees."""
    import torch
    d = _dsb()
    D, hq, hkv, C = 128, 10, 2, 512
    rng = np.random.default_rng(8)
    lens, window = np.array([200, 1, 390]), np.array([0, 0, 140])
    blocks = np.array([4, 4, 3])
    bt = np.zeros((3, 4), np.int32)
    perm = rng.permutation(12)
    bt[0], bt[1], bt[2, :3] = perm[:4], perm[4:8], perm[8:11]
    pool = torch.zeros((12, hkv, P * (D + 8)), dtype=torch.uint8, device="cuda")
    kv, rot = d.kv_q4_pages(pool, D), d.Rotary(1e4, rotary_dim=96)
    ws = d.Workspace(512, hq, D, C)
    new = np.array([200, 1, 140])
    for step in range(4):
        batch = d.PagedBatch(bt, blocks, window, new, lens)
        n_tok = int(new.sum())
        qkv = torch.from_numpy(rng.standard_normal((n_tok, (hq + 2 * hkv) * D)).astype(np.float32)).cuda()
        d.kv_append_q4(qkv, hq, kv, batch, rot, ws)
        q = qkv[:, :hq * D].unflatten(1, (hq, D))
        out = to_host(d.attention_decode_q4(q, kv, batch, ws))
        pos = [p for _, p in oq4.positions(new, lens)]
        if step:
            host = to_host(pool)
            kvals, vvals = oq4.pool_values(host, D)
            want, bound = oq4.attention(to_host(q.contiguous()), kvals, vvals, bt, blocks, window, new, lens,
                                        oq4.pool_sizes(host, D))
            assert (np.abs(out - want) <= bound).all()
            # sequence 0 and 1 read back into a contiguous bf16 cache
            sub = d.PagedBatch(bt[:2], blocks[:2], window[:2], new[:2], lens[:2])
            k, v = d.kv_gather_q4(kv, sub, [0, 0], lens[:2], 1, ws)
            kc = torch.zeros((2, hkv, C, D), dtype=torch.bfloat16, device="cuda")
            vc = torch.zeros_like(kc)
            a = 0
            for s in range(2):
                kc[s, :, :lens[s]] = k[a:a + lens[s]].transpose(0, 1)
                vc[s, :, :lens[s]] = v[a:a + lens[s]].transpose(0, 1)
                a += lens[s]
            m = int(new[:2].sum())
            wide = to_host(d.attention_decode_multi(q[:m].contiguous(), d.kv_cache(kc, vc, 1), [0, 1], int(new[0]), lens[:2], ws))
            # bf16 of the values: 2^-9 of every score term and value
            assert np.abs(wide - out[:m]).max() < 0.05
        new = np.array([1, 1, 1]) if step % 2 == 0 else np.array([3, 3, 3])
        lens = lens + new
    d.device_error()


def test_captured_and_replayed(cuda_device):
    """A layer's append, attention and read-back in two graphs that share a
    workspace, replayed in turn on new inputs; what is staged is refused."""
    import torch
    d = _dsb()
    D, hq, hkv = 64, 8, 2
    rng = np.random.default_rng(9)
    ws = d.Workspace(300, hq, D, 4096)
    rot = d.Rotary()
    setups = []
    for lens in ([900, 300], [2000, 40]):
        bt, blocks, n_pages = _geometry(lens, [1, 2], [0, 0], rng)
        pool = to_dev(_pool(rng, n_pages, hkv, D))
        batch = d.PagedBatch(bt, blocks, [0, 0], [1, 2], lens)
        qkv = torch.zeros((3, (hq + 2 * hkv) * D), device="cuda")
        kv = d.kv_q4_pages(pool, D)
        out = torch.zeros((3, hq, D), device="cuda")
        k, v = (torch.zeros((6, hkv, D), dtype=torch.float16, device="cuda") for _ in range(2))

        def layer(qkv=qkv, kv=kv, batch=batch, out=out, k=k, v=v, lens=lens):
            d.kv_append_q4(qkv, hq, kv, batch, rot, ws)
            d.attention_decode_q4(qkv[:, :hq * D].unflatten(1, (hq, D)), kv, batch, ws, out=out)
            d.kv_gather_q4(kv, batch, [n - 3 for n in lens], [3, 3], 0, ws, k=k, v=v)
        layer()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer()
        setups.append((g, layer, qkv, out, k, v, pool))
    for turn in range(3):
        for g, layer, qkv, out, k, v, pool in setups:
            x = torch.randn(qkv.shape, device="cuda")
            qkv.copy_(x)
            layer()
            want = [a.clone() for a in (qkv, out, k, v, pool)]
            qkv.copy_(x)
            for a in (out, k, v):
                a.zero_()
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip((qkv, out, k, v, pool), want):
                assert torch.equal(a, b)
    # 5000 positions apart are staged: not in a graph
    q = torch.zeros((5000, 2, D), device="cuda")
    big = d.Workspace(5000, 2, D, P)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q.add_(0.0)
        with pytest.raises(d.DsbError, match="captured"):
            d.rope_rotary(q, None, np.arange(0, 10000, 2), rot, big)
    d.rope_rotary(q, None, np.arange(0, 10000, 2), rot, big)
    torch.cuda.synchronize()


def test_staged_and_cut_metadata_give_the_same_bits(cuda_device):
    """700 sequences with tables of 40 blocks (some 20000 words: several launches,
    staged) against the same sequences a few at a time (in the parameters)."""
    import torch
    d = _dsb()
    D, hq, hkv, n = 64, 2, 1, 700
    rng = np.random.default_rng(10)
    pool = to_dev(_pool(rng, 30, hkv, D))
    kv = d.kv_q4_pages(pool, D)
    bt = rng.integers(0, 30, (n, 40)).astype(np.int32)
    lens = rng.integers(1, 40 * P + 1, n)
    new = rng.integers(0, 2, n)
    q = torch.from_numpy(rng.standard_normal((int(new.sum()), hq, D)).astype(np.float32)).cuda()
    ws = d.Workspace(n, hq, D, 40 * P)
    all_ = d.attention_decode_q4(q, kv, d.PagedBatch(bt, [40] * n, [0] * n, new, lens), ws)
    k, v = d.kv_gather_q4(kv, d.PagedBatch(bt, [40] * n, [0] * n, new, lens), np.zeros(n), np.minimum(lens, 1000), 0, ws)
    row = at = 0
    for s in range(0, n, 10):
        sl = slice(s, s + 10)
        m, c = int(new[sl].sum()), int(np.minimum(lens[sl], 1000).sum())
        part = d.PagedBatch(bt[sl], [40] * 10, [0] * 10, new[sl], lens[sl])
        assert torch.equal(d.attention_decode_q4(q[row:row + m], kv, part, ws), all_[row:row + m])
        pk, pv = d.kv_gather_q4(kv, part, np.zeros(10), np.minimum(lens[sl], 1000), 0, ws)
        assert torch.equal(pk, k[at:at + c]) and torch.equal(pv, v[at:at + c])
        row, at = row + m, at + c
    d.device_error()


def test_pool_offsets_past_32_bits(cuda_device):
    """Pages beyond the first 4 GiB of a pool."""
    import torch
    d = _dsb()
    D, hkv = 128, 8
    n_pages = (1 << 32) // (hkv * P * (D + 8)) + 40
    pool = torch.empty((n_pages, hkv, P * (D + 8)), dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(11)
    small = torch.from_numpy(_pool(rng, 2, hkv, D)).cuda()
    far = np.array([[n_pages - 1, n_pages - 2]])
    pool[n_pages - 1], pool[n_pages - 2] = small[0], small[1]
    kv_far, kv = d.kv_q4_pages(pool, D), d.kv_q4_pages(small, D)
    qkv = torch.from_numpy(rng.standard_normal((2, 24 * D)).astype(np.float32)).cuda()
    res = []
    for pages, table in ((kv_far, far), (kv, [[0, 1]])):
        b = d.PagedBatch(table, [2], [0], [2], [200])
        x, ws = qkv.clone(), d.Workspace(2, 8, D, 256)
        d.kv_append_q4(x, 8, pages, b, d.Rotary(), ws)
        res.append((d.attention_decode_q4(x[:, :8 * D].unflatten(1, (8, D)), pages, b, ws), *d.kv_gather_q4(pages, b, [0], [200], 0, ws)))
    for a, b in zip(*res):
        assert torch.equal(a, b)
    assert torch.equal(pool[n_pages - 2], small[1])


def test_on_another_stream_and_guarded(cuda_device):
    """A side stream's own work only, outputs between guard bands, two
    workspaces on two streams at once."""
    import torch
    from tests.test_gpu_guard import Guarded
    d = _dsb()
    D, hq, hkv = 128, 5, 1
    rng = np.random.default_rng(12)
    lens, new, window = [700, 50], [3, 1], [0, 33]
    bt, blocks, n_pages = _geometry(lens, new, window, rng)
    pool = to_dev(_pool(rng, n_pages, hkv, D))
    b = d.PagedBatch(bt, blocks, window, new, lens)
    q = torch.from_numpy(rng.standard_normal((4, hq, D)).astype(np.float32)).cuda()
    kv = d.kv_q4_pages(pool, D)
    want = d.attention_decode_q4(q, kv, b, d.Workspace(4, hq, D, 1024))
    gk, gv = d.kv_gather_q4(kv, b, [3, 20], [600, 30], 0, d.Workspace(1, 1, D, P))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, spaces, keep = [], [], []
    for s in streams:
        out, k, v = Guarded(4 * hq * D * 4), Guarded(630 * hkv * D * 2), Guarded(630 * hkv * D * 2)
        spaces.append(d.Workspace(4, hq, D, 1024))
        outs.append((out, k, v))
        keep.append([out.view(torch.float32, (4, hq, D)), k.view(torch.float16, (630, hkv, D)),
                     v.view(torch.float16, (630, hkv, D))])
    torch.cuda.synchronize()
    for s, ws, (o, k, v) in zip(streams, spaces, keep):
        with torch.cuda.stream(s):
            for _ in range(20):
                d.attention_decode_q4(q, kv, b, ws, out=o)
                d.kv_gather_q4(kv, b, [3, 20], [600, 30], 0, ws, k=k, v=v)
    for (o, k, v), g in zip(keep, outs):
        for x in g:
            x.check("4-bit KV outputs")
        assert torch.equal(o, want) and torch.equal(k, gk) and torch.equal(v, gv)


def test_a_short_workspace_is_refused(cuda_device):
    import torch
    d = _dsb()
    pool = torch.zeros((32, 1, P * 72), dtype=torch.uint8, device="cuda")
    b = d.PagedBatch([list(range(32))], [32], [0], [1], [4096])
    with pytest.raises(d.DsbError, match="partials"):
        d.attention_decode_q4(torch.zeros((1, 4, 64), device="cuda"), d.kv_q4_pages(pool, 64), b, d.Workspace(1, 4, 64, 128))


def test_a_nan_key_on_a_long_cache_of_many_rows(cuda_device):
    d = _dsb()
    rng = np.random.default_rng(8)
    L, T, hq = 2400, 3, 8
    pool = _pool(rng, 19, 1, 128)
    c = 64 * 128
    key = L - T + 1                                       # the second new token's: the first does not see it
    page, r = divmod(key, P)
    q = to_dev(rng.standard_normal((T, hq, 128)).astype(np.float32))
    b = d.PagedBatch([list(range(19))], [19], [0], [T], [L])
    for at in (c + 4 * r, 2 * c + 4 * P + 4 * r):          # its K numbers, its V numbers
        bad = pool.copy()
        bad[page, 0, at:at + 4] = 255
        got = to_host(d.attention_decode_q4(q, d.kv_q4_pages(to_dev(bad), 128), b, d.Workspace(T, hq, 128, L)))
        assert np.isfinite(got[0]).all() and np.isnan(got[1:]).all()


def test_a_thousand_sequences(cuda_device):
    """As many as a call may have: their metadata is staged, and every CTA looks
    its first one up among them."""
    d = _dsb()
    n, D, hq, hkv = 1024, 64, 2, 1
    rng = np.random.default_rng(21)
    lens = rng.integers(1, 300, n)
    new = np.where(rng.random(n) < 0.1, 0, 1)
    bt = rng.integers(0, 40, (n, 3))                      # pages shared by many: they are only read
    pool = _pool(rng, 40, hkv, D)
    q = rng.standard_normal((int(new.sum()), hq, D)).astype(np.float32)
    kv = d.kv_q4_pages(to_dev(pool), D)
    got = to_host(d.attention_decode_q4(to_dev(q), kv, d.PagedBatch(bt, [3] * n, [0] * n, new, lens),
                                        d.Workspace(n, hq, D, 384)))
    kvals, vvals = oq4.pool_values(pool, D)
    want, bound = oq4.attention(q, kvals, vvals, bt, [3] * n, [0] * n, new, lens, oq4.pool_sizes(pool, D))
    assert (np.abs(got - want) <= bound).all()


@pytest.mark.parametrize("n", [1, 240, 241, 4032, 4033])
def test_positions_in_and_beside_the_launch(cuda_device, n):
    """Metadata at the sizes where its way to the kernel changes."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(n)
    pos = rng.permutation(3 * n)[:n] * 2                  # no two in a row
    x = to_dev(rng.standard_normal((n, 1, 64)).astype(np.float32))
    rot, ws = d.Rotary(interleaved=True), d.Workspace(n, 1, 64, P)
    got = x.clone()
    d.rope_rotary(got, None, pos, rot, ws)
    order = np.argsort(pos)                               # one call for each half
    for part in (order[:n // 2], order[n // 2:]):
        if len(part):
            y = x[torch.from_numpy(part).cuda()].contiguous()
            d.rope_rotary(y, None, pos[part], rot, ws)
            assert torch.equal(y, got[torch.from_numpy(part).cuda()])


def test_a_given_stream_owns_what_the_call_makes(cuda_device):
    import torch
    d = _dsb()
    rng = np.random.default_rng(31)
    pool = to_dev(_pool(rng, 3, 2, 64))
    q = to_dev(rng.standard_normal((1, 4, 64)).astype(np.float32))
    kv, b = d.kv_q4_pages(pool, 64), d.PagedBatch([[2, 0, 1]], [3], [0], [1], [333])
    want = d.attention_decode_q4(q, kv, b, d.Workspace(1, 4, 64, 384))
    wk, wv = d.kv_gather_q4(kv, b, [5], [300], d.DSB_BF16, d.Workspace(1, 4, 64, 384))
    torch.cuda.synchronize()
    side, ws = torch.cuda.Stream(), d.Workspace(1, 4, 64, 384)
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        # memory that the current stream still writes is freed and must not be handed out
        busy = [torch.full_like(t, 7.0) for t in (want, wk, wv)]
        torch.cuda._sleep(20_000_000)
        for t in busy:
            t.fill_(9.0)
        del busy, t
        out = d.attention_decode_q4(q, kv, b, ws, stream=stream)
        k, v = d.kv_gather_q4(kv, b, [5], [300], d.DSB_BF16, ws, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(k, wk) and torch.equal(v, wv)


def test_two_graphs_on_one_workspace(cuda_device):
    """Captured calls carry their metadata; partial sums in the workspace they
    share are each replay's own, one replay after the other."""
    import torch
    d = _dsb()
    rng = np.random.default_rng(41)
    D, hq, hkv = 128, 8, 2
    pool = to_dev(_pool(rng, 40, hkv, D))
    kv = d.kv_q4_pages(pool, D)
    calls = []
    for lens, new in (([2000, 77], [1, 2]), ([2500, 300], [6, 1])):
        bt, blocks, _ = _geometry(lens, new, [0, 0], rng)
        q = to_dev(rng.standard_normal((sum(new), hq, D)).astype(np.float32))
        calls.append((q, d.PagedBatch(bt, blocks, [0, 0], new, lens)))
    want = [d.attention_decode_q4(q, kv, b, d.Workspace(7, hq, D, 2560)).clone() for q, b in calls]
    ws = d.Workspace(7, hq, D, 2560)
    outs = [torch.empty_like(w) for w in want]
    graphs = []
    for (q, b), o in zip(calls, outs):
        d.attention_decode_q4(q, kv, b, ws, out=o)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            d.attention_decode_q4(q, kv, b, ws, out=o)
        graphs.append(g)
    for _ in range(5):
        for o in outs:
            o.fill_(float("nan"))
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_threads_with_their_own_workspaces(cuda_device):
    """Four host threads on four streams, all four calls, the bits of one thread."""
    import threading

    import torch
    d = _dsb()
    rng = np.random.default_rng(43)
    D, hq, hkv = 64, 6, 2
    lens, new = [700, 200], [1, 3]
    bt, blocks, n_pages = _geometry(lens, new, [0, 0], rng)
    host_pool, rows = _pool(rng, n_pages, hkv, D), rng.standard_normal((4, (hq + 2 * hkv) * D)).astype(np.float32)
    batch, rot = d.PagedBatch(bt, blocks, [0, 0], new, lens), d.Rotary()

    def job(n, out):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            ws = d.Workspace(4, hq, D, 768)
            pool = to_dev(host_pool)
            kv = d.kv_q4_pages(pool, D)
            for _ in range(n):
                qkv = to_dev(rows)
                d.kv_append_q4(qkv, hq, kv, batch, rot, ws)
                q = qkv[:, :hq * D].unflatten(1, (hq, D))
                att = d.attention_decode_q4(q, kv, batch, ws)
                k, v = d.kv_gather_q4(kv, batch, [0, 0], lens, d.DSB_F16, ws)
                d.rope_rotary(q, None, np.arange(4), rot, ws)
            stream.synchronize()
            out.append([x.clone() for x in (att, k, v, qkv)])
            stream.synchronize()

    want, got = [], []
    job(1, want)
    threads = [threading.Thread(target=job, args=(25, got)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(got) == 4
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want[0]))
