"""The paged 4-bit KV cache and the rotary positions around it: what is measured.

Four operators, each in a plain form (elementary torch operations in 32 bits,
angles in 64) and through the library's own entry points (``own``):

``rope``    rotary positions on q and k rows in place: either pair layout, all
            or part of the head, plain or scaled for long contexts.
``append``  a step's (or a prompt's) [q | k | v] rows: q rotated in place, k
            rotated and k and v written as 4-bit rows into a paged cache; the
            rows just written are read back as the values they stand for.
``attn``    decode attention over the paged 4-bit cache.
``gather``  key and value rows of the 4-bit cache as 16-bit values.

The 4-bit row.  A head vector x of D values is stored as D codes 0..15 and two
fp16 numbers: d = fp16((max - min) / 15), z = fp16(min + 8 d), code =
clamp(round-half-even((x - z) / d) + 8, 0, 15) (8 where d is 0); it stands for
z + d (code - 8).  A page holds 128 keys; per page and kv head one block of
128 (D + 8) bytes:

    K codes   [128 keys][D/2] bytes, dimension 2i in the low half of byte i
    K (d, z)  [128 keys] pairs of fp16
    V codes   [64 key pairs][D/4 words][2 keys] 16-bit, word i of a key holding
              dimensions 4i .. 4i+3, the lowest four bits first
    V (d, z)  [128 keys] pairs of fp16
"""
import math

import numpy as np
import torch

own = False

PAGE = 128
THETA = 1e4
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one session, small heads: the smallest call
        {"name": "rope_one_token", "op": "rope", "n_tok": 1, "hq": 12, "hkv": 12, "d": 64, "rd": 64, "pairs": "half",
         "scale": "none", "far": 2000},
        # the rows of a long prompt, half of each head rotated in interleaved pairs, far positions
        {"name": "rope_prompt_part", "op": "rope", "n_tok": 6000, "hq": 40, "hkv": 8, "d": 128, "rd": 64,
         "pairs": "interleaved", "scale": "bands", "far": 120000},
        # one decode step of 16 sessions, per-head norms, grouped heads
        {"name": "append_step_16", "op": "append", "hq": 40, "hkv": 8, "d": 128, "rd": 128, "pairs": "half",
         "scale": "none", "seqs": 16, "new": 1, "len_lo": 1, "len_hi": 4096, "window": 0, "norm": True, "ragged": False,
         "mix": 1},
        # three drafts each of 8 sessions on sliding windows, part of the head rotated
        {"name": "append_draft_ring", "op": "append", "hq": 12, "hkv": 12, "d": 64, "rd": 48, "pairs": "interleaved",
         "scale": "linear", "seqs": 8, "new": 3, "len_lo": 128, "len_hi": 2048, "window": 300, "norm": False,
         "ragged": False, "mix": 2},
        # prompts of different lengths beside single tokens
        {"name": "append_prompts", "op": "append", "hq": 40, "hkv": 8, "d": 128, "rd": 128, "pairs": "half",
         "scale": "yarn", "seqs": 5, "new": 1600, "len_lo": 1600, "len_hi": 9000, "window": 0, "norm": True,
         "ragged": True, "mix": 3},
        # one short session: latency alone
        {"name": "attn_one_short", "op": "attn", "hq": 8, "hkv": 2, "d": 64, "seqs": 1, "new": 1, "len_lo": 200,
         "len_hi": 200, "window": 0, "ragged": False, "mix": 4},
        # the decode step of 16 sessions of all lengths
        {"name": "attn_step_16", "op": "attn", "hq": 40, "hkv": 8, "d": 128, "seqs": 16, "new": 1, "len_lo": 1,
         "len_hi": 4096, "window": 0, "ragged": False, "mix": 5},
        # many sessions, as many kv heads as query heads, four drafts, sliding windows
        {"name": "attn_draft_ring", "op": "attn", "hq": 12, "hkv": 12, "d": 64, "seqs": 64, "new": 4, "len_lo": 128,
         "len_hi": 2048, "window": 777, "ragged": True, "mix": 6},
        # eight drafts of 8 sessions on grouped heads: 40 query rows on each kv head
        {"name": "attn_draft_40_rows", "op": "attn", "hq": 40, "hkv": 8, "d": 128, "seqs": 8, "new": 8,
         "len_lo": 4096, "len_hi": 16384, "window": 0, "ragged": False, "mix": 7},
        # long contexts, as many kv heads as query heads: the largest read
        {"name": "attn_long", "op": "attn", "hq": 32, "hkv": 32, "d": 128, "seqs": 4, "new": 1, "len_lo": 16384,
         "len_hi": 65536, "window": 0, "ragged": False, "mix": 8},
        # a short prefix read back
        {"name": "gather_short", "op": "gather", "hkv": 2, "d": 64, "seqs": 1, "len_lo": 300, "len_hi": 300,
         "window": 0, "out": "f16", "mix": 9},
        # whole sessions read back (to move them to a 16-bit cache)
        {"name": "gather_sessions", "op": "gather", "hkv": 8, "d": 128, "seqs": 8, "len_lo": 4096, "len_hi": 16384,
         "window": 0, "out": "bf16", "mix": 10},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "gather"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 8, 12, 32])
    group = rng.choice([1, 2, 4, 5, 8])
    pairs, scale = rng.choice(["half", "interleaved"]), rng.choice(["none", "linear", "ntk", "bands", "yarn"])
    rd = rng.choice([d, d, d // 2, d - 16, d // 4 + 2])
    if op == "rope":
        n_tok = _log_int(rng, 1, 6000)
        while hkv * (group + 1) * n_tok > 48 * 6000:
            n_tok = (n_tok + 1) // 2
        return {"op": op, "n_tok": n_tok, "hq": hkv * group, "hkv": hkv, "d": d, "rd": rd, "pairs": pairs,
                "scale": scale, "far": _log_int(rng, 100, 1000000)}
    seqs = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, 65536)
    lo = rng.randint(max(1, hi // 4), hi)
    window = rng.choice([0, 0, 0, rng.randint(1, 1500)])
    if op == "append":
        new = _log_int(rng, 1, 2000)
        while seqs * new > 8000 or hkv * (group + 2) * seqs * new > 56 * 8000:
            seqs, new = (seqs + 1) // 2, (new + 1) // 2
        lo, hi = max(lo, new), max(hi, new)
        while seqs * hi > 200000:
            hi = max(lo, hi // 2)
            lo = max(new, lo // 2)
        return {"op": op, "hq": hkv * group, "hkv": hkv, "d": d, "rd": rd, "pairs": pairs, "scale": scale,
                "seqs": seqs, "new": new, "len_lo": lo, "len_hi": hi, "window": window,
                "norm": rng.random() < 0.5, "ragged": rng.random() < 0.5, "mix": rng.randint(100, 10 ** 6)}
    while seqs * hi * hkv * d > 4 * 40000 * 32 * 128:
        seqs, hi = (seqs + 1) // 2, (hi + 1) // 2
    lo = min(lo, hi)
    if op == "gather":
        while seqs * hi * hkv * d > 100000 * 8 * 128:
            seqs, hi = (seqs + 1) // 2, (hi + 1) // 2
        return {"op": op, "hkv": hkv, "d": d, "seqs": seqs, "len_lo": min(lo, hi), "len_hi": hi, "window": window,
                "out": rng.choice(["f16", "bf16"]), "mix": rng.randint(100, 10 ** 6)}
    new = rng.choice([1, 1, 1, 2, 4, 64 // group])
    new = min(new, 64 // group)
    lo, hi = max(lo, new), max(hi, new)
    while seqs > 1 and 4 * seqs * new * hkv * group * hi * d > 14e9:
        seqs = (seqs + 1) // 2
    return {"op": op, "hq": hkv * group, "hkv": hkv, "d": d, "seqs": seqs, "new": new, "len_lo": lo, "len_hi": hi,
            "window": window, "ragged": rng.random() < 0.4, "mix": rng.randint(100, 10 ** 6)}


# --------------------------------------------------- sizes that a seed fixes
def _lens(case):
    """Lengths after the step and new tokens of each sequence (host lists), one
    mix for each case's "mix"; the first sequence has the longest length."""
    g = torch.Generator().manual_seed(1000 + case["mix"])
    n, lo, hi, new = case["seqs"], case["len_lo"], case["len_hi"], case.get("new", 1)
    lens = torch.randint(lo, hi + 1, (n,), generator=g).tolist()
    lens[0] = hi
    fresh = [new] * n
    if case.get("ragged"):
        fresh = torch.randint(0, new + 1, (n,), generator=g).tolist()
        fresh[-1] = new
        if n > 2:
            fresh[1] = 1
    return lens, fresh


def _visited(length, new, window):
    """First key that any of the sequence's new tokens sees."""
    return max(0, length - max(new, 1) + 1 - window) if window else 0


def work(case):
    """The operands, each read once and each result written once (mean lengths)."""
    d = case["d"]
    if case["op"] == "rope":
        n = case["n_tok"] * (case["hq"] + case["hkv"]) * case["rd"]
        return {"bytes": 8 * n, "flops": 3 * n}
    hkv, n = case["hkv"], case["seqs"]
    mean = (case["len_lo"] + case["len_hi"]) / 2 * (n - 1) + case["len_hi"]
    if case["op"] == "gather":
        keys = min(mean, n * _ring(case["window"], 1) * PAGE) if case["window"] else mean
        return {"bytes": keys * hkv * (d + 8 + 4 * d), "flops": 4 * keys * hkv * d}
    rows = n * case["new"] * (0.5 if case["ragged"] else 1.0)
    if case["op"] == "append":
        hq = case["hq"]
        return {"bytes": rows * d * 4 * (2 * hq + 2 * hkv) + rows * hkv * (2 * (d + 8) + 4 * d),
                "flops": rows * d * (3 * hq + 15 * hkv)}
    if case["window"]:
        mean = min(mean, n * (case["window"] + case["new"] - 1))
    return {"bytes": mean * hkv * (d + 8) + 8 * rows * case["hq"] * d,
            "flops": 4.0 * mean / n * rows * case["hq"] * d}


def _ring(window, new):
    """Pages of a ring that keeps a window beside a call's new rows."""
    return (window + new - 1 + PAGE - 1) // PAGE + 1


# ------------------------------------------------------------------- inputs
def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(77000 + seed)


def _spread(x, g):
    """Head vectors as a trained model's: a few wide dimensions, a size of its own for each row."""
    d = x.shape[-1]
    wide = 1 + 6 * (torch.rand(d, device="cuda", generator=g) < 0.05).float()
    size = torch.exp(0.4 * torch.randn(x.shape[:-1] + (1,), device="cuda", generator=g))
    return x * wide * size


def _frequencies(case):
    """float64 frequency of each pair and the factor on the rotated values."""
    rd, theta, scale = case["rd"], THETA, case["scale"]
    i = torch.arange(rd // 2, dtype=torch.float64, device="cuda")
    if scale == "ntk":
        theta = theta * 4.0 ** (rd / (rd - 2))
    f = theta ** (-2.0 * i / rd)
    if scale == "linear":
        return f / 8.0, 1.0
    if scale == "bands":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0, 1)
        return f * keep + f / 8.0 * (1 - keep), 1.0
    if scale == "yarn":
        def at(b):
            return rd * math.log(4096 / (2 * math.pi * b)) / (2 * math.log(theta))
        low, high = max(math.floor(at(32.0)), 0), min(math.ceil(at(1.0)), rd - 1)
        ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
        return f * (1 - ramp) + f / 4.0 * ramp, 0.1 * math.log(4.0) + 1.0
    return f, 1.0


def _rotary(dsb, case):
    """The library's description of the same rotation."""
    kinds = {"none": {}, "linear": {"scaling": "linear", "factor": 8.0}, "ntk": {"scaling": "ntk", "factor": 4.0},
             "bands": {"scaling": "bands", "factor": 8.0, "orig_ctx": 8192, "low": 1.0, "high": 4.0},
             "yarn": {"yarn": dsb.Yarn(4.0, 4096)}}
    return dsb.Rotary(THETA, rotary_dim=case["rd"], interleaved=case["pairs"] == "interleaved", **kinds[case["scale"]])


def _tables(case, seed, lens, fresh):
    """Block tables over a shuffled pool (host lists) and the pool's page count."""
    g = torch.Generator().manual_seed(5000 + seed)
    w = case["window"]
    blocks = []
    for length, new in zip(lens, fresh):
        full = (length + PAGE - 1) // PAGE
        blocks.append(_ring(w, new) if w else full)
    total = sum(blocks) + 3
    order = torch.randperm(total, generator=g).tolist()
    table, at = torch.zeros((len(lens), max(blocks)), dtype=torch.int32), 0
    for s, n in enumerate(blocks):
        table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    return table, blocks, total


def _places(table, blocks, case, seqs, keys):
    """(page, row) on the device of key position keys[i] of sequence seqs[i]."""
    t, n = table.cuda().long(), torch.tensor(blocks, device="cuda")
    i = torch.div(keys, PAGE, rounding_mode="floor")
    i = i % n[seqs] if case["window"] else i
    return t[seqs, i], keys % PAGE


def _fill(pool, hkv, d, g):
    """Writes quantised rows of spread normal values into every page, some pages at a time."""
    step = max(1, (1 << 25) // (hkv * PAGE * d))
    for a in range(0, pool.shape[0], step):
        part = pool[a:a + step]
        n = part.shape[0]
        for which in (0, 1):
            x = _spread(torch.randn((n, hkv, PAGE, d), device="cuda", generator=g), g)
            codes, dz = _quantise(x)
            _pack(part, which, codes, dz)


def _sections(pool, d):
    """The four parts of every (page, head) block, as views."""
    c = PAGE * d // 2
    k, kz, v, vz = torch.split(pool, [c, 4 * PAGE, c, 4 * PAGE], dim=-1)
    return k, kz, v, vz


def _pack(pool, which, codes, dz):
    """Codes uint8 [n, hkv, 128, d] and (d, z) fp16 [n, hkv, 128, 2] into whole pages."""
    n, hkv, _, d = codes.shape
    part = _sections(pool, d)
    if which == 0:
        part[0].copy_((codes[..., 0::2] | codes[..., 1::2] << 4).reshape(n, hkv, -1))
    else:
        b = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(n, hkv, PAGE // 2, 2, d // 4, 2)
        part[2].copy_(b.permute(0, 1, 2, 4, 3, 5).reshape(n, hkv, -1))
    part[1 + 2 * which].copy_(dz.contiguous().view(torch.uint8).reshape(n, hkv, -1))


def prepare(case, seed):
    g = _gen(case, seed)
    s = {"case": case}
    op, d = case["op"], case["d"]
    if op == "rope":
        n = case["n_tok"]
        rows = torch.randn((n, case["hq"] + 2 * case["hkv"], d), device="cuda", generator=g)
        # prompt rows sit side by side, so do the heads of a projection's output
        s["q"], s["k"] = rows[:, :case["hq"]], rows[:, case["hq"]:case["hq"] + case["hkv"]]
        h = torch.Generator().manual_seed(9000 + seed)
        first = int(torch.randint(0, case["far"], (1,), generator=h))
        s["pos"] = np.arange(first, first + n, dtype=np.int32)
        s["pos_dev"] = torch.arange(first, first + n, device="cuda")
        s["freq"] = _frequencies(case)
        if own:
            from session_decode_step_dsb_gb300 import dsb
            s["rotary"], s["ws"] = _rotary(dsb, case), dsb.Workspace(n, case["hq"], d, PAGE)
        return s
    hkv = case["hkv"]
    lens, fresh = _lens(case)
    if op == "gather":
        fresh = [0] * len(lens)
    table, blocks, pages = _tables(case, seed, lens, fresh)
    pool = torch.empty((pages, hkv, PAGE * (d + 8)), dtype=torch.uint8, device="cuda")
    if op == "append":
        pool.fill_(0)
    else:
        _fill(pool, hkv, d, g)
    s.update(lens=lens, fresh=np.array(fresh, np.int32), pool=pool, table=table, blocks=blocks)
    n_tok = sum(fresh)
    s["lens_dev"], s["fresh_dev"] = torch.tensor(lens, device="cuda"), torch.tensor(fresh, device="cuda")
    if op == "gather":
        first = [max(0, n - b * PAGE) for n, b in zip(lens, blocks)] if case["window"] else [0] * len(lens)
        count = [n - f for n, f in zip(lens, first)]
        s["first"], s["count"] = np.array(first, np.int32), np.array(count, np.int32)
        seqs = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(count, device="cuda"))
        keys = torch.cat([torch.arange(f, f + c, device="cuda") for f, c in zip(first, count)])
        s["places"] = _places(table, blocks, case, seqs, keys)
    else:
        seqs = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(fresh, device="cuda"))
        pos = torch.cat([torch.arange(n - f, n, device="cuda") for n, f in zip(lens, fresh)])
        s["seqs"], s["pos_dev"] = seqs, pos
    if op == "append":
        s["qkv"] = torch.randn((n_tok, (case["hq"] + 2 * hkv) * d), device="cuda", generator=g)
        heads = s["qkv"].view(n_tok, -1, d)
        heads[:, case["hq"]:] = _spread(heads[:, case["hq"]:], g)
        s["places"], s["freq"] = _places(table, blocks, case, seqs, pos), _frequencies(case)
        if case["norm"]:
            s["q_norm"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
            s["k_norm"] = 1 + 0.1 * torch.randn(d, device="cuda", generator=g)
    if op == "attn":
        s["q"] = torch.randn((n_tok, case["hq"], d), device="cuda", generator=g)
        # the plain form's view: the pages each sequence visits, padded to the longest
        new, w = max(fresh), case["window"]
        first = [_visited(n, f, w) // PAGE for n, f in zip(lens, fresh)]
        many = [(n - 1) // PAGE - c + 1 for n, c in zip(lens, first)]
        idx = torch.arange(max(many))[None, :] + torch.tensor(first)[:, None]
        inside = idx < torch.tensor([(n + PAGE - 1) // PAGE for n in lens])[:, None]
        col = idx % torch.tensor(blocks)[:, None] if w else idx.clamp(max=table.shape[1] - 1)
        s["pages"] = torch.where(inside, torch.gather(table.long(), 1, col), 0).cuda()
        s["first_key"] = torch.tensor(first, device="cuda") * PAGE
        # rows of the ragged queries in a padded [sequence, draft] grid
        start = torch.tensor(fresh).cumsum(0) - torch.tensor(fresh)
        s["slot"] = (seqs * new + torch.arange(n_tok, device="cuda") - start.cuda()[seqs])
        s["new"] = new
    if own:
        from session_decode_step_dsb_gb300 import dsb
        s["kv"] = dsb.kv_q4_pages(pool, d)
        s["batch"] = dsb.PagedBatch(table.numpy(), blocks, [case["window"]] * len(lens), fresh, lens)
        s["ws"] = dsb.Workspace(max(n_tok, 1), case.get("hq", 1), d, max(lens))
        if op == "append":
            s["rotary"] = _rotary(dsb, case)
            s["got"] = np.array([n - f for n, f in zip(lens, fresh)], np.int32)
    return s


# ------------------------------------------------------------- plain forms
def _rotate(x, pos, case, freq):
    """x [n, heads, d] rotated by its rows' positions."""
    f, m = freq
    a = pos.double()[:, None, None] * f
    c, sn = (torch.cos(a) * m).float(), (torch.sin(a) * m).float()
    rd, half = case["rd"], case["rd"] // 2
    out = x.clone()
    if case["pairs"] == "interleaved":
        x1, x2 = x[..., 0:rd:2], x[..., 1:rd:2]
        out[..., 0:rd:2], out[..., 1:rd:2] = x1 * c - x2 * sn, x1 * sn + x2 * c
    else:
        x1, x2 = x[..., :half], x[..., half:rd]
        out[..., :half], out[..., half:rd] = x1 * c - x2 * sn, x1 * sn + x2 * c
    return out


def _norm(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _quantise(x):
    """Codes uint8 and (d, z) fp16 of every head vector of x."""
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    d = ((hi - lo) / 15).half()
    z = (lo + 8 * d.float()).half()
    q = torch.where(d == 0, 8.0, (torch.round((x - z.float()) / d.float()) + 8).clamp(0, 15))
    return q.to(torch.uint8), torch.cat([d, z], -1)


def _values(codes, dz):
    return dz[..., 1:].float() + dz[..., :1].float() * (codes.float() - 8)


def _page_values(pool, pages, d):
    """float32 K and V [..., hkv, 128, d] of whole pages."""
    blocks = pool[pages]
    lead = blocks.shape[:-1]
    k, kz, v, vz = _sections(blocks, d)
    low, high = k & 15, k >> 4
    codes = torch.stack([low, high], -1).reshape(*lead, PAGE, d)
    key = _values(codes, kz.contiguous().view(torch.float16).reshape(*lead, PAGE, 2))
    v = v.reshape(*lead, PAGE // 2, d // 4, 2, 2).transpose(-2, -3)  # pair, key, word, byte
    codes = torch.stack([v & 15, v >> 4], -1).reshape(*lead, PAGE, d)
    return key, _values(codes, vz.contiguous().view(torch.float16).reshape(*lead, PAGE, 2))


def _row_values(pool, page, row, d):
    """float32 K and V [n, hkv, d] of single rows."""
    k, kz, v, vz = _sections(pool, d)
    n, hkv = pool.shape[:2]
    r = row[:, None]
    h = torch.arange(hkv, device="cuda")[None]
    p = page[:, None]
    k = k.reshape(n, hkv, PAGE, d // 2)[p, h, r]
    key = _values(torch.stack([k & 15, k >> 4], -1).flatten(-2),
                  kz.reshape(n, hkv, PAGE, 4)[p, h, r].view(torch.float16))
    v = v.reshape(n, hkv, PAGE // 2, d // 4, 2, 2)[p, h, torch.div(r, 2, rounding_mode="floor"), :, r % 2]
    return key, _values(torch.stack([v & 15, v >> 4], -1).flatten(-3),
                        vz.reshape(n, hkv, PAGE, 4)[p, h, r].view(torch.float16))


def _write_rows(pool, page, row, which, codes, dz):
    """Codes [n, hkv, d] and (d, z) of the rows into their places of the pool."""
    n, hkv, d = pool.shape[0], pool.shape[1], codes.shape[-1]
    part = _sections(pool, d)
    h, p, r = torch.arange(hkv, device="cuda")[None], page[:, None], row[:, None]
    b = codes[..., 0::2] | codes[..., 1::2] << 4
    if which == 0:
        place = torch.arange(d // 2, device="cuda") + r[..., None] * (d // 2)
        part[0][p[..., None], h[..., None], place] = b
    else:
        byte = torch.arange(d // 2, device="cuda")
        place = torch.div(r, 2, rounding_mode="floor")[..., None] * d + (r % 2)[..., None] * 2 + byte % 2 + \
            torch.div(byte, 2, rounding_mode="floor") * 4
        part[2][p[..., None], h[..., None], place] = b
    place = r[..., None] * 4 + torch.arange(4, device="cuda")
    part[1 + 2 * which][p[..., None], h[..., None], place] = dz.contiguous().view(torch.uint8)


def _run_rope(s):
    case = s["case"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        dsb.rope_rotary(s["q"], s["k"], s["pos"], s["rotary"], s["ws"])
    else:
        s["q"].copy_(_rotate(s["q"], s["pos_dev"], case, s["freq"]))
        s["k"].copy_(_rotate(s["k"], s["pos_dev"], case, s["freq"]))
    return {"q": s["q"], "k": s["k"]}


def _run_append(s):
    case = s["case"]
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        dsb.kv_append_q4(s["qkv"], hq, s["kv"], s["batch"], s["rotary"], s["ws"], q_norm=s.get("q_norm"),
                         k_norm=s.get("k_norm"), eps=EPS if case["norm"] else 0.0)
        k, v = dsb.kv_gather_q4(s["kv"], s["batch"], s["got"], s["fresh"], dsb.DSB_F16, s["ws"])
        return {"qkv": s["qkv"], "k": k, "v": v}
    heads = s["qkv"].view(s["qkv"].shape[0], hq + 2 * hkv, d)
    q, k, v = heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:]
    if case["norm"]:
        q, k = _norm(q, s["q_norm"]), _norm(k, s["k_norm"])
    heads[:, :hq] = _rotate(q, s["pos_dev"], case, s["freq"])
    page, row = s["places"]
    _write_rows(s["pool"], page, row, 0, *_quantise(_rotate(k, s["pos_dev"], case, s["freq"])))
    _write_rows(s["pool"], page, row, 1, *_quantise(v))
    k, v = _row_values(s["pool"], page, row, d)
    return {"qkv": s["qkv"], "k": k.half(), "v": v.half()}


def _run_attn(s):
    case = s["case"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        return dsb.attention_decode_q4(s["q"], s["kv"], s["batch"], s["ws"])
    hq, hkv, d, new, w = case["hq"], case["hkv"], case["d"], s["new"], case["window"]
    n = len(s["lens"])
    key, val = _page_values(s["pool"], s["pages"], d)  # [n, pages, hkv, 128, d]
    key, val = (x.transpose(1, 2).reshape(n, hkv, -1, d) for x in (key, val))
    q = torch.zeros((n * new, hq, d), device="cuda").index_copy_(0, s["slot"], s["q"])
    q = q.view(n, new, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    score = q @ key.transpose(-1, -2) / math.sqrt(d)
    score = score.view(n, hkv, new, hq // hkv, -1)
    at = s["first_key"][:, None] + torch.arange(key.shape[2], device="cuda")
    pos = s["lens_dev"][:, None] - s["fresh_dev"][:, None] + torch.arange(new, device="cuda")
    seen = at[:, None] <= pos[..., None]
    if w:
        seen = seen & (at[:, None] > pos[..., None] - w)
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    # the weights of a page past a sequence's last key are zero, whatever the page holds
    e = (e / e.sum(-1, keepdim=True)).view(n, hkv, -1, key.shape[2])
    out = (e @ val).view(n, hkv, new, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n * new, hq, d)
    return out[s["slot"]]


def _run_gather(s):
    case = s["case"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        return dsb.kv_gather_q4(s["kv"], s["batch"], s["first"], s["count"],
                                dsb.DSB_F16 if case["out"] == "f16" else dsb.DSB_BF16, s["ws"])
    to = torch.float16 if case["out"] == "f16" else torch.bfloat16
    k, v = _row_values(s["pool"], *s["places"], case["d"])
    return k.to(to), v.to(to)


def run(state):
    return {"rope": _run_rope, "append": _run_append, "attn": _run_attn, "gather": _run_gather}[state["case"]["op"]](
        state)


# ------------------------------------------------ the definition in 64 bits
def _exact_rotation(case, pos):
    """Complex float64 turn [n, rd/2] of each pair of each row."""
    rd, s = case["rd"], case["scale"]
    base = THETA if s != "ntk" else THETA * 4.0 ** (rd / (rd - 2.0))
    freq, gain = [], 1.0
    for i in range(rd // 2):
        f = math.pow(base, -2.0 * i / rd)
        if s == "linear":
            f /= 8.0
        elif s == "bands":
            turns = 8192.0 * f / (2.0 * math.pi)
            blend = min(1.0, max(0.0, (turns - 1.0) / 3.0))
            f = blend * f + (1.0 - blend) * f / 8.0
        elif s == "yarn":
            lo = max(0, math.floor(rd * math.log(4096 / (64.0 * math.pi)) / (2 * math.log(base))))
            hi = min(rd - 1, math.ceil(rd * math.log(4096 / (2.0 * math.pi)) / (2 * math.log(base))))
            t = min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001)))
            f, gain = f * (1 - t) + t * f / 4.0, 1.0 + 0.1 * math.log(4.0)
        freq.append(f)
    angle = torch.outer(pos.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    return torch.polar(torch.full_like(angle, gain), angle)


def _exact_turn(x, turn, case):
    y, rd = x.double().clone(), case["rd"]
    if case["pairs"] == "interleaved":
        pair = torch.view_as_complex(y[..., :rd].reshape(*y.shape[:-1], rd // 2, 2).contiguous())
        y[..., :rd] = torch.view_as_real(pair * turn[:, None]).flatten(-2)
    else:
        z = torch.complex(y[..., :rd // 2], y[..., rd // 2:rd]) * turn[:, None]
        y[..., :rd // 2], y[..., rd // 2:rd] = z.real, z.imag
    return y


def _exact_row(x):
    """The values that the 4-bit rows of float64 head vectors stand for."""
    least, most = x.min(-1, keepdim=True)[0], x.max(-1, keepdim=True)[0]
    step = ((most - least) / 15.0).half().double()
    mid = (least + 8.0 * step).half().double()
    level = torch.where(step > 0, torch.round((x - mid) / step.clamp(min=1e-300)), torch.zeros_like(x))
    return mid + step * level.clamp(-8, 7)


def _exact_pages(pool, d, pages):
    """float64 K and V [pages * 128, d] of one head's pages; pool: that head's blocks."""
    raw = pool[pages].to(torch.int32)
    c = PAGE * d // 2

    def numbers(b):  # (d, z) from little-endian bytes
        return (b[:, 0::2] + 256 * b[:, 1::2]).to(torch.int16).view(torch.float16).double().view(-1, PAGE, 2)

    byte = torch.arange(d, device="cuda") // 2
    up = 4 * (torch.arange(d, device="cuda") % 2)
    kc = raw[:, :c].view(-1, PAGE, d // 2)[..., byte] >> up & 15
    key = torch.arange(PAGE, device="cuda")[:, None]
    where = key // 2 * d + byte // 2 * 4 + key % 2 * 2 + byte % 2
    vc = raw[:, c + 4 * PAGE:2 * c + 4 * PAGE][:, where] >> up & 15
    kn, vn = numbers(raw[:, c:c + 4 * PAGE]), numbers(raw[:, 2 * c + 4 * PAGE:])
    return ((kn[..., 1:] + kn[..., :1] * (kc - 8)).view(-1, d), (vn[..., 1:] + vn[..., :1] * (vc - 8)).view(-1, d))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turn = _exact_rotation(case, s["pos_dev"])
        return {"q": _exact_turn(s["q"], turn, case), "k": _exact_turn(s["k"], turn, case)}
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "append":
        hq = case["hq"]
        x = s["qkv"].double().view(-1, hq + 2 * hkv, d)
        turn = _exact_rotation(case, s["pos_dev"])
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        if case["norm"]:
            q = q / (q.square().mean(-1, keepdim=True) + EPS).sqrt() * s["q_norm"].double()
            k = k / (k.square().mean(-1, keepdim=True) + EPS).sqrt() * s["k_norm"].double()
        qkv = x.clone()
        qkv[:, :hq] = _exact_turn(q, turn, case)
        return {"qkv": qkv.view(s["qkv"].shape), "k": _exact_row(_exact_turn(k, turn, case)), "v": _exact_row(v)}
    if case["op"] == "gather":
        ks, vs = [], []
        for b in range(len(s["lens"])):
            t = s["table"][b]
            first, n = s["first"][b], s["count"][b]
            i = torch.arange(first // PAGE, (first + n - 1) // PAGE + 1)
            pages = t[i % s["blocks"][b] if case["window"] else i].long().cuda()
            at = first - first // PAGE * PAGE
            rows = [_exact_pages(s["pool"][:, h], d, pages) for h in range(hkv)]
            ks.append(torch.stack([r[0][at:at + n] for r in rows], 1))
            vs.append(torch.stack([r[1][at:at + n] for r in rows], 1))
        return torch.cat(ks), torch.cat(vs)
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    group, row = case["hq"] // hkv, 0
    if sum(n * f for n, f in zip(s["lens"], s["fresh"])) * case["hq"] * d > 4e10:
        return None
    for b, (length, new) in enumerate(zip(s["lens"], s["fresh"])):
        if new == 0:
            continue
        c = _visited(length, new, case["window"]) // PAGE
        i = torch.arange(c, (length - 1) // PAGE + 1)
        pages = s["table"][b][i % s["blocks"][b] if case["window"] else i].long().cuda()
        for h in range(hkv):
            key, val = _exact_pages(s["pool"][:, h], d, pages)
            at = c * PAGE + torch.arange(key.shape[0], device="cuda")
            for j in range(new):
                pos = length - new + j
                see = (at <= pos) & ((at > pos - case["window"]) if case["window"] else (at >= 0))
                logit = s["q"][row + j, h * group:(h + 1) * group].double() @ key[see].T / d ** 0.5
                out[row + j, h * group:(h + 1) * group] = torch.softmax(logit, -1) @ val[see]
        row += new
    return out
