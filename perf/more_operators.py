"""Pages that sequences share, copy and leave out: what is measured.

A cache of 16-bit (or 4-bit) pages of 128 keys, as a batch of sessions keeps
it, and what a server does with whole pages of it.  Four operators, each in a
plain form (elementary torch operations in 32 bits) and through the library's
own entry points (``own``):

``copy``    rows of pages into other pages, in every layer's pool: a fork copies
            the last, partly filled page of a session (the full ones are
            shared), a compaction moves whole pages.
``shared``  decode attention over a ragged paged batch whose sequences begin with
            the same pages (a system prompt, the samples of one question).
``select``  the smallest and largest value of each key dimension over the pages
            that new tokens touched, then, for every new token and kv head,
            the pages with the largest score.
``sparse``  decode attention over the selected pages alone.

The score of a page for the query rows r of a kv head's group is
sum_d a_d hi_d + b_d lo_d with a_d = sum_r max(q_rd, 0), b_d = sum_r min(q_rd, 0)
and lo, hi the page's bounds: no key of the page has a larger sum of q_r . k.
Every product and sum is rounded to 32 bits; sums are added pairwise, neighbours
first (the rows of a group padded with zeros to a power of two), so that a
selection has one right answer.  Always selected: the first ``first`` pages and
the newest ``last``, up to the token's own; then the largest scores, ties to the
lowest index.
"""
import math

import numpy as np
import torch

own = False

PAGE = 128


# ------------------------------------------------------------------- cases
def listed():
    return [
        # three sessions of a small model forked in the middle of a page, two layers: the smallest call
        {"name": "copy_fork_small", "op": "copy", "kind": "f16", "layers": 2, "hkv": 12, "d": 64, "copies": 3,
         "whole": False, "mix": 1},
        # 16 forks in the 40 layers of the 14B-shaped model
        {"name": "copy_fork_40_layers", "op": "copy", "kind": "bf16", "layers": 40, "hkv": 8, "d": 128, "copies": 16,
         "whole": False, "mix": 2},
        # a pool of 4-bit pages compacted: whole pages move in 40 layers
        {"name": "copy_compact_q4", "op": "copy", "kind": "q4", "layers": 40, "hkv": 8, "d": 128, "copies": 50,
         "whole": True, "mix": 3},
        # four sessions of the small model behind a short common prompt
        {"name": "shared_small", "op": "shared", "kind": "f16", "hq": 12, "hkv": 12, "d": 64, "groups": 1, "per": 4,
         "common": 2, "branch": 0, "tail_lo": 20, "tail_hi": 200, "new": 1, "ragged": False, "mix": 4},
        # a decode step of 16 sessions behind one system prompt, the 14B-shaped model
        {"name": "shared_step_16", "op": "shared", "kind": "bf16", "hq": 40, "hkv": 8, "d": 128, "groups": 1,
         "per": 16, "common": 16, "branch": 0, "tail_lo": 1, "tail_hi": 2048, "new": 1, "ragged": False, "mix": 5},
        # eight questions behind one prompt, eight samples of each
        {"name": "shared_samples_8x8", "op": "shared", "kind": "f16", "hq": 40, "hkv": 8, "d": 128, "groups": 8,
         "per": 8, "common": 8, "branch": 9, "tail_lo": 1, "tail_hi": 700, "new": 1, "ragged": False, "mix": 6},
        # 32 sessions with up to four drafts each on one document of 32768 keys
        {"name": "shared_document_32k", "op": "shared", "kind": "f16", "hq": 40, "hkv": 8, "d": 128, "groups": 1,
         "per": 32, "common": 256, "branch": 0, "tail_lo": 4, "tail_hi": 1000, "new": 4, "ragged": True, "mix": 7},
        # prompts of a thousand tokens that arrive behind a cached prefix
        {"name": "shared_prompts", "op": "shared", "kind": "bf16", "hq": 40, "hkv": 8, "d": 128, "groups": 1, "per": 4,
         "common": 32, "branch": 0, "tail_lo": 1000, "tail_hi": 1000, "new": 1000, "ragged": False, "mix": 8},
        # one session of the small model
        {"name": "select_small", "op": "select", "kind": "f16", "hq": 12, "hkv": 12, "d": 64, "seqs": 1, "new": 1,
         "len_lo": 5000, "len_hi": 5000, "n_select": 8, "first": 1, "last": 1, "mix": 9},
        # 16 sessions of long contexts, an eighth to a half of the pages
        {"name": "select_step_64k", "op": "select", "kind": "bf16", "hq": 40, "hkv": 8, "d": 128, "seqs": 16, "new": 1,
         "len_lo": 16384, "len_hi": 65536, "n_select": 64, "first": 1, "last": 2, "mix": 10},
        # the attention that follows, of the one session and of the 16
        {"name": "sparse_small", "op": "sparse", "kind": "f16", "hq": 12, "hkv": 12, "d": 64, "seqs": 1, "new": 1,
         "len_lo": 5000, "len_hi": 5000, "n_select": 8, "mix": 11},
        {"name": "sparse_step_64k", "op": "sparse", "kind": "bf16", "hq": 40, "hkv": 8, "d": 128, "seqs": 16, "new": 1,
         "len_lo": 16384, "len_hi": 65536, "n_select": 64, "mix": 12},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["copy", "shared", "shared", "select", "sparse"])
    d = rng.choice([64, 128])
    hkv = rng.choice([1, 2, 3, 8, 12, 32])
    group = rng.choice([1, 2, 4, 5, 8])
    kind = rng.choice(["f16", "bf16"])
    mix = rng.randint(100, 10 ** 6)
    if op == "copy":
        kind = rng.choice(["f16", "bf16", "q4"])
        layers, copies = _log_int(rng, 1, 48), _log_int(rng, 1, 200)
        while layers * copies * hkv * d > 40 * 16 * 8 * 128:
            copies = (copies + 1) // 2
            layers = layers if copies > 1 else (layers + 1) // 2
        return {"op": op, "kind": kind, "layers": layers, "hkv": hkv, "d": d, "copies": copies,
                "whole": rng.random() < 0.3, "mix": mix}
    if op == "shared":
        groups, per = _log_int(rng, 1, 8), _log_int(rng, 1, 32)
        common = rng.choice([0, _log_int(rng, 1, 256)])
        branch = rng.choice([0, _log_int(rng, 1, 64)])
        new = rng.choice([1, 1, 1, 2, 4, _log_int(rng, 5, 1000)])
        tail_hi = max(new, _log_int(rng, 1, 3000))
        tail_lo = rng.randint(max(new, tail_hi // 8), tail_hi)
        while groups * per > 1 and (groups * per * hkv * d * ((common + branch) * PAGE + tail_hi) > 3.4e4 * 32 * 1024
                                    or groups * per * new * hkv * group * ((common + branch) * PAGE + tail_hi) > 4e8):
            groups, per = (groups + 1) // 2, (per + 1) // 2 if groups == 1 else per
        while new * hkv * group * ((common + branch) * PAGE + tail_hi) > 4e8:
            new = (new + 1) // 2
        return {"op": op, "kind": kind, "hq": hkv * group, "hkv": hkv, "d": d, "groups": groups, "per": per,
                "common": common, "branch": branch, "tail_lo": tail_lo, "tail_hi": tail_hi, "new": new,
                "ragged": rng.random() < 0.4, "mix": mix}
    seqs = _log_int(rng, 1, 32)
    new = rng.choice([1, 1, 1, 2, 4, _log_int(rng, 5, 60)])
    hi = max(new, _log_int(rng, 1, 65536))
    n_select = _log_int(rng, 3, 100)
    while seqs > 1 and (seqs * hi * hkv * d > 16 * 41000 * 1024 or seqs * new * hkv * d * (hi // PAGE + 1) > 1.2e8
                        or seqs * new * hkv * d * n_select > 3e6):
        seqs = (seqs + 1) // 2
    while new > 1 and (new * hkv * d * (hi // PAGE + 1) > 1.2e8 or new * hkv * d * n_select > 3e6):
        new = (new + 1) // 2
    case = {"op": op, "kind": kind, "hq": hkv * group, "hkv": hkv, "d": d, "seqs": seqs, "new": new,
            "len_lo": rng.randint(max(new, hi // 4), hi), "len_hi": hi, "n_select": n_select, "mix": mix}
    if op == "select":
        case.update(first=rng.randint(0, 1), last=rng.randint(1, 2))
    return case


# --------------------------------------------------- sizes that a case fixes
def _host(case, more=0):
    return torch.Generator().manual_seed(4000 + case["mix"] + more)


def _lens(case):
    """Lengths after the step and new tokens of each sequence (host lists)."""
    g, new = _host(case), case["new"]
    if case["op"] == "shared":
        n = case["groups"] * case["per"]
        base = (case["common"] + case["branch"]) * PAGE
        lens = torch.randint(case["tail_lo"], case["tail_hi"] + 1, (n,), generator=g)
        lens = (base + lens.clamp(min=new)).tolist()
    else:
        n = case["seqs"]
        lens = torch.randint(case["len_lo"], case["len_hi"] + 1, (n,), generator=g).tolist()
        lens[0] = case["len_hi"]
    fresh = [new] * n
    if case.get("ragged"):
        fresh = torch.randint(0, new + 1, (n,), generator=g).tolist()
        fresh[-1] = new
    return lens, fresh


def _copied(case):
    """Keys that each copy takes."""
    if case["whole"]:
        return [PAGE] * case["copies"]
    return torch.randint(1, PAGE + 1, (case["copies"],), generator=_host(case)).tolist()


def work(case):
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "copy":
        one = hkv * (d + 8 if case["kind"] == "q4" else 4 * d)
        return {"bytes": 2 * sum(_copied(case)) * case["layers"] * one, "flops": 0}
    lens, fresh = _lens(case)
    hq, rows = case["hq"], sum(fresh)
    if case["op"] == "shared":
        base = (case["common"] + case["branch"]) * PAGE
        keys = case["common"] * PAGE + case["groups"] * case["branch"] * PAGE + \
            sum(n - base for n, f in zip(lens, fresh) if f)
        seen = sum(f * n - f * (f - 1) // 2 for n, f in zip(lens, fresh))
        return {"bytes": keys * hkv * d * 4 + 8 * rows * hq * d, "flops": 4 * d * hq * seen}
    blocks = [(n + PAGE - 1) // PAGE for n in lens]
    if case["op"] == "select":
        touched = sum(n - (n - f) // PAGE * PAGE for n, f in zip(lens, fresh))
        return {"bytes": 4 * d * hkv * sum(blocks) + 2 * d * hkv * touched + 4 * rows * hq * d
                + 4 * rows * hkv * case["n_select"],
                "flops": sum(f * b for f, b in zip(fresh, blocks)) * hkv * 4 * d}
    keys = sum(f * min(b, case["n_select"]) for f, b in zip(fresh, blocks)) * PAGE
    # a page that several tokens of a sequence select need be read once
    once = sum(min(b, f * case["n_select"]) for f, b in zip(fresh, blocks)) * PAGE
    return {"bytes": once * hkv * d * 4 + 8 * rows * hq * d, "flops": 4 * d * hq * keys}


# ------------------------------------------------------------------- inputs
def _type(case):
    return {"f16": torch.float16, "bf16": torch.bfloat16}[case["kind"]]


def _fill(pool, g, wide):
    """Head vectors as a trained model's: a few wide dimensions (keys), a size of its own for each row."""
    step = max(1, (1 << 26) // pool[0].numel())
    d = pool.shape[-1]
    scale = 1 + wide * (torch.rand(d, device="cuda", generator=g) < 0.05).float()
    for a in range(0, pool.shape[0], step):
        part = pool[a:a + step]
        x = torch.randn(part.shape, device="cuda", generator=g)
        size = torch.exp(0.3 * torch.randn(part.shape[:-1] + (1,), device="cuda", generator=g))
        part.copy_(x * scale * size)


def _chains(case, seed, lens):
    """Block table over a shuffled pool: common pages, a group's pages, own pages."""
    g = torch.Generator().manual_seed(6000 + seed)
    blocks = [(n + PAGE - 1) // PAGE for n in lens]
    common, branch = case.get("common", 0), case.get("branch", 0)
    per = case.get("per", 1)
    groups = case.get("groups", len(lens))
    total = common + groups * branch + sum(b - common - branch for b in blocks) + 2
    order = torch.randperm(total, generator=g)
    table, at = torch.zeros((len(lens), max(blocks)), dtype=torch.int32), common + groups * branch
    for s, n in enumerate(blocks):
        k = s // per
        own_pages = n - common - branch
        table[s, :n] = torch.cat([order[:common], order[common + k * branch:common + (k + 1) * branch],
                                  order[at:at + own_pages]]).to(torch.int32)
        at += own_pages
    return table, blocks, total


def _key_of_byte(d):
    """The key that each byte of a 4-bit page's block of one head belongs to."""
    k = torch.arange(PAGE).repeat_interleave(d // 2)
    n = torch.arange(PAGE).repeat_interleave(4)
    at = torch.arange(PAGE * d // 2)
    v = at // d * 2 + at % 4 // 2  # pairs of keys, two bytes of each in turn
    return torch.cat([k, n, v, n]).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(88000 + seed)
    s, op, d, hkv = {"case": case}, case["op"], case["d"], case["hkv"]
    if op == "copy":
        keys, n, layers = _copied(case), case["copies"], case["layers"]
        pages = 2 * n + 3
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(6000 + seed))
        src, dst = order[:n], order[n:2 * n]
        if n > 2:
            src[1] = src[0]  # two forks of one session
        if case["kind"] == "q4":
            pool = torch.randint(0, 256, (layers, pages, hkv, PAGE * (d + 8)), dtype=torch.uint8, device="cuda",
                                 generator=g)
            s["pool"], s["key_of"] = pool, _key_of_byte(d)
        else:
            s["pool"] = torch.empty((layers, 2, pages, hkv, PAGE, d), dtype=_type(case), device="cuda")
            _fill(s["pool"].flatten(0, 1), g, 0.0)
            s["key_of"] = torch.arange(PAGE, device="cuda")
        s["host"] = [np.array(x, np.int32) for x in (src, dst, keys)]
        s["src"], s["dst"] = src.cuda(), dst.cuda()
        s["keys"] = torch.tensor(keys, device="cuda")
        if own:
            from session_decode_step_dsb_gb300 import dsb
            if case["kind"] == "q4":
                s["pools"] = [dsb.kv_q4_pages(p, d) for p in s["pool"]]
            else:
                dt = dsb.DSB_F16 if case["kind"] == "f16" else dsb.DSB_BF16
                s["pools"] = [dsb.kv_pages(p[0], p[1], dt) for p in s["pool"]]
        return s
    lens, fresh = _lens(case)
    table, blocks, pages = _chains(case, seed, lens)
    n_tok, new, hq = sum(fresh), max(fresh), case["hq"]
    k = torch.empty((pages, hkv, PAGE, d), dtype=_type(case), device="cuda")
    v = torch.empty_like(k) if op != "select" else k
    _fill(k, g, 4.0)
    if op != "select":
        _fill(v, g, 0.0)
    s.update(k=k, v=v, lens=lens, fresh=fresh, table=table, new=new)
    s["q"] = torch.randn((n_tok, hq, d), device="cuda", generator=g)
    s["table_dev"] = table.cuda().long()
    # rows of the ragged queries in a padded [sequence, new token] grid
    f = torch.tensor(fresh)
    seqs = torch.repeat_interleave(torch.arange(len(lens)), f)
    s["slot"] = (seqs * new + torch.arange(n_tok) - (f.cumsum(0) - f)[seqs]).cuda()
    s["seqs"] = seqs.cuda()
    s["pos"] = torch.tensor(lens)[:, None] - f[:, None] + torch.arange(new)[None]  # of the grid
    s["pos"] = s["pos"].cuda()
    if op == "select":
        b = torch.stack([k.amin(2), k.amax(2)], 2)
        s["bounds"] = b  # of whole pages; those that the new tokens touch are made again by the call
        at = [(i, j) for i, (n, m) in enumerate(zip(lens, fresh)) for j in range((n - m) // PAGE, (n + PAGE - 1) // PAGE)
              if m]
        s["touched"] = torch.tensor([int(table[i, j]) for i, j in at], device="cuda")
        s["held"] = torch.tensor([min(PAGE, lens[i] - j * PAGE) for i, j in at], device="cuda")
    if op == "sparse":
        own_block = torch.div(s["pos"].reshape(-1)[s["slot"]], PAGE, rounding_mode="floor")[:, None]
        score = torch.rand((n_tok, hkv, max(blocks)), device="cuda", generator=g)
        j = torch.arange(max(blocks), device="cuda")
        score = torch.where(j == own_block[..., None], 2.0, torch.where(j > own_block[..., None], -math.inf, score))
        s["selected"] = _listed(score, case["n_select"])
    if own:
        from session_decode_step_dsb_gb300 import dsb
        dt = dsb.DSB_F16 if case["kind"] == "f16" else dsb.DSB_BF16
        s["kv"] = dsb.kv_pages(k, v if op != "select" else torch.empty_like(k), dt)
        # a call serves up to 8192 new tokens: larger batches go in several, sequence by sequence
        at, s["calls"] = 0, []
        while at < len(lens):
            end, rows = at, 0
            while end < len(lens) and rows + fresh[end] <= 8192:
                rows, end = rows + fresh[end], end + 1
            first = sum(fresh[:at])
            s["calls"].append((s["q"][first:first + rows], slice(first, first + rows),
                               dsb.PagedBatch(table[at:end].numpy(), blocks[at:end], [0] * (end - at), fresh[at:end],
                                              lens[at:end])))
            at = end
        s["batch"] = s["calls"][0][2]
        s["ws"] = dsb.Workspace(max(max(len(q) for q, _, _ in s["calls"]), 1), hq, d, max(lens))
    return s


# ------------------------------------------------------------- plain forms
def _listed(score, n):
    """Ascending indices of the n largest scores (ties: the lowest index), -1 behind the last; blocks that are not
    there score negative infinity."""
    n_blocks = score.shape[-1]
    order = torch.sort(score, dim=-1, descending=True, stable=True)
    index = torch.where(order.values > -math.inf, order.indices, n_blocks)[..., :n]
    if n > n_blocks:
        index = torch.cat([index, index.new_full(index.shape[:-1] + (n - n_blocks,), n_blocks)], -1)
    index = torch.sort(index, dim=-1).values
    return torch.where(index < n_blocks, index, -1).to(torch.int32)


def _run_copy(s):
    case = s["case"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        copy = dsb.kv_copy_pages_q4 if case["kind"] == "q4" else dsb.kv_copy_pages
        copy(s["pools"], *s["host"])
        return s["pool"]
    pool, src, dst = s["pool"], s["src"], s["dst"]
    taken = s["key_of"] < s["keys"][:, None]
    if case["kind"] == "q4":
        pool[:, dst] = torch.where(taken[:, None], pool[:, src], pool[:, dst])
    else:
        pool[:, :, dst] = torch.where(taken[:, None, :, None], pool[:, :, src], pool[:, :, dst])
    return pool


def _grid(s):
    """q as [sequence, kv head, new token, row of the group, d], zeros where a sequence brings fewer tokens."""
    case, new = s["case"], s["new"]
    n, hkv, hq, d = len(s["lens"]), case["hkv"], case["hq"], case["d"]
    q = torch.zeros((n * new, hq, d), device="cuda").index_copy_(0, s["slot"], s["q"])
    return q.view(n, new, hkv, hq // hkv, d).transpose(1, 2)


def _run_shared(s):
    if own:
        from session_decode_step_dsb_gb300 import dsb
        if len(s["calls"]) == 1:
            return dsb.attention_decode_shared(s["q"], s["kv"], s["batch"], s["ws"])
        out = torch.empty_like(s["q"])
        for q, rows, batch in s["calls"]:
            dsb.attention_decode_shared(q, s["kv"], batch, s["ws"], out=out[rows])
        return out
    case, new = s["case"], s["new"]
    n, hkv, hq, d = len(s["lens"]), case["hkv"], case["hq"], case["d"]
    key, val = (x[s["table_dev"]].transpose(1, 2).reshape(n, hkv, -1, d).float() for x in (s["k"], s["v"]))
    score = _grid(s).reshape(n, hkv, -1, d) @ key.transpose(-1, -2) / math.sqrt(d)
    score = score.view(n, hkv, new, hq // hkv, -1)
    hidden = torch.arange(key.shape[2], device="cuda") > s["pos"][..., None]
    score.masked_fill_(hidden[:, None, :, None], -math.inf)
    e = score.sub_(score.amax(-1, keepdim=True)).exp_()
    e /= e.sum(-1, keepdim=True)
    out = (e.view(n, hkv, -1, key.shape[2]) @ val).view(n, hkv, new, hq // hkv, d)
    return out.transpose(1, 2).reshape(n * new, hq, d)[s["slot"]]


def _pairwise(x):
    """Sum over the last dimension (a power of two), neighbours first, each sum rounded."""
    while x.shape[-1] > 1:
        x = x[..., 0::2] + x[..., 1::2]
    return x[..., 0]


def _scores(s):
    """Scores [sequence, new token, kv head, block]."""
    q = _grid(s)  # [n, hkv, new, group, d]
    group = q.shape[3]
    q = torch.nn.functional.pad(q, (0, 0, 0, (1 << (group - 1).bit_length()) - group)).transpose(-1, -2)
    a, b = _pairwise(q.clamp(min=0)), _pairwise(q.clamp(max=0))  # [n, hkv, new, d]
    bounds = s["bounds"][s["table_dev"]].float()  # [n, blocks, hkv, 2, d]
    lo, hi = (bounds[:, :, :, i].permute(0, 2, 1, 3)[:, None] for i in (0, 1))  # [n, 1, hkv, blocks, d]
    a, b = (x.transpose(1, 2)[:, :, :, None] for x in (a, b))
    return _pairwise(a * hi + b * lo)


def _run_select(s):
    case = s["case"]
    if own:
        from session_decode_step_dsb_gb300 import dsb
        dsb.kv_page_bounds(s["kv"], s["batch"], s["bounds"])
        got = dsb.kv_select_pages(s["q"], s["kv"], s["bounds"], s["batch"], case["n_select"], s["ws"],
                                  keep_first=case["first"], keep_last=case["last"])
        return {"bounds": s["bounds"], "selected": got}
    k = s["k"][s["touched"]]
    past = (torch.arange(PAGE, device="cuda") >= s["held"][:, None])[:, None, :, None]
    s["bounds"][s["touched"]] = torch.stack([k.masked_fill(past, math.inf).amin(2),
                                             k.masked_fill(past, -math.inf).amax(2)], 2)
    score = _scores(s)
    block = torch.arange(score.shape[-1], device="cuda")
    mine = torch.div(s["pos"], PAGE, rounding_mode="floor")[:, :, None, None]
    always = (block < case["first"]) | (block > mine - case["last"])
    score = score.masked_fill(always, math.inf).masked_fill(block > mine, -math.inf)
    return {"bounds": s["bounds"], "selected": _listed(score.flatten(0, 1)[s["slot"]], case["n_select"])}


def _run_sparse(s):
    if own:
        from session_decode_step_dsb_gb300 import dsb
        return dsb.attention_decode_selected(s["q"], s["kv"], s["batch"], s["selected"], s["ws"])
    case = s["case"]
    hkv, hq, d = case["hkv"], case["hq"], case["d"]
    sel = s["selected"].long()  # [token, hkv, n_select]
    page = s["table_dev"][s["seqs"][:, None, None], sel.clamp(min=0)]
    head = torch.arange(hkv, device="cuda")[:, None]
    key, val = (x[page, head].float().flatten(2, 3) for x in (s["k"], s["v"]))  # [token, hkv, keys, d]
    at = (sel[..., None] * PAGE + torch.arange(PAGE, device="cuda")).flatten(2)
    hidden = (at > s["pos"].reshape(-1)[s["slot"]][:, None, None]) | (sel < 0).repeat_interleave(PAGE, 2)
    q = s["q"].view(-1, hkv, hq // hkv, d)
    score = (q @ key.transpose(-1, -2) / math.sqrt(d)).masked_fill(hidden[:, :, None], -math.inf)
    e = torch.exp(score - score.amax(-1, keepdim=True))
    return (e / e.sum(-1, keepdim=True) @ val).view(-1, hq, d)


def run(state):
    return {"copy": _run_copy, "shared": _run_shared, "select": _run_select, "sparse": _run_sparse}[
        state["case"]["op"]](state)


# ------------------------------------------------ the definition in 64 bits
def _exact_copy(s):
    out = s["pool"].clone()
    src, dst, keys = (x.tolist() for x in s["host"])
    d = s["case"]["d"]
    for a, b, n in zip(src, dst, keys):
        if s["case"]["kind"] != "q4":
            out[:, :, b, :, :n] = s["pool"][:, :, a, :, :n]
            continue
        x, y, half = s["pool"][:, a], out[:, b], PAGE * d // 2
        y[..., :n * d // 2] = x[..., :n * d // 2]
        for z in (half, 2 * half + 4 * PAGE):
            y[..., z:z + 4 * n] = x[..., z:z + 4 * n]
        v = half + 4 * PAGE
        y[..., v:v + n // 2 * d] = x[..., v:v + n // 2 * d]
        if n % 2:  # the first key of a pair: two bytes of every four
            for i in (0, 1):
                last = slice(v + n // 2 * d + i, v + n // 2 * d + d, 4)
                y[..., last] = x[..., last]
    return out if s["case"]["kind"] == "q4" else out.double()


def exact(case, seed):
    s = prepare(case, seed)
    d, hkv = case["d"], case["hkv"]
    if case["op"] == "copy":
        return _exact_copy(s) if s["pool"].numel() < 1 << 29 else None
    group, row = case["hq"] // hkv, 0
    if case["op"] == "select":
        bounds = s["bounds"].double()
        for length, new, pages in zip(s["lens"], s["fresh"], s["table"].tolist()):
            for i in range((length - new) // PAGE, (length - 1) // PAGE + 1) if new else ():
                held = s["k"][pages[i], :, :length - i * PAGE].double()
                bounds[pages[i]] = torch.stack([held.min(1)[0], held.max(1)[0]], 1)
        return {"bounds": bounds, "selected": None}
    cost = sum(n * f for n, f in zip(s["lens"], s["fresh"])) * case["hq"] * d
    if case["op"] == "shared" and cost > 1.2e12:
        return None
    out = torch.zeros_like(s["q"], dtype=torch.float64)
    for length, new, pages in zip(s["lens"], s["fresh"], s["table"]):
        n = (length + PAGE - 1) // PAGE
        for h in range(hkv if new else 0):
            rows = s["q"][row:row + new, h * group:(h + 1) * group].double()
            if case["op"] == "shared":
                p = pages[:n].long().cuda()
                key, val = (x[p, h].double().flatten(0, 1) for x in (s["k"], s["v"]))
                logit = torch.einsum("jgd,kd->jgk", rows, key) / d ** 0.5
                at = torch.arange(n * PAGE, device="cuda")
                limit = torch.arange(length - new, length, device="cuda")[:, None, None]
                w = torch.softmax(logit.masked_fill_(at > limit, -math.inf), -1)
                out[row:row + new, h * group:(h + 1) * group] = torch.einsum("jgk,kd->jgd", w, val)
                continue
            for j in range(new):
                blocks = s["selected"][row + j, h]
                blocks = blocks[blocks >= 0].cpu().long()
                p = pages[blocks].long().cuda()
                at = (blocks[:, None] * PAGE + torch.arange(PAGE)).flatten().cuda()
                see = at <= length - new + j
                key, val = (x[p, h].double().flatten(0, 1)[see] for x in (s["k"], s["v"]))
                w = torch.softmax(rows[j] @ key.T / d ** 0.5, -1)
                out[row + j, h * group:(h + 1) * group] = w @ val
        row += new
    return out
