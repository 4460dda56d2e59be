"""Workloads of the paged key-value cache: attention over it, appending to it, and its page operations.

A cache is a pool ``[pages][layers][2][kv_heads][page_size][head_dim]`` (0 keys, 1 values), page tables
``tables[slot][i]`` (page of tokens ``[i * page_size, (i + 1) * page_size)``, -1 for none), lengths ``lens[slot]`` and
reference counts ``refs[page]``.

``own`` false: the plain torch forms, in 32 bits.  ``own`` true: ``bit_weight_only_packed_amd.KVCache``.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------------------------------- cases

def listed():
    # heads 40 / 8 x 128: the 5120-wide q and 1024-wide k, v projections of the 27B-class layer shapes
    h = dict(q_heads=40, kv_heads=8, head_dim=128)
    return [
        # one request early in its answer: latency
        dict(name="step_one", op="attend", dtype="f16", page=16, batch=1, rows_min=1, rows_max=1, len_min=1025,
             len_max=1025, window=0, sinks=0, idle=0, **h),
        # one request at a long context (128k): the cache's bytes
        dict(name="step_long", op="attend", dtype="f16", page=16, batch=1, rows_min=1, rows_max=1, len_min=131071,
             len_max=131071, window=0, sinks=0, idle=0, **h),
        # a serving batch at every stage of its requests, one slot idle
        dict(name="step_ragged", op="attend", dtype="bf16", page=64, batch=48, rows_min=1, rows_max=1, len_min=3,
             len_max=24577, window=0, sinks=0, idle=1, **h),
        # a batch of streams with a sliding window and sinks, wide heads
        dict(name="step_window", op="attend", dtype="bf16", page=32, batch=32, rows_min=1, rows_max=1, len_min=900,
             len_max=20011, window=4096, sinks=4, idle=0, q_heads=16, kv_heads=2, head_dim=256),
        # eight drafted tokens verified at once, two requests
        dict(name="verify_8", op="attend", dtype="f16", page=16, batch=2, rows_min=8, rows_max=8, len_min=4100,
             len_max=12290, window=0, sinks=0, idle=0, **h),
        # a chunk of a long prompt under a sliding window with sinks
        dict(name="chunk_window", op="attend", dtype="bf16", page=16, batch=1, rows_min=4096, rows_max=4096,
             len_min=16411, len_max=16411, window=2048, sinks=8, idle=0, **h),
        # one whole prompt
        dict(name="prompt_full", op="attend", dtype="f16", page=16, batch=1, rows_min=8191, rows_max=8191, len_min=8191,
             len_max=8191, window=0, sinks=0, idle=0, **h),
        # short prompts of many lengths together, some behind a shared history, one head per kv head
        dict(name="prompts_ragged", op="attend", dtype="f16", page=32, batch=16, rows_min=1, rows_max=1901, len_min=40,
             len_max=2500, window=512, sinks=4, idle=0, q_heads=16, kv_heads=16, head_dim=64),
        # one new token of each of 64 requests into its page, k and v as columns of the stacked q|k|v rows
        dict(name="append_step", op="append", dtype="bf16", page=16, batch=64, rows_min=1, rows_max=1, len_min=5,
             len_max=1500, window=0, sinks=0, idle=0, **h),
        # a whole prompt's keys and values
        dict(name="append_prompt", op="append", dtype="f16", page=16, batch=1, rows_min=16383, rows_max=16383,
             len_min=16383, len_max=16383, window=0, sinks=0, idle=0, **h),
        # sixteen requests forked three times each, then one more token everywhere: shared tails are copied
        dict(name="fork_grow", op="fork", dtype="f16", page=16, layers=4, pages=1500, sources=16, forks=3,
             len_min=301, len_max=909, kv_heads=8, head_dim=128),
        # a fragmented pool after requests have ended: freed, then moved together
        dict(name="compact_pool", op="compact", dtype="f16", page=16, layers=16, pages=1600, live=900, moved=350,
             ended=100, slots=60, kv_heads=8, head_dim=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "step", "verify", "prompt", "prompt", "append", "pages"])
    dtype = rng.choice(["f16", "bf16"])
    page = rng.choice([16, 32, 64, 128, 256])
    hd = rng.choice([64, 128, 256])
    kvh = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 2, 3, 4, 5, 7, 8])
    c = dict(dtype=dtype, page=page, q_heads=kvh * g, kv_heads=kvh, head_dim=hd, idle=0, window=0, sinks=0)
    windowed = rng.random() < 0.5
    if kind in ("step", "verify"):
        rows = 1 if kind == "step" else rng.randint(2, 32)
        batch = _log(rng, 1, 64)
        # at most the largest listed step's bytes
        cap = max(64, min(131071, (1 << 27) // (batch * kvh * hd)))
        hi = _log(rng, 64, cap)
        c.update(op="attend", batch=batch, rows_min=rows, rows_max=rows, len_min=max(1, hi // rng.choice([1, 3, 40])),
                 len_max=hi, idle=rng.choice([0, 1]) if batch > 1 else 0)
    elif kind == "prompt":
        batch = _log(rng, 1, 12)
        budget = 6.5e11 / (4.0 * hd * kvh * g * batch)          # visible pairs of one entry
        length = _log(rng, 33, min(16000, max(64, int(math.sqrt(2 * budget)))))
        rows = max(1, _log(rng, max(1, length // 8), length))
        c.update(op="attend", batch=batch, rows_min=max(1, rows // rng.choice([1, 5])), rows_max=rows,
                 len_min=max(1, length // rng.choice([1, 3])), len_max=length)
    elif kind == "append":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, 16383 // batch))
        c.update(op="append", batch=batch, rows_min=max(1, rows // rng.choice([1, 7])), rows_max=rows, len_min=rows,
                 len_max=rows + _log(rng, 1, 2000))
    else:
        layers = rng.choice([1, 3, 8])
        page = rng.choice([16, 32])
        pages = _log(rng, 200, 1500)
        base = dict(dtype=dtype, page=page, layers=layers, pages=pages, kv_heads=kvh, head_dim=rng.choice([64, 128]))
        if rng.random() < 0.5:
            n = rng.randint(1, 12)
            f = rng.randint(1, 4)
            top = max(2, (pages - 2 * n * (f + 1)) // n * page)
            hi = rng.randint(2, min(top, 60 * page))
            return dict(base, op="fork", sources=n, forks=f, len_min=max(1, hi // 3), len_max=hi)
        live = rng.randint(pages // 4, (3 * pages) // 4)
        ended = rng.randint(1, live // 4)
        moved = rng.randint(1, min(live, pages - live) - 1)
        return dict(base, op="compact", live=live, moved=moved, ended=ended, slots=rng.randint(4, 40))
    if windowed and c["op"] == "attend":
        c.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 37]))
    return c


def _ladder(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _entries(c):
    """Lengths and new rows of the batch's entries; the idle ones have length 0 (and rows that see nothing)."""
    n = c["batch"]
    lens = _ladder(c["len_min"], c["len_max"], n)
    rows = _ladder(c["rows_min"], c["rows_max"], n)
    if c["rows_min"] != c["rows_max"]:
        rows = [min(r, length) for r, length in zip(rows, lens)]
    for i in range(c["idle"]):
        lens[i] = 0
    return lens, rows


def _seen(c, length, rows):
    """(row, token) pairs that are visible, and tokens that some row sees."""
    w, s = c["window"], c["sinks"]
    pairs = 0
    p0 = length - rows
    if not w:
        lo = max(0, p0)
        pairs = sum(range(lo + 1, length + 1)) if length - lo < 64 else (length - lo) * (lo + 1 + length) // 2
        return pairs, length
    for p in range(max(0, p0), length):
        first = max(0, p - w + 1)
        pairs += p + 1 - first + min(s, first)
    first = max(0, max(0, p0) - w + 1)
    return pairs, (length - first) + min(s, first) if length else 0


def _rows_of_pages(c):
    """Tokens of each forked source: never a whole number of pages, so that a shared tail has to be copied."""
    return [n + 1 if n % c["page"] == 0 else n for n in _ladder(c["len_min"], c["len_max"], c["sources"])]


def work(case):
    c = case
    if c["op"] in ("attend", "append"):
        lens, rows = _entries(c)
        tok = c["kv_heads"] * c["head_dim"] * 2 * 2
        if c["op"] == "append":
            return {"bytes": 2 * tok * sum(rows), "flops": 0}
        pairs = toks = 0
        for n, r in zip(lens, rows):
            a, b = _seen(c, n, r)
            pairs, toks = pairs + a, toks + b
        return {"bytes": tok * toks + 2 * 2 * sum(rows) * c["q_heads"] * c["head_dim"],
                "flops": 4 * pairs * c["q_heads"] * c["head_dim"]}
    page_bytes = c["layers"] * 2 * c["kv_heads"] * c["page"] * c["head_dim"] * 2
    if c["op"] == "fork":
        n = sum(-(-x // c["page"]) for x in _rows_of_pages(c))
        return {"bytes": 2 * page_bytes * c["sources"] * c["forks"] + 4 * c["pages"] * 2 + 4 * n * (1 + c["forks"]),
                "flops": 0}
    return {"bytes": 2 * page_bytes * c["moved"] + 4 * c["pages"] * 2 + 2 * 4 * (c["live"] + c["ended"]), "flops": 0}


# ------------------------------------------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(shape, dtype, g, scale=1.0):
    x = torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)
    return x


def _inputs(case, seed):
    """Everything a pass works on, from the case and the seed alone."""
    c, g, hg = case, _gen(seed), _gen(seed, "cpu")
    dt = _DT[c["dtype"]]
    page, kvh, d = c["page"], c["kv_heads"], c["head_dim"]
    if c["op"] in ("attend", "append"):
        lens, rows = _entries(c)
        n = len(lens)
        need = [-(-x // page) for x in lens]
        pages = sum(need) + 8
        width = max(need) + 1
        order = torch.randperm(pages, generator=hg).tolist()     # a pool in use: pages in no order
        slots = torch.randperm(n, generator=hg).tolist()         # entry j of the batch is slot slots[j]
        tables = torch.full((n, width), -1, dtype=torch.int32)
        lens_s = torch.zeros(n, dtype=torch.int32)
        at = 0
        for j, s in enumerate(slots):
            tables[s, :need[j]] = torch.tensor(order[at:at + need[j]], dtype=torch.int32)
            at += need[j]
            lens_s[s] = lens[j]
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[order[:at]] = 1
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        st = dict(case=c, pool=_randn((pages, 1, 2, kvh, page, d), dt, g), tables=tables.cuda(), lens=lens_s.cuda(),
                  refs=refs.cuda(), seqs=torch.tensor(slots, dtype=torch.int32).cuda(),
                  row_start=torch.tensor(starts, dtype=torch.int32).cuda(), host=(lens, rows, slots, starts))
        if c["op"] == "attend":
            st["q"] = _randn((starts[-1], c["q_heads"], d), dt, g, 1.5)
        else:
            qkv = _randn((starts[-1], c["q_heads"] + 2 * kvh, d), dt, g)
            st["k"], st["v"] = qkv[:, c["q_heads"]:c["q_heads"] + kvh], qkv[:, c["q_heads"] + kvh:]
        return st
    pages = c["pages"]
    pool = _randn((pages, c["layers"], 2, kvh, page, d), dt, g)
    order = torch.randperm(pages, generator=hg)
    refs = torch.zeros(pages, dtype=torch.int32)
    if c["op"] == "fork":
        lens = _rows_of_pages(c)
        n, f = c["sources"], c["forks"]
        slots = n * (1 + f)
        place = torch.randperm(slots, generator=hg).tolist()
        width = max(-(-x // page) for x in lens) + 1
        tables = torch.full((slots, width), -1, dtype=torch.int32)
        lens_s = torch.zeros(slots, dtype=torch.int32)
        at = 0
        for i, length in enumerate(lens):
            k = -(-length // page)
            tables[place[i], :k] = order[at:at + k].int()
            refs[order[at:at + k]] = 1
            lens_s[place[i]] = length
            at += k
        src = [place[i] for i in range(n) for _ in range(f)]
        extra = dict(src=torch.tensor(src, dtype=torch.int32).cuda(),
                     dst=torch.tensor(place[n:], dtype=torch.int32).cuda(),
                     n_new=torch.ones(slots, dtype=torch.int32).cuda())
    else:
        # after the ended requests are freed, `live` pages stay in use and exactly `moved` of them lie past `live`
        live, moved, ended = c["live"], c["moved"], c["ended"]
        low, high = order[order < live], order[order >= live]
        keep = torch.cat([low[:live - moved], high[:moved]])
        keep = keep[torch.randperm(live, generator=hg)]
        rest = torch.cat([low[live - moved:], high[moved:]])
        rest = rest[torch.randperm(rest.numel(), generator=hg)][:ended]
        m = min(c["slots"], live)
        cuts = [i * live // m for i in range(m + 1)]
        e = min(max(1, c["slots"] // 8), ended)
        ecuts = [i * ended // e for i in range(e + 1)]
        parts = [keep[a:b] for a, b in zip(cuts, cuts[1:])] + [rest[a:b] for a, b in zip(ecuts, ecuts[1:])]
        place = torch.randperm(m + e, generator=hg).tolist()
        width = max(p.numel() for p in parts)
        tables = torch.full((m + e, width), -1, dtype=torch.int32)
        lens_s = torch.zeros(m + e, dtype=torch.int32)
        for s, p in zip(place, parts):
            tables[s, :p.numel()] = p.int()
            refs[p] = 1
            lens_s[s] = p.numel() * page - s % page
        extra = dict(gone=torch.tensor(place[m:], dtype=torch.int32).cuda())
    state = dict(case=c, pool=pool, tables=tables.cuda(), lens=lens_s.cuda(), refs=refs.cuda(), **extra)
    state["start"] = tuple(state[k].clone() for k in ("tables", "lens", "refs"))
    return state


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        from bit_weight_only_packed_amd import KVCache
        st["kv"] = KVCache.of(st["pool"], st["tables"], st["lens"], st["refs"])
    return st


# ------------------------------------------------------------------------------------------------- passes

def run(state):
    c = state["case"]
    if c["op"] == "attend":
        return _attend_own(state) if own else _attend_plain(state)
    if c["op"] == "append":
        if own:
            state["kv"].append(state["k"], state["v"], seqs=state["seqs"], row_start=state["row_start"],
                               max_rows=max(state["host"][1]))
            return state["pool"]
        return _append_plain(state)
    # the state that the operation starts from: each pass begins with the same tables, lengths and counts
    for k, t in zip(("tables", "lens", "refs"), state["start"]):
        state[k].copy_(t)
    if own:
        kv = state["kv"]
        if c["op"] == "fork":
            kv.fork(state["src"], state["dst"])
            kv.extend(state["n_new"])
        else:
            kv.trim(state["gone"])
            kv.compact()
    elif c["op"] == "fork":
        _fork_plain(state)
        _extend_plain(state)
    else:
        _free_plain(state)
        _compact_plain(state)
    return {k: state[k] for k in ("pool", "tables", "lens", "refs")}


def _attend_own(st):
    c = st["case"]
    return st["kv"].attend(st["q"], seqs=st["seqs"], row_start=st["row_start"], max_rows=max(st["host"][1]),
                           scale=c["head_dim"] ** -0.5, window=c["window"], sinks=c["sinks"])


def _attend_plain(st):
    c = st["case"]
    d, kvh, page = c["head_dim"], c["kv_heads"], c["page"]
    g = c["q_heads"] // kvh
    lens, rows, slots, starts = st["host"]
    out = torch.zeros_like(st["q"])
    for j, (n, r) in enumerate(zip(lens, rows)):
        if n == 0 or r == 0:
            continue
        ids = st["tables"][slots[j], :-(-n // page)]
        p0 = n - r
        skip = max(0, -p0)                                        # rows before the sequence's start see nothing
        first = max(0, p0 + skip - c["window"] + 1) if c["window"] else 0
        pos = torch.arange(n, device="cuda")
        if first > c["sinks"]:                                    # leave out the tokens that no row sees
            pos = torch.cat([pos[:c["sinks"]], pos[first:]])
        pg, sl = ids[pos // page].long(), pos % page
        kv = st["pool"][pg, 0, :, :, sl].float()                  # [tokens][2][kvh][d]
        k = kv[:, 0].permute(1, 2, 0).contiguous()                # [kvh][d][tokens]
        v = kv[:, 1].permute(1, 0, 2).contiguous()                # [kvh][tokens][d]
        step = max(1, (1 << 28) // (kvh * g * pos.numel()))
        for a in range(skip, r, step):
            b = min(r, a + step)
            q = st["q"][starts[j] + a:starts[j] + b].float().reshape(b - a, kvh, g, d)
            q = q.permute(1, 2, 0, 3).reshape(kvh, g * (b - a), d).contiguous()
            s = torch.matmul(q, k) * (d ** -0.5)
            at = torch.arange(p0 + a, p0 + b, device="cuda")[:, None]
            hide = pos[None] > at
            if c["window"]:
                hide |= (pos[None] <= at - c["window"]) & (pos[None] >= c["sinks"])
            s = s.view(kvh, g, b - a, -1).masked_fill_(hide, float("-inf")).view(kvh, g * (b - a), -1)
            s -= s.amax(-1, keepdim=True)
            s.exp_()
            s /= s.sum(-1, keepdim=True)
            o = torch.matmul(s, v).view(kvh, g, b - a, d).permute(2, 0, 1, 3).reshape(b - a, kvh * g, d)
            out[starts[j] + a:starts[j] + b] = o.to(out.dtype)
    return out


def _append_plain(st):
    c = st["case"]
    t = torch.arange(st["k"].shape[0], device="cuda")
    j = torch.searchsorted(st["row_start"], t, right=True) - 1    # the entry of each row
    s = st["seqs"][j].long()
    pos = st["lens"][s].long() - st["row_start"][j + 1] + t
    pg = st["tables"][s, pos // c["page"]].long()
    sl = pos % c["page"]
    st["pool"][pg, 0, 0, :, sl] = st["k"]
    st["pool"][pg, 0, 1, :, sl] = st["v"]
    return st["pool"]


def _pages_used(lens, page):
    return (lens + page - 1) // page


def _fork_plain(st):
    src, dst = st["src"].long(), st["dst"].long()
    rows = st["tables"][src]
    st["tables"][dst] = rows
    st["lens"][dst] = st["lens"][src]
    held = rows[rows >= 0].long()
    st["refs"].index_add_(0, held, torch.ones_like(held, dtype=torch.int32))


def _extend_plain(st):
    page, tables, lens, refs = st["case"]["page"], st["tables"], st["lens"].long(), st["refs"]
    dev = tables.device
    slot = torch.arange(lens.numel(), device=dev)
    n_new = st["n_new"].long()
    used, grown = _pages_used(lens, page), _pages_used(lens + n_new, page)
    tail = tables[slot, (used - 1).clamp(min=0)].long().clamp(min=0)
    shared = (n_new > 0) & (lens % page != 0) & (refs[tail] > 1)
    holders = torch.zeros(refs.numel(), dtype=torch.int64, device=dev).index_add_(0, tail, shared.long())
    lowest = torch.full((refs.numel(),), lens.numel(), dtype=torch.int64, device=dev)
    lowest.scatter_reduce_(0, tail, torch.where(shared, slot, lens.numel()), "amin")
    copy = shared & ~((holders[tail] == refs[tail]) & (lowest[tail] == slot))
    take = grown - used + copy
    begin = take.cumsum(0) - take
    free = (refs == 0).nonzero()[:, 0]
    i = torch.arange(tables.shape[1], device=dev)[None]
    fresh = (i >= used[:, None]) & (i < grown[:, None])
    which = (begin + copy)[:, None] + i - used[:, None]
    from_, to = tail[copy], free[begin[copy]]
    st["pool"][to] = st["pool"][from_]
    refs.index_add_(0, from_, torch.full_like(from_, -1, dtype=torch.int32))
    refs[free[:int(take.sum())]] = 1
    tables[fresh] = free[which[fresh]].int()
    tables[slot[copy], used[copy] - 1] = to.int()
    st["lens"] += st["n_new"]


def _free_plain(st):
    gone = st["gone"].long()
    rows = st["tables"][gone]
    held = rows[rows >= 0].long()
    st["refs"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    st["tables"][gone] = -1
    st["lens"][gone] = 0


def _compact_plain(st):
    refs, tables = st["refs"], st["tables"]
    live = refs > 0
    n = int(live.sum())
    ids = torch.arange(refs.numel(), device=refs.device)
    from_, to = ids[live & (ids >= n)], ids[~live & (ids < n)]
    st["pool"][to] = st["pool"][from_]
    place = ids.clone()
    place[from_] = to
    tables.copy_(torch.where(tables >= 0, place[tables.long().clamp(min=0)].int(), tables))
    refs[to] = refs[from_]
    refs[from_] = 0


# ------------------------------------------------------------------------------------------------- exact

def exact(case, seed):
    """Attention from its definition in 64 bits; the other operators move values and have no computed ones."""
    if case["op"] != "attend":
        return None
    c, st = case, _inputs(case, seed)
    lens, rows, slots, starts = st["host"]
    d, page = c["head_dim"], c["page"]
    group = c["q_heads"] // c["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    for j, (n, r) in enumerate(zip(lens, rows)):
        if n == 0:
            continue
        tok = torch.arange(n, device="cuda")
        where = st["tables"][slots[j]][torch.div(tok, page, rounding_mode="floor")].long()
        span = max(1, (1 << 27) // n)
        for h in range(c["kv_heads"]):
            key = st["pool"][where, 0, 0, h, tok % page].double()
            val = st["pool"][where, 0, 1, h, tok % page].double()
            for a in range(0, r, span):
                pos = torch.arange(n - r + a, n - r + min(r, a + span), device="cuda")
                ok = tok[None, :] <= pos[:, None]
                if c["window"]:
                    ok &= (tok[None, :] > pos[:, None] - c["window"]) | (tok[None, :] < c["sinks"])
                some = ok.any(1)
                for x in range(h * group, (h + 1) * group):
                    q = st["q"][starts[j] + a:starts[j] + a + pos.numel(), x].double()
                    s = (q @ key.T) / math.sqrt(d)
                    s = torch.where(ok, s, torch.full_like(s, -math.inf))
                    norm = torch.where(some, torch.logsumexp(s, 1), torch.zeros_like(some, dtype=torch.float64))
                    out[starts[j] + a:starts[j] + a + pos.numel(), x] = torch.exp(s - norm[:, None]) @ val
    return out
