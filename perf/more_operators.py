"""Workloads of what lies between a layer's products besides plain attention: norms with the residual's addition, rotary
positions (alone, and on the way into the paged cache), attention of sequences that share a long prefix, and sampling.

``own`` false: the plain torch forms, in 32 bits (angles, and what decides between tokens, in 64).  ``own`` true:
``rms_norm``, ``Rotary``, ``KVCache.append_rotated``, ``KVCache.attend_shared`` and ``sample`` of
``bit_weight_only_packed_amd``.
"""
from __future__ import annotations

import math

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
_HEADS = dict(q_heads=40, kv_heads=8, head_dim=128)  # the 5120-wide q and 1024-wide k, v projections of the 27B-class shapes


# ------------------------------------------------------------------------------------------------- cases

def listed():
    rope = dict(base=10000.0, interleaved=False, scaling="none", factor=1.0, original=4096)
    return [
        # one request's decode step: the residual stream of 5120, latency
        dict(name="norm_step", op="norm", dtype="f16", rows=1, n=5120, residual=True, quant="none", group=0),
        # a whole prompt
        dict(name="norm_prompt", op="norm", dtype="bf16", rows=8191, n=5120, residual=True, quant="none", group=0),
        # a prompt's down projection input in 8 bits, a scale for each 128
        dict(name="norm_codes", op="norm", dtype="f16", rows=2047, n=17408, residual=False, quant="e4m3", group=128),
        # a whole prompt's q rows
        dict(name="rotate_prompt", op="rotate", dtype="f16", rows=8191, heads=40, head_dim=128, far=8191,
             **dict(rope, dim=128, interleaved=True)),
        # a chunk far along a long context, a quarter of wide heads rotated
        dict(name="rotate_far", op="rotate", dtype="bf16", rows=1021, heads=16, head_dim=256, far=1 << 20,
             **dict(rope, dim=64, base=500000.0, scaling="yarn", factor=32.0, original=32768)),
        # one new token of each of 64 requests, one slot idle
        dict(name="append_step", op="append", dtype="bf16", page=16, batch=64, rows_min=1, rows_max=1, len_min=5,
             len_max=9000, idle=1, **_HEADS, **dict(rope, dim=128)),
        # ragged prompts together, positions scaled for a longer context
        dict(name="append_prompts", op="append", dtype="f16", page=32, batch=9, rows_min=63, rows_max=3001, len_min=63,
             len_max=9001, idle=0, **_HEADS, **dict(rope, dim=128, scaling="linear", factor=4.0)),
        # eight answers to one prompt, early
        dict(name="share_step", op="share", dtype="f16", page=16, answers="8", prefix="2048", own_min=1, own_max=300,
             rows_min=1, rows_max=1, window=0, sinks=0, idle=0, **_HEADS),
        # sixty-four answers behind one long context, one slot idle
        dict(name="share_long", op="share", dtype="bf16", page=64, answers="64", prefix="32768", own_min=9, own_max=1500,
             rows_min=1, rows_max=1, window=0, sinks=0, idle=1, **_HEADS),
        # drafts of the answers to two prompts verified at once, wide heads
        dict(name="share_verify", op="share", dtype="bf16", page=32, answers="11,6", prefix="8192,4096", own_min=9,
             own_max=700, rows_min=2, rows_max=5, window=0, sinks=0, idle=0, q_heads=16, kv_heads=2, head_dim=256),
        # one request's next token from a large vocabulary
        dict(name="sample_one", op="sample", dtype="f16", rows=1, vocab=131071, mix="both"),
        # a serving batch, every request with settings of its own
        dict(name="sample_batch", op="sample", dtype="bf16", rows=128, vocab=100003, mix="any"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rotate", "append", "share", "share", "sample"])
    dtype = rng.choice(["f16", "bf16"])
    hd, kvh, g = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 5, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8])
    heads = dict(q_heads=kvh * g, kv_heads=kvh, head_dim=hd)
    rope = dict(dim=rng.choice([hd, hd, hd // 2, hd // 4]), base=rng.choice([10000.0, 500000.0, 1e6]),
                interleaved=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]), factor=1.0,
                original=rng.choice([2048, 4096, 32768]))
    if rope["scaling"] != "none":
        rope["factor"] = rng.choice([2.0, 4.0, 10.5, 32.0])
    if op == "norm":
        n = _log(rng, 64, 17408)
        n = n if rng.random() < 0.5 else -(-n // 8) * 8
        rows = _log(rng, 1, min(8191, (8191 * 5120) // n))
        return dict(op=op, dtype=dtype, rows=rows, n=n, residual=rng.random() < 0.7,
                    quant=rng.choice(["none", "none", "int8", "e4m3"]), group=rng.choice([0, 32, 64, 128]))
    if op == "rotate":
        h = rng.choice([1, 3, 8, 16, 40])
        return dict(op=op, dtype=dtype, rows=_log(rng, 1, (8191 * 5120) // (h * hd)), heads=h, head_dim=hd,
                    far=_log(rng, 64, 1 << 20), **rope)
    if op == "append":
        batch = _log(rng, 1, 64)
        rows = _log(rng, 1, max(2, (9000 * 5120) // (batch * max(5120, kvh * g * hd))))
        return dict(op=op, dtype=dtype, page=rng.choice([16, 32, 64, 128, 256]), batch=batch,
                    rows_min=max(1, rows // rng.choice([1, 7])), rows_max=rows, len_min=rows,
                    len_max=rows + _log(rng, 1, 8000), idle=rng.choice([0, 1]) if batch > 1 else 0, **heads, **rope)
    if op == "share":
        page = rng.choice([16, 32, 64, 128, 256])
        answers = [_log(rng, 2, 64) for _ in range(rng.choice([1, 1, 2, 3]))]
        rows = rng.choice([1, 1, rng.randint(2, 8)])
        cost = sum(answers) * rows * kvh * g * hd
        far = max(256, min(32768, (64 * 5120 * 32768) // cost, (32768 * 1024) // (kvh * hd * len(answers))))
        prefix = [max(page, _log(rng, 128, far) // page * page) for _ in answers]
        hi = _log(rng, 8, max(16, min(1500, (64 * 1500 * 1024) // (sum(answers) * kvh * hd))))
        window = rng.choice([0, 0, _log(rng, 64, 16384)])
        return dict(op=op, dtype=dtype, page=page, answers=",".join(map(str, answers)),
                    prefix=",".join(map(str, prefix)), own_min=max(1, hi // rng.choice([1, 3, 40])), own_max=hi,
                    rows_min=max(1, rows // rng.choice([1, 3])), rows_max=rows, window=window,
                    sinks=rng.choice([0, 4, 37]) if window else 0, idle=rng.choice([0, 1]), **heads)
    vocab = _log(rng, 1000, 131071)
    return dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), rows=_log(rng, 1, max(2, min(256, (128 * 100003) // vocab))),
                vocab=vocab, mix=rng.choice(["none", "greedy", "k", "p", "min", "both", "any", "any"]))


def _ladder(lo, hi, n):
    """n whole numbers from lo to hi, evenly spaced in their logarithm."""
    if n == 1:
        return [hi]
    return [int(round(lo * (hi / lo) ** (i / (n - 1)))) for i in range(n)]


def _append_entries(c):
    lens, rows = _ladder(c["len_min"], c["len_max"], c["batch"]), _ladder(c["rows_min"], c["rows_max"], c["batch"])
    rows = [min(r, n) for r, n in zip(rows, lens)]
    return [0 if i < c["idle"] else n for i, n in enumerate(lens)], rows


def _numbers(text):
    """A number for each group."""
    return [int(x) for x in text.split(",")]


def _share_entries(c):
    """Each group's (prefix, lengths, rows); an idle slot, length 0, is the first group's last entry."""
    out = []
    for i, (a, p) in enumerate(zip(_numbers(c["answers"]), _numbers(c["prefix"]))):
        rows = _ladder(c["rows_min"], c["rows_max"], a)
        lens = [p + max(x, r) for x, r in zip(_ladder(c["own_min"], c["own_max"], a), rows)]
        if i == 0 and c["idle"]:
            lens[-1] = 0
        out.append((p, lens, rows))
    return out


def work(case):
    c = case
    if c["op"] == "norm":
        el, n = c["rows"] * c["n"], 1 if c["quant"] != "none" else 2
        scales = 0 if n == 2 else 4 * c["rows"] * (-(-c["n"] // c["group"]) if c["group"] else 1)
        return {"bytes": el * (2 + (4 if c["residual"] else 0) + n) + 2 * c["n"] + scales, "flops": 6 * el}
    if c["op"] == "rotate":
        return {"bytes": 4 * c["rows"] * c["heads"] * c["head_dim"] + 4 * c["rows"], "flops": 3 * c["rows"] * c["heads"] * c["dim"]}
    if c["op"] == "append":
        lens, rows = _append_entries(c)
        n = sum(rows)
        return {"bytes": 4 * n * (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"],
                "flops": 3 * n * (c["q_heads"] + c["kv_heads"]) * c["dim"]}
    if c["op"] == "share":
        toks = pairs = n = 0
        for p, lens, rows in _share_entries(c):
            lo = p  # the oldest shared token that some row sees, past the sinks
            for length, r in zip(lens, rows):
                n += r
                if not length:
                    continue
                for pos in range(length - r, length):
                    first = max(0, pos - c["window"] + 1) if c["window"] else 0
                    pairs += pos + 1 - first + min(c["sinks"], first)
                first = max(0, length - r - c["window"] + 1) if c["window"] else 0
                lo = min(lo, first)
                toks += length - max(p, first)
            toks += p - lo + min(c["sinks"], lo)
        return {"bytes": 4 * toks * c["kv_heads"] * c["head_dim"] + 4 * n * c["q_heads"] * c["head_dim"],
                "flops": 4 * pairs * c["q_heads"] * c["head_dim"]}
    size = 4 if c["dtype"] == "f32" else 2
    return {"bytes": c["rows"] * (c["vocab"] * size + 20), "flops": 4 * c["rows"] * c["vocab"]}


# ------------------------------------------------------------------------------------------------- inputs

def _gen(seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(shape, dtype, g, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()



def _inputs(case, seed):
    """Everything a pass works on, from the case and the seed alone."""
    c, g, hg = case, _gen(seed), _gen(seed, "cpu")
    dt = _DT[c["dtype"]]
    if c["op"] == "norm":
        st = dict(x=_randn((c["rows"], c["n"]), dt, g, 0.7), weight=(1 + 0.1 * _randn((c["n"],), torch.float32, g)).to(dt))
        if c["residual"]:
            st["start"] = _randn((c["rows"], c["n"]), dt, g, 3.0)
            st["residual"] = torch.empty_like(st["start"])
        return dict(st, case=c)
    if c["op"] == "rotate":
        return dict(case=c, x=_randn((c["rows"], c["heads"], c["head_dim"]), dt, g),
                    positions=torch.randint(0, c["far"], (c["rows"],), generator=hg, dtype=torch.int32).cuda())
    if c["op"] == "sample":
        n, v = c["rows"], c["vocab"]
        x = _randn((n, v), torch.float32, g, 2.2)
        likely = torch.randint(0, v, (n, 24), generator=hg).cuda()  # a few tokens stand out, as a trained model's do
        x.scatter_add_(1, likely, torch.rand((n, 24), generator=hg).cuda() * 9)
        i = torch.arange(n)
        pick = {"none": i * 0, "greedy": i * 0 + 5, "k": i * 0 + 1, "p": i * 0 + 2, "min": i * 0 + 3, "both": i * 0 + 4,
                "any": (i * 7 + 1) % 6}[c["mix"]]
        few = torch.tensor([50, 1, 7, 200, 1000, 20])[i % 6]
        share = torch.tensor([0.95, 0.5, 0.9, 0.99, 0.1, 0.8])[i % 6]
        heat = torch.tensor([0.8, 1.0, 0.6, 1.3, 0.3])[i % 5]
        off = torch.zeros(n)
        return dict(case=c, logits=x.to(dt), u=torch.rand((n,), generator=hg).cuda(),
                    temperature=torch.where(pick == 5, off, heat).cuda(),
                    top_k=torch.where((pick == 1) | (pick == 4), few, 0).int().cuda(),
                    top_p=torch.where((pick == 2) | (pick == 4), share, 1.0).cuda(),
                    min_p=torch.where(pick == 3, 0.05, off).cuda())
    page = c["page"]
    if c["op"] == "append":
        lens, rows = _append_entries(c)
        need = [-(-x // page) for x in lens]
        pages, width = sum(need) + 8, max(need) + 1
        order = torch.randperm(pages, generator=hg).int()
        tables, at = torch.full((len(lens), width), -1, dtype=torch.int32), 0
        for j, k in enumerate(need):
            tables[j, :k] = order[at:at + k]
            at += k
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[order[:at].long()] = 1
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        qkv = _randn((starts[-1], c["q_heads"] + 2 * c["kv_heads"], c["head_dim"]), dt, g)
        q, k, v = qkv.split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)  # columns of the stacked q|k|v rows
        return dict(case=c, q=q, k=k, v=v, pool=_randn((pages, 1, 2, c["kv_heads"], page, c["head_dim"]), dt, g),
                    tables=tables.cuda(), lens=_ints(lens), refs=refs.cuda(), row_start=_ints(starts), max_rows=max(rows))
    groups = _share_entries(c)
    shared = [p // page for p, _, _ in groups]
    need = [[max(0, -(-n // page) - s) for n in lens] for (_, lens, _), s in zip(groups, shared)]
    pages = sum(shared) + sum(map(sum, need)) + 8
    width = max(s + max(k) for s, k in zip(shared, need)) + 1
    order = torch.randperm(pages, generator=hg).int()
    lens, rows = [n for _, x, _ in groups for n in x], [r for _, _, x in groups for r in x]
    tables, refs = torch.full((len(lens), width), -1, dtype=torch.int32), torch.zeros(pages, dtype=torch.int32)
    at = j = 0
    for (_, some, _), s, k in zip(groups, shared, need):
        common = order[at:at + s]
        at += s
        for length, own_pages in zip(some, k):
            if length:
                tables[j, :s] = common
                tables[j, s:s + own_pages] = order[at:at + own_pages]
                refs[common.long()] += 1
                refs[order[at:at + own_pages].long()] = 1
                at += own_pages
            j += 1
    starts = [0]
    for r in rows:
        starts.append(starts[-1] + r)
    begins = [0]
    for a in _numbers(c["answers"]):
        begins.append(begins[-1] + a)
    return dict(case=c, q=_randn((starts[-1], c["q_heads"], c["head_dim"]), dt, g, 1.5),
                pool=_randn((pages, 1, 2, c["kv_heads"], page, c["head_dim"]), dt, g), tables=tables.cuda(),
                lens=_ints(lens), refs=refs.cuda(), row_start=_ints(starts), groups=_ints(begins), max_rows=max(rows),
                host=(groups, starts))


def prepare(case, seed):
    st = _inputs(case, seed)
    c = case
    if own:
        import bit_weight_only_packed_amd as Q
        if "pool" in st:
            st["kv"] = Q.KVCache.of(st["pool"], st["tables"], st["lens"], st["refs"])
        if "dim" in c:
            st["rotary"] = Q.Rotary(c["dim"], c["base"], interleaved=c["interleaved"], scaling=c["scaling"],
                                    factor=c["factor"], original=c["original"])
    elif "dim" in c:
        st["freqs"], st["size"] = _frequencies(c)
    return st


# ------------------------------------------------------------------------------------------------- passes

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm(state)
    if op == "rotate":
        if own:
            return state["rotary"].rotate(state["x"], state["positions"])
        return _rotated(state, state["x"], state["positions"]).to(state["x"].dtype)
    if op == "append":
        if own:
            q = state["kv"].append_rotated(state["q"], state["k"], state["v"], state["rotary"],
                                           row_start=state["row_start"], max_rows=state["max_rows"])
        else:
            q = _append_plain(state)
        return {"q": q, "pool": state["pool"]}
    if op == "share":
        c = state["case"]
        if own:
            return state["kv"].attend_shared(state["q"], groups=state["groups"], row_start=state["row_start"],
                                             max_rows=state["max_rows"], window=c["window"], sinks=c["sinks"])
        return _share_plain(state)
    if own:
        from bit_weight_only_packed_amd import sample
        tokens, probs = sample(state["logits"], state["u"], temperature=state["temperature"], top_k=state["top_k"],
                               top_p=state["top_p"], min_p=state["min_p"], probs=True)
        return {"tokens": tokens, "probs": probs}
    return _sample_plain(state)


def _norm(st):
    c, x = st["case"], st["x"]
    res = st.get("residual")
    if res is not None:
        res.copy_(st["start"])  # each pass begins with the same residual stream
    top = {"none": 0.0, "int8": 127.0, "e4m3": 448.0}[c["quant"]]
    if own:
        from bit_weight_only_packed_amd import rms_norm
        if not top:
            y = rms_norm(x, st["weight"], residual=res, eps=1e-6)
        else:
            kind = torch.int8 if c["quant"] == "int8" else torch.float8_e4m3fn
            codes, scales = rms_norm(x, st["weight"], residual=res, eps=1e-6, quant=kind, group=c["group"])
            y = _values(codes, scales, c, x.dtype)
    else:
        h = x
        if res is not None:
            res.add_(x)
            h = res
        f = h.float()
        y = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * st["weight"].float()
        if not top:
            y = y.to(x.dtype)
        else:
            g = c["group"] or c["n"]
            full = torch.nn.functional.pad(y, (0, -c["n"] % g)).view(c["rows"], -1, g)
            scales = full.abs().amax(-1) / top  # of all-zero groups 0
            codes = (full / torch.where(scales > 0, scales, 1.0)[..., None]).view(c["rows"], -1)[:, :c["n"]]
            codes = codes.round().to(torch.int8) if c["quant"] == "int8" else codes.to(torch.float8_e4m3fn)
            y = _values(codes, scales, c, x.dtype)
    return {"y": y} if res is None else {"y": y, "residual": res}


def _values(codes, scales, c, dtype):
    """What the codes stand for (a code is exact in either type; the product is rounded once)."""
    n, g = c["n"], c["group"] or c["n"]
    part = codes.to(dtype)
    if n % g:
        part = torch.nn.functional.pad(part, (0, -n % g))
    part = part.view(c["rows"], -1, g)
    return torch.mul(part, scales[..., None], out=torch.empty_like(part)).view(c["rows"], -1)[:, :n]


def _frequencies(c):
    """Radians per position of each pair, in 64 bits, and the factor on rotated values."""
    d, base = c["dim"], c["base"]
    j = torch.arange(d // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk":
        base = base * c["factor"] ** (d / (d - 2))
    f = base ** (-2 * j / d)
    if c["scaling"] == "linear":
        f = f / c["factor"]
    if c["scaling"] != "yarn":
        return f, 1.0
    turn = [d * math.log(c["original"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (32, 1)]
    lo, hi = max(math.floor(turn[0]), 0), min(math.ceil(turn[1]), d - 1)
    slow = ((j - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - slow) + f / c["factor"] * slow, 0.1 * math.log(c["factor"]) + 1


def _rotated(st, x, positions):
    """x [rows][heads][head_dim] rotated, in 32 bits."""
    c = st["case"]
    a = positions.double()[:, None] * st["freqs"]
    cos, sin = (a.cos() * st["size"]).float()[:, None], (a.sin() * st["size"]).float()[:, None]
    d, f = c["dim"], x.float()
    out = f.clone()
    if c["interleaved"]:
        u, v = f[..., 0:d:2], f[..., 1:d:2]
        out[..., 0:d:2], out[..., 1:d:2] = u * cos - v * sin, u * sin + v * cos
    else:
        u, v = f[..., :d // 2], f[..., d // 2:d]
        out[..., :d // 2], out[..., d // 2:d] = u * cos - v * sin, u * sin + v * cos
    return out


def _append_plain(st):
    c = st["case"]
    t = torch.arange(st["k"].shape[0], device="cuda")
    j = torch.searchsorted(st["row_start"], t, right=True) - 1  # the entry of each row
    pos = st["lens"][j].long() - st["row_start"][j + 1] + t
    live = pos >= 0
    q = (_rotated(st, st["q"], pos) * live[:, None, None]).to(st["q"].dtype)
    k = _rotated(st, st["k"], pos).to(st["k"].dtype)
    spot = pos.clamp(min=0)
    pg, sl = st["tables"][j, spot // c["page"]].long(), spot % c["page"]
    st["pool"][pg[live], 0, 0, :, sl[live]] = k[live]
    st["pool"][pg[live], 0, 1, :, sl[live]] = st["v"][live]
    return q


def _share_plain(st):
    """Each group's shared tokens against all of its rows at once, the sequences' own tokens padded to the longest."""
    c, page = st["case"], st["case"]["page"]
    d, kvh = c["head_dim"], c["kv_heads"]
    g = c["q_heads"] // kvh
    groups, starts = st["host"]
    out = torch.zeros_like(st["q"])
    j0 = 0
    for p, lens, rows in groups:
        n, r = len(lens), max(rows)
        i = torch.arange(r, device="cuda")
        first = torch.tensor(starts[j0:j0 + n], device="cuda")[:, None]
        count = torch.tensor(rows, device="cuda")[:, None]
        length = torch.tensor(lens, device="cuda")[:, None]
        some = i < count
        at = torch.where(some, first + i, 0)                                    # [n][r] rows of the call
        pos = torch.where(some, length - count + i, -1)
        q = st["q"][at].float().view(n, r, kvh, g, d).permute(2, 0, 1, 3, 4)   # [kvh][n][r][g][d]
        tables = st["tables"][j0:j0 + n].long()
        live = max(range(n), key=lambda x: lens[x])

        def scores(k, tok):                                                     # k [kvh][n or 1][tokens][d]
            flat = q.reshape(kvh, k.shape[1], -1, d)
            s = torch.matmul(flat, k.transpose(2, 3).contiguous()) * (d ** -0.5)
            seen = tok[..., None, None, :] <= pos[..., None, None]              # [n][r][1][tokens]
            if c["window"]:
                seen = seen & ((tok[..., None, None, :] > pos[..., None, None] - c["window"]) | (tok[..., None, None, :] < c["sinks"]))
            return s.view(kvh, n, r, g, -1).masked_fill_(~seen, float("-inf"))

        ids = tables[live, :p // page]
        kv = st["pool"][ids, 0].float().permute(1, 2, 0, 3, 4).reshape(2, kvh, 1, p, d)  # the shared tokens
        s0 = scores(kv[0], torch.arange(p, device="cuda")[None, None])
        m = max(1, max(lens) - p)
        tok = p + torch.arange(m, device="cuda")
        ids = tables[:, (tok // page).clamp(max=tables.shape[1] - 1)].clamp(min=0)
        mine = st["pool"][ids, 0, :, :, tok % page].float().permute(2, 3, 0, 1, 4).contiguous()  # [2][kvh][n][m][d]
        s1 = scores(mine[0], tok[None, None])
        top = torch.maximum(s0.amax(-1, keepdim=True), s1.amax(-1, keepdim=True)).clamp(min=-3e38)
        s0, s1 = s0.sub_(top).exp_(), s1.sub_(top).exp_()
        total = s0.sum(-1, keepdim=True) + s1.sum(-1, keepdim=True)
        o = torch.matmul(s0.view(kvh, 1, -1, p), kv[1]).view(kvh, n, r, g, d)
        o = o + torch.matmul(s1.reshape(kvh, n, r * g, m), mine[1]).view(kvh, n, r, g, d)
        o = torch.where(total > 0, o / total, 0.0).permute(1, 2, 0, 3, 4).reshape(n, r, kvh * g, d)
        out[at[some]] = o[some].to(out.dtype)
        j0 += n
    return out


def _sample_plain(st):
    x = st["logits"].float()
    v = x.shape[1]
    v0, index = x.sort(dim=-1, descending=True, stable=True)  # equal logits in the order of their tokens
    heat = st["temperature"].double()[:, None]
    greedy = heat <= 0
    w = torch.exp((v0.double() - v0[:, :1].double()) / torch.where(greedy, 1.0, heat))
    rank = torch.arange(v, device="cuda")[None]
    k = torch.where(st["top_k"] > 0, st["top_k"], v)[:, None]
    w = w * (rank < torch.where(greedy, 1, k))
    running = w.cumsum(-1)
    before = torch.cat([torch.zeros_like(running[:, :1]), running[:, :-1]], 1)
    p = st["top_p"].double()[:, None]
    w = w * ((before < p * running[:, -1:]) | (p >= 1)) * (w >= st["min_p"].double()[:, None])
    w = torch.empty_like(w).scatter_(1, index, w)
    running = w.cumsum(-1)
    total = running[:, -1:]
    token = torch.searchsorted(running, st["u"].double()[:, None] * total, right=True)
    return {"tokens": token[:, 0].int(), "probs": (w.gather(1, token) / total)[:, 0].float()}


# ------------------------------------------------------------------------------------------------- exact

def _turned(c, x, positions):
    """x rotated, in 64 bits: pairs as complex numbers, times the unit of their angle."""
    d, half = c["dim"], c["dim"] // 2
    base = c["base"] * (c["factor"] ** (d / (d - 2)) if c["scaling"] == "ntk" else 1.0)
    freq = []
    size = 1.0
    for j in range(half):
        f = math.exp(-math.log(base) * j / half)
        if c["scaling"] == "linear":
            f /= c["factor"]
        elif c["scaling"] == "yarn":
            edge = [half * math.log(c["original"] / (2 * math.pi * r)) / math.log(base) for r in (32.0, 1.0)]
            a, b = max(0, math.floor(edge[0])), min(d - 1, math.ceil(edge[1]))
            t = min(1.0, max(0.0, (j - a) / max(b - a, 0.001)))
            f *= t / c["factor"] + 1.0 - t
            size = 1.0 + math.log(c["factor"]) / 10
        freq.append(f)
    ang = torch.outer(positions.double(), torch.tensor(freq, dtype=torch.float64, device="cuda"))
    unit = torch.polar(torch.full_like(ang, size), ang)[:, None]
    y = x.double()
    head = y[..., :d]
    pair = head.reshape(*head.shape[:-1], half, 2) if c["interleaved"] else head.reshape(*head.shape[:-1], 2, half).transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * unit)
    z = z.reshape(head.shape) if c["interleaved"] else z.transpose(-1, -2).reshape(head.shape)
    return torch.cat([z, y[..., d:]], -1)


def exact(case, seed):
    """What a pass returns, from the definitions in 64 bits (a sum with the residual is rounded, as it is stored, before
    its norm is taken; of sampling the probabilities of the tokens)."""
    c, st = case, _inputs(case, seed)
    if c["op"] == "norm":
        h = st["x"].double()
        if c["residual"]:
            h = (h + st["start"].double()).to(st["x"].dtype).double()
        y = h * st["weight"].double() / torch.sqrt((h * h).sum(-1, keepdim=True) / c["n"] + 1e-6)
        if c["quant"] != "none":
            top, g = (127.0 if c["quant"] == "int8" else 448.0), c["group"] or c["n"]
            for a in range(0, c["n"], g):
                part = y[:, a:a + g]
                s = part.abs().amax(-1, keepdim=True) / top
                z = part / torch.where(s > 0, s, torch.ones_like(s))
                if c["quant"] == "int8":
                    z = torch.round(z)
                else:  # three bits behind the leading one, steps of 2^-9 at least
                    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
                    z = torch.round(z / step) * step
                y[:, a:a + g] = z * s
        return {"y": y, "residual": h} if c["residual"] else {"y": y}
    if c["op"] == "rotate":
        return _turned(c, st["x"], st["positions"])
    if c["op"] == "append":
        lens, rows = _append_entries(c)
        pool, q = st["pool"].double(), torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        at = 0
        for j, (n, r) in enumerate(zip(lens, rows)):
            if n:
                pos = torch.arange(n - r, n, device="cuda")
                q[at:at + r] = _turned(c, st["q"][at:at + r], pos)
                where = st["tables"][j][torch.div(pos, c["page"], rounding_mode="floor")].long()
                pool[where, 0, 0, :, pos % c["page"]] = _turned(c, st["k"][at:at + r], pos)
                pool[where, 0, 1, :, pos % c["page"]] = st["v"][at:at + r].double()
            at += r
        return {"q": q, "pool": pool}
    if c["op"] == "share":
        return _attended(c, st)
    probs = torch.empty(c["rows"], dtype=torch.float64, device="cuda")
    for i in range(c["rows"]):
        x, t = st["logits"][i].double(), float(st["temperature"][i])
        if t <= 0:
            probs[i] = 1.0
            continue
        order = torch.argsort(x, dim=0, descending=True, stable=True)
        k = int(st["top_k"][i])
        order = order[:k] if k > 0 else order
        w = torch.softmax(x[order] / t, 0)
        run_ = torch.cumsum(w, 0)
        p = float(st["top_p"][i])
        if p < 1:
            order = order[:int((run_ < p * run_[-1]).sum()) + 1]
        w = torch.exp((x[order] - x[order[0]]) / t)
        order, w = order[w >= float(st["min_p"][i])], w[w >= float(st["min_p"][i])]
        by = torch.argsort(order)
        run_ = torch.cumsum(w[by], 0)
        probs[i] = w[by][int((run_ <= float(st["u"][i]) * run_[-1]).sum())] / run_[-1]
    return {"tokens": None, "probs": probs}


def _attended(c, st):
    """Every sequence by itself."""
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    group, page = c["q_heads"] // c["kv_heads"], c["page"]
    lens = [n for _, x, _ in st["host"][0] for n in x]
    starts = st["host"][1]
    for j, n in enumerate(lens):
        if not n:
            continue
        a, b = starts[j], starts[j + 1]
        tok, pos = torch.arange(n, device="cuda"), torch.arange(n - (b - a), n, device="cuda")[:, None]
        hidden = tok > pos
        if c["window"]:
            hidden |= (tok <= pos - c["window"]) & (tok >= c["sinks"])
        where = st["tables"][j][torch.div(tok, page, rounding_mode="floor")].long()
        for h in range(c["kv_heads"]):
            key, val = st["pool"][where, 0, 0, h, tok % page].double(), st["pool"][where, 0, 1, h, tok % page].double()
            q = st["q"][a:b, h * group:(h + 1) * group].double().transpose(0, 1)
            s = (q @ key.T / math.sqrt(c["head_dim"])).masked_fill(hidden, -math.inf)
            out[a:b, h * group:(h + 1) * group] = (torch.softmax(s, -1) @ val).transpose(0, 1)
    return out
