"""Cases that measure the operators of shared pages in the paged cache: the fork
of requests, the compaction of the pool, finding common prefixes, attention
that computes a common prefix once for all, and rotary positions of several axes.

With ``own`` false, ``run`` computes each operator in its plain form from
elementary torch operations; with ``own`` true it makes the calls a user of
``decode_serving_gb300.paged`` makes.  Sizes follow this repository's
workloads (8 kv-heads, 4 query heads per kv-head, head width 128, contexts up
to 65536, 16-token pages).

Layouts: K and V pages [layers][num_pages][kv_heads][page][head_dim]; block
tables [requests][max_pages]; ``shares`` [num_pages] counts the requests that
hold a page beyond the first.  The new tokens of a step are ragged: request r
owns rows first[r] .. first[r+1].
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def _fork(name, groups, width, beams, layers, kv_heads, head_dim, page, ctx_lo, ctx_hi, tail, dtype, ragged):
    return {"name": name, "op": "fork", "groups": groups, "width": width, "beams": beams, "layers": layers,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi,
            "tail": tail, "dtype": dtype, "ragged": ragged}


def _compact(name, requests, layers, kv_heads, head_dim, page, ctx_lo, ctx_hi, spare, dtype, ragged):
    return {"name": name, "op": "compact", "requests": requests, "layers": layers, "kv_heads": kv_heads,
            "head_dim": head_dim, "page": page, "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "spare": spare,
            "dtype": dtype, "ragged": ragged}


def _find(name, groups, width, alone, page, ctx_lo, ctx_hi, tail, new_hi, least, ragged):
    return {"name": name, "op": "find", "groups": groups, "width": width, "alone": alone, "page": page,
            "ctx_lo": ctx_lo, "ctx_hi": ctx_hi, "tail": tail, "new_lo": 0, "new_hi": new_hi, "least": least,
            "ragged": ragged}


def _attend(name, groups, width, alone, kv_heads, q_per_kv, head_dim, page, ctx_lo, ctx_hi, tail, new_lo,
            new_hi, tree, cap, window, slopes, dtype, ragged):
    return {"name": name, "op": "attend", "groups": groups, "width": width, "alone": alone,
            "kv_heads": kv_heads, "q_per_kv": q_per_kv, "head_dim": head_dim, "page": page, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "tail": tail, "new_lo": new_lo, "new_hi": new_hi, "tree": tree, "cap": cap,
            "window": window, "slopes": slopes, "dtype": dtype, "ragged": ragged}


def _rotary(name, tokens, axes, dealt, kv_heads, q_per_kv, head_dim, rot, offset, interleaved, far, page,
            step_rows, dtype):
    return {"name": name, "op": "rotary", "tokens": tokens, "axes": axes, "dealt": dealt,
            "kv_heads": kv_heads, "q_per_kv": q_per_kv, "head_dim": head_dim, "rot": rot, "offset": offset,
            "interleaved": interleaved, "far": far, "page": page, "step_rows": step_rows, "dtype": dtype}


def listed():
    return [
        # Eight samples of one prompt in a draft model's only layer: latency.
        _fork("fork samples", 1, 8, False, 1, 8, 128, 16, 1000, 1000, 0, "bf16", 1),
        # Beam search, four beams of each of 64 requests: every step, some beams replace others.
        _fork("fork beams", 64, 4, True, 16, 8, 128, 16, 60, 500, 40, "bf16", 2),
        # Few long contexts in large pages, 16 samples each.
        _fork("fork long", 6, 16, False, 8, 4, 64, 64, 1000, 32768, 0, "fp16", 3),
        # A small pool of one layer: latency.
        _compact("compact small", 4, 1, 8, 128, 16, 17, 300, 0.5, "bf16", 4),
        # A pool after a busy hour, a third of it free, through 8 layers.
        _compact("compact pool", 64, 8, 8, 128, 16, 5, 1500, 0.33, "bf16", 5),
        # One step of 8 samples of a prompt: latency.
        _find("find samples", 1, 8, 0, 16, 4096, 4096, 100, 1, 64, 6),
        # A large batch: 40 system prompts with 12 requests each, others alone, long contexts.
        _find("find batch", 40, 12, 29, 16, 64, 65536, 2000, 4, 256, 7),
        # Four samples on one kv-head, one token each: latency.
        _attend("attend samples", 1, 4, 0, 1, 4, 128, 16, 1024, 1024, 40, 1, 1, False, 0.0, 0, False, "bf16", 8),
        # 64 requests behind one long document, one token each.
        _attend("attend document", 1, 64, 0, 8, 4, 128, 16, 32768, 32768, 500, 1, 1, False, 0.0, 0, False,
                "bf16", 9),
        # Draft trees in four ragged groups, a few requests alone (the largest).
        _attend("attend trees", 4, 16, 5, 8, 4, 128, 16, 4096, 32768, 1000, 1, 16, True, 0.0, 0, False,
                "bf16", 10),
        # One decode step's rows with positions of three axes, the pairs dealt out in turn.
        _rotary("rotary axes decode", 8, 3, True, 8, 4, 128, 128, 0, False, 32768, 16, 0, "bf16"),
        # The patches of a long video prompt: time, height and width in sections of each head.
        _rotary("rotary axes video", 16381, 3, False, 8, 4, 128, 128, 0, False, 4096, 16, 0, "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fork", "compact", "find", "attend", "attend", "rotary"))
    ragged = rng.randrange(1 << 20)
    dtype = rng.choice(("bf16", "fp16"))
    page = rng.choice((1, 4, 8, 16, 32, 64))
    if op == "fork":
        h, d, groups, width = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 256)), _log(rng, 1, 64), rng.randint(2, 16)
        layers = _log(rng, 1, 16)
        # 2 GB of pages, tables of 2 million entries
        most = max(2, min((1 << 31) // (h * d * layers * 4 * groups), page * 2000000 // (groups * width)))
        c = _fork("", groups, width, rng.random() < 0.5, layers, h, d, page, rng.choice((1, 17)),
                  max(18, _log(rng, 2, min(32768, most))), rng.choice((0, 40)), dtype, ragged)
    elif op == "compact":
        h, d, n, layers = rng.choice((1, 2, 8)), rng.choice((64, 128, 256)), _log(rng, 1, 64), _log(rng, 1, 12)
        most = max(2, (1 << 31) // (h * d * layers * 4 * n))
        c = _compact("", n, layers, h, d, page, rng.choice((0, 5)), max(6, _log(rng, 2, min(8192, most))),
                     rng.uniform(0.05, 0.8), dtype, ragged)
    elif op == "find":
        groups, width, alone = _log(rng, 1, 64), rng.randint(2, 12), rng.choice((0, _log(rng, 1, 64)))
        most = max(130, min(65536, page * 2000000 // (groups * width + alone)))
        c = _find("", groups, width, alone, page, rng.choice((0, 64)), _log(rng, 65, most), _log(rng, 1, min(2000, most)),
                  rng.choice((1, _log(rng, 1, 64))), rng.choice((1, 64, 256)), ragged)
    elif op == "attend":
        groups, width, alone = _log(rng, 1, 6), rng.randint(2, 16), rng.choice((0, 0, _log(rng, 1, 8)))
        h, g, d = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 5, 8, 16)), rng.choice((64, 128, 256))
        tree = rng.random() < 0.5
        new = _log(rng, 1, 64) if tree else rng.choice((1, 1, _log(rng, 1, 300)))
        n = groups * width + alone
        most = min(65536, (64 * 8 * 128 * 33000) // (n * h * d), (1 << 31) // (n * h * g * new) + 1)
        c = _attend("", groups, width, alone, h, g, d, page, rng.choice((1, 64)), max(65, _log(rng, 2, max(3, most))),
                    _log(rng, 1, 1000), rng.choice((0, 1, new)), new, tree, rng.choice((0.0, 0.0, 50.0)),
                    rng.choice((0, 0, 0, _log(rng, 16, 8192))), rng.random() < 0.3, dtype, ragged)
    else:
        d = rng.choice((64, 128, 256))
        rot = rng.choice((d, d // 2, 48))
        h, g = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
        step = rng.choice((0, 0, 0, 1, 3))
        t = _log(rng, 1, min(16384, (16384 * 48 * 128) // (d * h * (g + 2))))
        t = max(1, t // step) * step if step else t
        c = _rotary("", t, rng.randint(2, 4), rng.random() < 0.5, h, g, d, rot, rng.choice((0, d - rot)),
                    rng.random() < 0.5, _log(rng, 64, 1 << 20), 1 if step else page, step, dtype)
    del c["name"]
    return c


# ------------------------------------------- what follows from a case's numbers

def _groups(case):
    """Of every request: its group (-1: alone), the tokens of its group's prompt, its own
    committed tokens behind them, its new tokens (int64 arrays, by group)."""
    r = random.Random(case["ragged"])
    groups, width, alone = case["groups"], case["width"], case.get("alone", 0)
    span = case["ctx_hi"] - case["ctx_lo"]
    prompt = [case["ctx_lo"] + round(span * r.random()) for _ in range(groups)]
    prompt[-1] = case["ctx_hi"]
    rows = []
    for a in range(groups):
        tail = r.randint(0, case["tail"])
        for _ in range(width):
            # the beams of a request are of one length; samples and users are not
            rows.append((a, prompt[a], tail if case["op"] == "fork" else r.randint(0, case["tail"])))
    for _ in range(alone):
        rows.append((-1, 0, case["ctx_lo"] + round(span * r.random()) + 1))
    new = [r.randint(case["new_lo"], case["new_hi"]) if "new_hi" in case else 0 for _ in rows]
    if "new_hi" in case:
        new[0] = case["new_hi"]
    group, pre, tail = (np.array(x, np.int64) for x in zip(*rows))
    return group, pre, tail, np.array(new, np.int64)


def _parents(case):
    """Which request each request becomes: samples all start again from their group's first
    request; of beams, about half are replaced by others of their group."""
    r = random.Random(case["ragged"] + 1)
    w = case["width"]
    out = []
    for i in range(case["groups"] * w):
        first = i - i % w
        stays = not case["beams"] or r.random() < 0.5
        out.append(first if not case["beams"] else i if stays else first + r.randrange(w))
    return np.array(out, np.int64)


def _copies(case, length, parent):
    """Requests that get a copy of their parent's partly filled page."""
    i = np.arange(len(parent))
    moved, part = parent != i, length % case["page"] > 0
    heir = np.full(len(parent), len(parent))
    np.minimum.at(heir, parent[moved], i[moved])
    goes = parent[parent] != parent
    return moved & part[parent] & ~(goes & (heir[parent] == i))


def _contexts(case):
    r = random.Random(case["ragged"])
    span = case["ctx_hi"] - case["ctx_lo"]
    ctx = [case["ctx_lo"] + round(span * r.random()) for _ in range(case["requests"])]
    ctx[-1] = case["ctx_hi"]
    return np.array(ctx, np.int64)


def _trees(new, seed):
    """Ancestor masks (own bit included) of random trees of up to 64 new tokens."""
    r = np.random.default_rng([seed, 11])
    n, most = len(new), int(max(1, new.max()))
    word = np.zeros((n, most), np.uint64)
    for i in range(most):
        bit = np.uint64(1 << i)
        parent = np.maximum(0, i - 1 - r.integers(0, 4, n))
        word[:, i] = bit if i == 0 else word[np.arange(n), parent] | bit
    first = np.concatenate([[0], np.cumsum(new)])
    req = np.repeat(np.arange(n), new)
    return word[req, np.arange(int(new.sum())) - first[req]].view(np.int64)


def work(case):
    op = case["op"]
    if op == "rotary":
        t, h, g, d = case["tokens"], case["kv_heads"], case["q_per_kv"], case["head_dim"]
        q_out = 4 if case["step_rows"] else 2
        return {"bytes": t * d * (h * g * (2 + q_out) + h * 8) + (4 + 4 * case["axes"]) * t,
                "flops": 6 * t * (case["rot"] // 2) * h * (g + 1)}
    page = case["page"]
    if op == "compact":
        held = int((-(-_contexts(case) // page)).sum())
        pool = _pool(case, held)
        moved = held * (pool - held) / pool                               # on the average
        row = case["layers"] * case["kv_heads"] * case["head_dim"] * page * 2 * 2
        return {"bytes": int(2 * moved * row) + 8 * held + 8 * pool, "flops": 0}
    group, pre, tail, new = _groups(case)
    if op == "fork":
        length, parent = pre + tail, _parents(case)
        copied = _copies(case, length, parent)
        rows = int((length[parent] % page)[copied].sum())
        entries = int((-(-length // page))[parent][parent != np.arange(len(parent))].sum())
        row = case["layers"] * case["kv_heads"] * case["head_dim"] * 2 * 2
        return {"bytes": 2 * rows * row + 8 * entries + 12 * len(parent), "flops": 0}
    if op == "find":
        full = np.where(new > 0, pre + tail, 0) // page
        shared = np.where((group >= 0) & (new > 0), pre // page, np.minimum(1, full))
        return {"bytes": 4 * int(shared.sum()) + 24 * len(pre) + 8 * int(new.sum()), "flops": 0}
    h, g, d, total = case["kv_heads"], case["q_per_kv"], case["head_dim"], int(new.sum())
    win = case["window"] or 1 << 40
    ctx = pre + tail
    pairs = new * np.minimum(ctx, win) + new * (new + 1) // 2
    # a prompt's keys once per group, as far as some row's window reaches
    keys = np.where(new > 0, np.minimum(tail, win) + new, 0).sum()
    for a in range(case["groups"]):
        of = (group == a) & (new > 0)
        if of.any():
            keys += min(pre[of][0], max(0, win - int(tail[of].min())))
    return {"bytes": int(keys) * h * d * 4 + total * h * g * (4 * d + 4), "flops": int(pairs.sum()) * h * g * 4 * d}


# ------------------------------------------------------------------ the inputs

def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _normal(seed, *shape, dtype):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _pool(case, held):
    return max(held + 3, int(round(held / (1 - case["spare"]))))


def _axes(case):
    """Axis of every pair: sections as even as they go, or dealt out in turn."""
    half, n = case["rot"] // 2, case["axes"]
    i = np.arange(half)
    return i % n if case["dealt"] else i * n // half


def _shared_tables(case, group, pre, length, new, r, room):
    """Tables in which the requests of a group hold the same full pages of their prompt;
    (tables, free stack, count, shares)."""
    page, n = case["page"], len(length)
    held = -(-(length + new) // page)
    common = np.where(group >= 0, pre // page, 0)
    first = np.array([int(np.argmax(group == a)) if a >= 0 else i for i, a in enumerate(group)])
    lead = first == np.arange(n)
    mine = np.where(lead, held, held - common)
    pool = int(mine.sum()) + room
    ids = r.permutation(pool)
    width = max(1, int(held.max()))
    x = np.arange(width)[None, :]
    fresh = (x < held[:, None]) & (lead[:, None] | (x >= common[:, None]))
    tables = np.zeros((n, width), np.int64)
    tables[fresh] = ids[:int(mine.sum())]
    tables = np.where(x < np.where(lead, 0, common)[:, None], tables[first], tables)
    shares = np.zeros(pool, np.int64)
    np.add.at(shares, tables[x < held[:, None]], 1)
    left = ids[int(mine.sum()):]
    free = np.zeros(pool, np.int64)
    free[:len(left)] = left
    return tables, free, len(left), np.maximum(shares - 1, 0)


def prepare(case, seed):
    """What a program has before the call: the cache, the step's rows, the plan's arrays."""
    s = {"case": case}
    op, page = case["op"], case["page"]
    if op == "rotary":
        _prepare_rotary(s, case, seed)
    elif op == "compact":
        ctx = _contexts(case)
        held = -(-ctx // page)
        pool, width = _pool(case, int(held.sum())), max(1, int(held.max()))
        r = np.random.default_rng([seed, 5])
        ids = r.permutation(pool)
        tables = np.zeros((len(ctx), width), np.int64)
        tables[np.arange(width)[None, :] < held[:, None]] = ids[:int(held.sum())]
        left = ids[int(held.sum()):]
        free = np.zeros(pool, np.int64)
        free[:len(left)] = left
        s["tables"], s["lens"], s["free"], s["count"] = _dev(tables), _dev(ctx), _dev(free), _dev([len(left)])
        s["shares"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        s["tables_out"], s["free_out"] = s["tables"].clone(), s["free"].clone()
        s["shares_out"], s["map"] = torch.zeros_like(s["shares"]), torch.zeros_like(s["shares"])
    else:
        group, pre, tail, new = _groups(case)
        r = np.random.default_rng([seed, 4])
        if op == "find":                                    # a batch in any order
            order = r.permutation(len(group))
            group, pre, tail, new = (x[order] for x in (group, pre, tail, new))
        elif op == "attend":
            order = np.random.default_rng([case["ragged"], 6]).permutation(len(group))
            group, pre, tail, new = (x[order] for x in (group, pre, tail, new))
        length = pre + tail
        # (a find's new tokens have their pages already; a fork may take a page for every request)
        tables, free, count, shares = _shared_tables(case, group, pre, length, new, r, len(length) + 3)
        s["tables"], s["lens"], s["free"], s["count"] = _dev(tables), _dev(length), _dev(free), _dev([count])
        s["shares"] = _dev(shares)
        s["total"], s["most"] = int(new.sum()), int(max(1, new.max()))
        s["first"] = _dev(np.concatenate([[0], np.cumsum(new)]))
        if op == "fork":
            s["parent"] = _dev(_parents(case))
        if op == "attend":
            h, g, d, dt = case["kv_heads"], case["q_per_kv"], case["head_dim"], DTYPES[case["dtype"]]
            s["mask"] = _dev(_trees(new, seed), torch.int64) if case["tree"] else None
            s["q"] = _normal(seed + 7, s["total"], h * g, d, dtype=dt)
            s["out"] = torch.empty_like(s["q"])
            s["lse"] = torch.empty(s["total"], h * g, dtype=torch.float32, device="cuda")
            s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, h * g + 1, device="cuda") / (h * g))
                           if case["slopes"] else None)
    if op == "find":
        s["k"] = s["v"] = torch.zeros(1, s["free"].numel(), 1, page, 8, dtype=torch.bfloat16, device="cuda")
    elif op != "rotary":
        shape = (case.get("layers", 1), s["free"].numel(), case["kv_heads"], page, case["head_dim"])
        s["k"] = _normal(seed, *shape, dtype=DTYPES[case["dtype"]])
        s["v"] = _normal(seed + (1 << 40), *shape, dtype=DTYPES[case["dtype"]])
    if own:
        from decode_serving_gb300 import paged
        s["cache"] = cache = paged.PagedCache(s["k"], s["v"], s["tables"], s["lens"], s["free"], s["count"],
                                              shares=s.get("shares"))
        if op == "rotary":
            s["freq"] = paged.rotary_frequencies(case["rot"], base=10000.0).cuda()
        if op == "fork":
            s["work"] = cache.fork_workspace()
        if op == "compact":
            s["work"] = cache.compact_workspace()
        if op in ("find", "attend"):
            s["prefixes"], s["work"] = cache.prefix_arrays(s["total"]), cache.prefix_workspace()
        if op == "attend":                                  # once per step, for all layers
            cache.find_prefixes(s["first"], s["prefixes"], s["work"])
            s["work"] = cache.attend_prefixes_workspace(case["q_per_kv"], s["most"], s["total"])
    return s


def _prepare_rotary(s, case, seed):
    dt, page = DTYPES[case["dtype"]], case["page"]
    t, h, g, d = case["tokens"], case["kv_heads"], case["q_per_kv"], case["head_dim"]
    r = np.random.default_rng([seed, 3])
    s["qkv"] = _normal(seed, t, (h * g + 2 * h) * d, dtype=dt)
    # the first axis runs on with the sequence, the others go over a picture's rows and columns
    start = r.integers(0, case["far"])
    pos = start + r.integers(0, 128, (case["axes"], t))
    pos[0] = start + np.arange(t) // 64
    s["pos"] = _dev(pos)
    pool = t if case["step_rows"] else -(-t // page) + 2
    s["slots"] = None if case["step_rows"] else _dev(r.permutation(pool * page)[:t])
    s["k"], s["v"] = (torch.zeros(1, pool, h, page, d, dtype=dt, device="cuda") for _ in "kv")
    half = case["rot"] // 2
    s["inv"] = torch.from_numpy(10000.0 ** (-np.arange(half, dtype=np.float64) / half)).cuda()
    s["axes"] = _dev(_axes(case))
    s["q_out"] = torch.empty(t, h * g, d, device="cuda", dtype=torch.float32 if case["step_rows"] else dt)
    s["tables"] = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    s["lens"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    s["free"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
    s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the passes

def run(s):
    op = s["case"]["op"]
    if own:
        return {"fork": _own_fork, "compact": _own_compact, "find": _own_find, "attend": _own_attend,
                "rotary": _own_rotary}[op](s)
    return {"fork": _plain_fork, "compact": _plain_compact, "find": _plain_find, "attend": _plain_attend,
            "rotary": _plain_rotary}[op](s)


def _cache_of(s):
    return {x: s[x] for x in ("k", "v", "tables", "lens", "free", "count", "shares")}


def _own_fork(s):
    s["cache"].fork(s["parent"], s["work"])
    return _cache_of(s)


def _own_compact(s):
    s["cache"].compact(s["map"], s["work"], tables_out=s["tables_out"], free_out=s["free_out"],
                       shares_out=s["shares_out"])
    return {"k": s["k"], "v": s["v"], "tables": s["tables_out"], "free": s["free_out"],
            "shares": s["shares_out"], "map": s["map"]}


def _own_find(s):
    p = s["prefixes"]
    s["cache"].find_prefixes(s["first"], p, s["work"], min_tokens=s["case"]["least"])
    return {"leader": p.leader, "shared": p.shared, "first": p.first, "token": p.token, "request": p.request}


def _own_attend(s):
    c = s["case"]
    s["cache"].attend_prefixes(s["q"], s["first"], s["prefixes"], s["out"], s["most"], s["work"], mask=s["mask"],
                               lse=s["lse"], softcap=c["cap"], window=c["window"], slopes=s["slopes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_rotary(s):
    c = s["case"]
    h, g, d = c["kv_heads"], c["q_per_kv"], c["head_dim"]
    q, k, v = s["qkv"].split((h * g * d, h * d, h * d), 1)
    s["cache"].rotary(q, k, v, s["pos"], s["slots"], s["freq"], s["q_out"], rot_offset=c["offset"],
                      interleaved=c["interleaved"], tokens_per_request=max(1, c["step_rows"]), axes=s["axes"])
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _plain_fork(s):
    page = s["case"]["page"]
    lens, parent, tables, free = (s[x].long() for x in ("lens", "parent", "tables", "free"))
    count, n = s["count"].long(), len(lens)
    i, x = torch.arange(n, device=lens.device), torch.arange(tables.shape[1], device=lens.device)[None, :]
    full, held = lens // page, (lens + page - 1) // page
    alive, q = parent >= 0, parent.clamp(min=0)
    stays = parent == i
    moved = alive & ~stays
    children = torch.zeros_like(lens).scatter_add_(0, q, moved.long())
    heir = torch.full_like(lens, n).scatter_reduce_(0, q, torch.where(moved, i, n), "amin")
    # partly filled pages: one request keeps the parent's, the others get a copy
    copied = moved & (held > full)[q] & ~(~stays[q] & (heir[q] == i))
    fresh = free[(count - copied.long().cumsum(0)).clamp(min=0)]
    spare = free[0]                       # a page that nobody holds stands in for requests without a copy
    src = torch.where(copied, tables[q, full[q].clamp(max=tables.shape[1] - 1)], spare)
    dst = torch.where(copied, fresh, spare)
    row = torch.arange(page, device=lens.device)[None, :]
    fill = (copied[:, None] & (row < (lens % page)[q][:, None]))[None, :, None, :, None]
    for a in (s["k"], s["v"]):
        a[:, dst] = torch.where(fill, a[:, src], a[:, dst])
    # holders: an old row counts once for each request that continues it
    times = stays.long() + children
    change = torch.where(x < full[:, None], times[:, None] - 1, -(times == 0).long()[:, None])
    change = torch.where(x < held[:, None], change, 0)
    flat = tables.flatten()
    holders = s["shares"].long().scatter_add(0, flat, change.flatten())
    gone = (times == 0)[:, None] & (x < held[:, None])
    last = torch.full_like(holders, -1).scatter_reduce_(0, flat, torch.where(gone, i[:, None], -1).flatten(), "amax")
    back = (gone & (holders < 0)[tables] & (last[tables] == i[:, None])).flatten()
    count = count - copied.long().sum()
    order = back.long().cumsum(0) - 1
    at = torch.where(back, count + back.sum() - 1 - order, len(free))
    free = torch.cat([free, free[:1]])
    free[at] = flat
    new = torch.where(moved[:, None] & (x < held[q][:, None]), tables[q], tables)
    new = torch.where(copied[:, None] & (x == full[q][:, None]), fresh[:, None], new)
    s["tables"].copy_(new)
    s["free"].copy_(free[:-1])
    s["count"].copy_(count + back.sum())
    s["shares"].copy_(holders.clamp(min=0))
    s["lens"].copy_(torch.where(alive, lens[q], 0))
    return _cache_of(s)


def _plain_compact(s):
    page = s["case"]["page"]
    lens, tables, free, count = (s[x].long() for x in ("lens", "tables", "free", "count"))
    pool = len(free)
    i = torch.arange(pool, device=lens.device)
    is_free = torch.zeros(pool + 1, dtype=torch.bool, device=lens.device)
    is_free[torch.where(i < count, free, pool)] = True
    is_free = is_free[:pool]
    live = pool - count
    hole, mover = is_free & (i < live), ~is_free & (i >= live)
    # the n-th hole is filled by the n-th page that moves; a page beyond all stands for none
    spot = torch.full((pool + 1,), pool, device=lens.device)
    spot[torch.where(hole, hole.long().cumsum(0) - 1, pool)] = i
    to = torch.where(mover, spot[(mover.long().cumsum(0) - 1).clamp(min=0)], torch.where(is_free, -1, i))
    # At most half of the pool moves; places in the list behind the last move repeat the first one
    # (with no move at all: a page onto itself).
    order = torch.argsort(~mover, stable=True)[:max(1, pool // 2)]
    keep, lead = mover[order], order[0]
    a = torch.where(keep, order, lead)
    b = torch.where(keep, to[order], torch.where(mover[lead], to[lead], lead))
    for pages in (s["k"], s["v"]):
        pages[:, b] = pages[:, a]
    x = torch.arange(tables.shape[1], device=lens.device)[None, :]
    held = x < ((lens + page - 1) // page)[:, None]
    shares = torch.zeros(pool + 1, dtype=torch.long, device=lens.device)
    shares[torch.where(is_free, pool, to)] = s["shares"].long()
    free = torch.where(i < count, pool - 1 - i, free)
    s["tables_out"].copy_(torch.where(held, to[tables], tables))
    s["free_out"].copy_(free)
    s["shares_out"].copy_(shares[:pool])
    s["map"].copy_(to)
    return {"k": s["k"], "v": s["v"], "tables": s["tables_out"], "free": s["free_out"],
            "shares": s["shares_out"], "map": s["map"]}


def _plain_find(s):
    c = s["case"]
    page = c["page"]
    lens, tables, first = (s[x].long() for x in ("lens", "tables", "first"))
    n, pool = len(lens), s["free"].numel()
    i, x = torch.arange(n, device=lens.device), torch.arange(tables.shape[1], device=lens.device)[None, :]
    new = first[1:] - first[:-1]
    full = torch.where(new > 0, lens // page, 0)
    has = full > 0
    page0 = torch.where(has, tables[:, 0], pool)
    lowest = torch.full((pool + 1,), n, device=lens.device).scatter_reduce_(0, page0, i, "amin")
    leader = torch.where(has, lowest[page0], i)
    same = (tables == tables[leader]) & (x < torch.minimum(full, full[leader])[:, None])
    common = same.long().cumprod(1).sum(1)
    least = torch.full_like(lens, 1 << 30).scatter_reduce_(0, leader, common, "amin")
    members = torch.zeros_like(lens).scatter_add_(0, leader, has.long())
    shared = torch.where(has & (members[leader] > 1) & (least[leader] * page >= c["least"]), least[leader] * page, 0)
    leader = torch.where(shared > 0, leader, i)
    rows = torch.zeros_like(lens).scatter_add_(0, leader, torch.where(shared > 0, new, 0))
    ends = rows.cumsum(0)
    t = torch.arange(s["total"], device=lens.device)
    req = torch.searchsorted(first[1:].contiguous(), t, right=True).clamp(max=n - 1)
    order = torch.argsort(torch.where(shared[req] > 0, leader[req], n), stable=True)
    live = t < ends[-1]
    return {"leader": leader.int(), "shared": shared.int(), "first": torch.cat([ends.new_zeros(1), ends]).int(),
            "token": torch.where(live, order, -1).int(), "request": torch.where(live, req[order], -1).int()}


def _popcount(x):
    """Set bits of 64-bit words."""
    shifts = torch.arange(64, device=x.device)
    return ((x[..., None] >> shifts) & 1).sum(-1)


def _plain_attend(s):
    c = s["case"]
    h, g, d = c["kv_heads"], c["q_per_kv"], c["head_dim"]
    first, lens, most = s["first"].long(), s["lens"].long(), s["most"]
    n = len(lens)
    new = first[1:] - first[:-1]
    rows = lambda x: x[0][s["tables"].long()].transpose(1, 2).reshape(n, h, -1, d).float()  # noqa: E731
    i = torch.arange(most, device=lens.device)
    at = (first[:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][at].float().reshape(n, most, h, g, d).permute(0, 2, 1, 3, 4).reshape(n, h, most * g, d)
    score = (q @ rows(s["k"]).transpose(-1, -2)).mul_(d ** -0.5).reshape(n, h, most, g, -1)
    if c["cap"]:
        score = torch.tanh(score / c["cap"]) * c["cap"]
    j = torch.arange(score.shape[-1], device=lens.device)
    draft = j[None, :] - lens[:, None]                                     # [n, keys]
    inside = (draft >= 0) & (draft < new[:, None])
    q_pos = lens[:, None] + i
    k_pos = j[None, :].expand(n, -1)
    if s["mask"] is None:
        see = inside[:, None, :] & (draft[:, None, :] <= i[None, :, None])
    else:
        words = s["mask"][at]                                             # [n, most]
        see = inside[:, None, :] & ((words[:, :, None] >> draft.clamp(0, 63)[:, None, :]) & 1).bool()
        depth = torch.where(words != 0, _popcount(words) - 1, i)  # ancestors of each draft
        q_pos = lens[:, None] + depth
        k_pos = torch.where(inside, lens[:, None] + depth.gather(1, draft.clamp(0, most - 1)), k_pos)
    see = see | (draft < 0)[:, None, :]
    far = q_pos[:, :, None] - k_pos[:, None, :]                           # [n, most, keys]
    if c["window"]:
        see = see & (far < c["window"])
    if s["slopes"] is not None:
        score = score - s["slopes"].reshape(1, h, 1, g, 1) * far[:, None, :, None, :]
    score = score.masked_fill_(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    sums = p.sum(-1, keepdim=True)
    out = (p.reshape(n, h, most * g, -1) @ rows(s["v"])).reshape(n, h, most, g, d) / torch.where(sums == 0, 1.0, sums)
    lse = (top + torch.log(sums))[..., 0]
    t = torch.arange(s["total"], device=lens.device)
    req = torch.searchsorted(first[1:].contiguous(), t, right=True)
    at = t - first[req]
    out = out.permute(0, 2, 1, 3, 4).reshape(n, most, h * g, d)[req, at]
    lse = lse.permute(0, 2, 1, 3).reshape(n, most, h * g)[req, at]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _turned(x, cos, sin, c):
    """Rotates part of each head: x [T, heads, D] float32."""
    rot, o = c["rot"], c["offset"]
    part = x[..., o:o + rot]
    if c["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        new = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        new = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([x[..., :o], new, x[..., o + rot:]], -1)


def _plain_rotary(s):
    c = s["case"]
    h, g, d, t = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["tokens"]
    q, k, v = s["qkv"].split((h * g * d, h * d, h * d), 1)
    angle = (s["pos"].long()[s["axes"].long()].T.double() * s["inv"])[:, None, :]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    q = _turned(q.reshape(t, h * g, d).float(), cos, sin, c)
    k = _turned(k.reshape(t, h, d).float(), cos, sin, c).to(s["k"].dtype)
    v = v.reshape(t, h, d)
    if c["step_rows"]:
        n = c["step_rows"]
        q = q.reshape(t // n, n, h, g, d).transpose(1, 2).reshape(t, h * g, d)
        at, off = torch.arange(t, device=q.device), 0
    else:
        at, off = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    s["k"][0, at, :, off] = k
    s["v"][0, at, :, off] = v
    return {"q": q.to(s["q_out"].dtype), "k": s["k"], "v": s["v"]}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    if case["op"] == "find":
        return None
    s = prepare(case, seed)
    return {"fork": _exact_fork, "compact": _exact_compact, "attend": _exact_attend,
            "rotary": _exact_rotary}[case["op"]](case, s)


def _exact_fork(c, s):
    page, lens, tables = c["page"], s["lens"].tolist(), s["tables"].tolist()
    parent, free, count = s["parent"].tolist(), s["free"].tolist(), s["count"].item()
    k, v = s["k"].double(), s["v"].double()
    old, kept = (k.clone(), v.clone()), set()
    for r in range(len(lens)):                    # whoever goes on with a row by itself keeps its last page
        if parent[r] == r:
            kept.add(r)
    for r, q in enumerate(parent):
        if q in (r, -1):
            continue
        full, fill = divmod(lens[q], page)
        if fill == 0:
            continue
        if q not in kept:
            kept.add(q)
            continue
        count -= 1
        for now, before in zip((k, v), old):
            now[:, free[count], :, :fill] = before[:, tables[q][full], :, :fill]
    out = dict.fromkeys(("tables", "lens", "free", "count", "shares"))
    return {"k": k, "v": v, **out}


def _exact_compact(c, s):
    count = s["count"].item()
    free = set(s["free"].tolist()[:count])
    pool = s["free"].numel()
    live = pool - count
    holes = [i for i in range(live) if i in free]
    movers = [i for i in range(live, pool) if i not in free]
    k, v = s["k"].double(), s["v"].double()
    if movers:
        for x in (k, v):
            x[:, holes] = x[:, movers]
    return {"k": k, "v": v, "tables": None, "free": None, "shares": None, "map": None}


def _exact_attend(c, s):
    h, g, d, page = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["page"]
    first, ctx = s["first"].tolist(), s["lens"].tolist()
    if sum((b - a) * n for a, b, n in zip(first, first[1:], ctx)) * h * g * d > 1 << 40:
        return None
    words = None if s["mask"] is None else s["mask"].tolist()
    out = torch.zeros(s["total"], h * g, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], h * g, dtype=torch.float64, device="cuda")
    for r, L in enumerate(ctx):
        at, n = first[r], first[r + 1] - first[r]
        if n == 0:
            continue
        ids = s["tables"][r, :-(-(L + n) // page)].long()
        pos = torch.arange(L + n, device="cuda")
        see = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        if words is None:
            see[:, L:] = torch.tril(see[:, L:])
        else:
            w = words[at:at + n]
            see[:, L:] = torch.tensor([[(w[a] >> b) & 1 for b in range(n)] for a in range(n)],
                                      dtype=torch.bool, device="cuda")
            depth = see[:, L:].sum(1)
            pos[L:] = torch.where(depth > 0, L + depth - 1, pos[L:])
        far = pos[L:, None] - pos[None, :]
        if c["window"]:
            see &= far < c["window"]
        for a in range(h):
            kd, vd = (x[0, ids, a].reshape(-1, d)[:L + n].double() for x in (s["k"], s["v"]))
            z = torch.einsum("ngd,kd->gnk", s["q"][at:at + n, a * g:(a + 1) * g].double(), kd) / math.sqrt(d)
            if c["cap"]:
                z = c["cap"] * torch.tanh(z / c["cap"])
            if s["slopes"] is not None:
                z = z - s["slopes"][a * g:(a + 1) * g, None, None].double() * far
            z[:, ~see] = -math.inf
            lse[at:at + n, a * g:(a + 1) * g] = torch.logsumexp(z, 2).T
            out[at:at + n, a * g:(a + 1) * g] = (torch.nan_to_num(torch.softmax(z, 2)) @ vd).transpose(0, 1)
    return {"out": out, "lse": lse}


def _exact_rotary(c, s):
    h, g, d, t = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["tokens"]
    x = s["qkv"].double().reshape(t, h * g + 2 * h, d)
    half = c["rot"] // 2
    lo = torch.arange(half, device=x.device)
    lo, hi = (2 * lo, 2 * lo + 1) if c["interleaved"] else (lo, lo + half)
    lo, hi = lo + c["offset"], hi + c["offset"]
    angle = torch.stack([s["pos"][a].double() * s["inv"][i] for i, a in enumerate(s["axes"].tolist())], 1)
    z = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.clone()
    w = torch.complex(x[:, :h * g + h, lo], x[:, :h * g + h, hi]) * z
    y[:, :h * g + h, lo], y[:, :h * g + h, hi] = w.real, w.imag
    q, k, v = y.split((h * g, h, h), 1)
    n = c["step_rows"]
    if n:
        q = torch.cat([q[i:i + n].reshape(n, h, g, d).transpose(0, 1).reshape(n, h * g, d)
                       for i in range(0, t, n)])
    pages = []
    for rows in (k, v):
        p = torch.zeros(s["k"].shape, dtype=torch.float64, device=x.device).transpose(2, 3)
        flat = p.reshape(-1, h, d)
        flat[torch.arange(t, device=x.device) if n else s["slots"].long()] = rows
        pages.append(flat.reshape(p.shape).transpose(2, 3))
    return {"q": q, "k": pages[0], "v": pages[1]}
