"""Cases that measure the paged-cache operators: page planning, rotary write,
tree attention and the keep of accepted drafts.

With ``own`` false, ``run`` computes each operator in its plain form from
elementary torch operations; with ``own`` true it makes the calls a user of
``decode_serving_gb300.paged`` makes.  Sizes follow this repository's
workloads (8 kv-heads, 4 query heads per kv-head, head width 128, contexts up
to 65536 for multi-token decoding, 16-token pages).

Layouts: K and V pages [layers][num_pages][kv_heads][page][head_dim]; block
tables [requests][max_pages]; slot of a token = page id * page + offset.  The
new tokens of a step are ragged: request r owns rows first[r] .. first[r+1].
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ the cases

def _plan(name, requests, page, ctx_lo, ctx_hi, new_lo, new_hi, chunk, tree, ragged):
    return {"name": name, "op": "plan", "requests": requests, "page": page, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "new_lo": new_lo, "new_hi": new_hi, "chunk": chunk, "tree": tree,
            "ragged": ragged}


def _rotary(name, tokens, kv_heads, q_per_kv, head_dim, rot, offset, interleaved, scaled, far,
            page, step_rows, dtype):
    return {"name": name, "op": "rotary", "tokens": tokens, "kv_heads": kv_heads,
            "q_per_kv": q_per_kv, "head_dim": head_dim, "rot": rot, "offset": offset,
            "interleaved": interleaved, "scaled": scaled, "far": far, "page": page,
            "step_rows": step_rows, "dtype": dtype}


def _attend(name, requests, kv_heads, q_per_kv, head_dim, page, ctx_lo, ctx_hi, new_lo, new_hi,
            tree, cap, window, slopes, dtype, ragged):
    return {"name": name, "op": "attend", "requests": requests, "kv_heads": kv_heads,
            "q_per_kv": q_per_kv, "head_dim": head_dim, "page": page, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "new_lo": new_lo, "new_hi": new_hi, "tree": tree, "cap": cap,
            "window": window, "slopes": slopes, "dtype": dtype, "ragged": ragged}


def _keep(name, requests, layers, kv_heads, head_dim, page, ctx_lo, ctx_hi, new_hi, keep_hi,
          dtype, ragged):
    return {"name": name, "op": "keep", "requests": requests, "layers": layers,
            "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "ctx_lo": ctx_lo,
            "ctx_hi": ctx_hi, "new_lo": 1, "new_hi": new_hi, "keep_hi": keep_hi, "tree": True,
            "dtype": dtype, "ragged": ragged}


def listed():
    return [
        # One new token for each of 8 decoding requests: pure latency.
        _plan("plan decode", 8, 16, 1, 32768, 1, 1, 0, False, 1),
        # A scheduler's mixed step: draft trees for most requests, prompt chunks for every eighth.
        _plan("plan mixed", 509, 16, 0, 65536, 1, 64, 2048, True, 2),
        # The projections of one decode step of 8 requests, written to their pages.
        _rotary("rotary decode", 8, 8, 4, 128, 128, 0, False, False, 32768, 16, 0, "bf16"),
        # Three tokens for each of 16 requests: fp32 queries in the sparse step's layout, K and V
        # as one row per token.
        _rotary("rotary step", 48, 8, 4, 128, 128, 0, False, False, 65536, 1, 3, "bf16"),
        # A long prompt's chunk at far positions: half of each head, neighbouring pairs, scaled.
        _rotary("rotary prompt", 16381, 8, 4, 128, 64, 0, True, True, 1 << 20, 16, 0, "fp16"),
        # One token of one request on one head: latency.
        _attend("attend tiny", 1, 1, 1, 128, 16, 4096, 4096, 1, 1, False, 0.0, 0, False, "bf16", 3),
        # A ragged batch, one token each.
        _attend("attend decode", 8, 8, 4, 128, 16, 1, 32768, 1, 1, False, 0.0, 0, False, "bf16", 4),
        # Draft trees of up to 64 tokens over long ragged contexts (the largest).
        _attend("attend trees", 16, 8, 4, 128, 16, 1024, 65536, 1, 64, True, 0.0, 0, False, "bf16", 5),
        # Capped scores, distance bias and a window, narrow heads, five query heads per kv-head.
        _attend("attend capped", 6, 4, 5, 64, 8, 3, 20000, 1, 29, True, 30.0, 8192, True, "fp16", 6),
        # Prompt chunks: causal rows over an earlier part.
        _attend("attend prompt", 2, 8, 4, 128, 16, 4099, 8192, 2000, 4096, False, 0.0, 0, False, "bf16", 7),
        # The kept paths of a few small trees in one layer.
        _keep("keep small", 4, 1, 8, 128, 16, 17, 200, 16, 5, "bf16", 8),
        # The same for a batch through 16 layers, some requests ending.
        _keep("keep layers", 64, 16, 8, 128, 16, 5, 120, 64, 8, "bf16", 9),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "rotary", "attend", "attend", "keep"))
    ragged = rng.randrange(1 << 20)
    dtype = rng.choice(("bf16", "fp16"))
    page = rng.choice((1, 8, 16, 32, 64))
    if op == "plan":
        hi = _log(rng, 1, 64)
        c = _plan("", _log(rng, 1, 512), page, 0, _log(rng, 16, 65536), 0, hi,
                  rng.choice((0, _log(rng, 65, 2048))), rng.random() < 0.5, ragged)
    elif op == "rotary":
        d = rng.choice((64, 128, 256))
        rot = rng.choice((d, d // 2, d // 4, 24))
        offset = rng.choice((0, d - rot))
        h, g = rng.choice((1, 2, 4, 8)), rng.choice((1, 2, 3, 4, 8))
        step = rng.choice((0, 0, 1, 2, 3))
        t = _log(rng, 1, min(16384, (16384 * 48 * 128) // (d * h * (g + 2))))
        t = max(1, t // step) * step if step else t
        c = _rotary("", t, h, g, d, rot, offset, rng.random() < 0.5, rng.random() < 0.5,
                    _log(rng, 64, 1 << 20), 1 if step else page, step, dtype)
    elif op == "attend":
        r, h = _log(rng, 1, 32), rng.choice((1, 2, 4, 8))
        g, d = rng.choice((1, 2, 3, 4, 5, 8, 16)), rng.choice((64, 128, 256))
        tree = rng.random() < 0.6
        new = _log(rng, 1, 64) if tree else rng.choice((1, _log(rng, 1, 2048)))
        rows = r * h * d
        most = min(131072, (16 * 8 * 128 * 40000) // rows, (1 << 31) // (r * h * g * new) + 1)
        c = _attend("", r, h, g, d, page, rng.choice((0, 1)), _log(rng, 1, max(2, most)),
                    rng.choice((0, 1, new)), new, tree, rng.choice((0.0, 0.0, 50.0)),
                    rng.choice((0, 0, _log(rng, 16, 8192))), rng.random() < 0.3, dtype, ragged)
    else:
        new = _log(rng, 1, 64)
        c = _keep("", _log(rng, 1, 64), _log(rng, 1, 16), rng.choice((1, 2, 8)),
                  rng.choice((64, 128)), page, 0, _log(rng, 1, 150), new,
                  rng.randint(0, min(new, 9)), dtype, ragged)
    del c["name"]
    return c


# ------------------------------------------- what follows from a case's lengths

def _lengths(case):
    """Context length and count of new tokens of every request (int64 arrays)."""
    r = random.Random(case["ragged"])
    n = case["requests"]
    ctx = [case["ctx_lo"] + round((case["ctx_hi"] - case["ctx_lo"]) * r.random()) for _ in range(n)]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n)]
    ctx[-1] = case["ctx_hi"]
    new[0] = case["new_hi"]
    chunk = case.get("chunk", 0)
    if chunk:
        for i in range(0, n, 8):
            new[i] = r.randint(65, chunk)
    return np.array(ctx, np.int64), np.array(new, np.int64)


def _pages(case, ctx, new):
    """(table width, pages in the pool)"""
    need = -(-(ctx + new) // case["page"])
    return max(1, int(need.max())), int(need.sum()) + 3


def _kept(case, new):
    """Kept drafts per request (-1: the request ends), from the lengths alone."""
    r = random.Random(case["ragged"] + 1)
    out = []
    for n in new:
        if r.random() < 0.1:
            out.append(-1)
        else:
            out.append(min(r.randint(0, case["keep_hi"]), int(n)))
    return np.array(out, np.int64)


def _paths(case, new, keep):
    """Kept paths: the first drafts stay, the later ones come from behind the kept range."""
    r = random.Random(case["ragged"] + 2)
    rows = []
    for n, k in zip(new.tolist(), keep.tolist()):
        row = list(range(n))
        if k > 0:
            tail = r.randint(0, min(k, n - k))
            row[:k] = list(range(k - tail)) + sorted(r.sample(range(k, n), tail))
        rows += row
    return np.array(rows, np.int64)


def _trees(case, new, seed):
    """Ancestor masks (own bit included) of random trees, one 64-bit word per new token;
    requests with more than 64 new tokens are chains and get zeros."""
    r = np.random.default_rng([seed, 11])
    n, most = len(new), int(min(64, new.max()))
    word = np.zeros((n, most), np.uint64)
    for i in range(most):
        bit = np.uint64(1 << i)
        if i == 0:
            word[:, 0] = bit
        else:
            parent = np.maximum(0, i - 1 - r.integers(0, 4, n))
            word[:, i] = word[np.arange(n), parent] | bit
    total = int(new.sum())
    out = np.zeros(total, np.uint64)
    first = np.concatenate([[0], np.cumsum(new)])
    req = np.repeat(np.arange(n), new)
    i = np.arange(total) - first[req]
    small = new[req] <= 64
    out[small] = word[req[small], i[small]]
    return out.view(np.int64)


def work(case):
    op = case["op"]
    if op == "rotary":
        t, h, g, d = case["tokens"], case["kv_heads"], case["q_per_kv"], case["head_dim"]
        q_out = 4 if case["step_rows"] else 2
        return {"bytes": t * d * (h * g * (2 + q_out) + h * 8) + 8 * t,
                "flops": 6 * t * (case["rot"] // 2) * h * (g + 1)}
    ctx, new = _lengths(case)
    total = int(new.sum())
    page = case["page"]
    if op == "plan":
        extra = int((-(-(ctx + new) // page) + (-ctx // page)).sum())
        return {"bytes": 8 * total + (8 * total if case["tree"] else 0) + 12 * len(ctx) + 8 * extra,
                "flops": 0}
    if op == "keep":
        keep = _kept(case, new)
        path = _paths(case, new, keep)
        first = np.concatenate([[0], np.cumsum(new)])[:-1]
        moved = sum(int((path[f:f + k] != np.arange(k)).sum())
                    for f, k in zip(first.tolist(), np.maximum(keep, 0).tolist()))
        row = case["layers"] * case["kv_heads"] * case["head_dim"] * 2 * 2
        return {"bytes": 2 * moved * row + 4 * total + 16 * len(ctx), "flops": 0}
    h, g, d = case["kv_heads"], case["q_per_kv"], case["head_dim"]
    seen = ctx if not case["window"] else np.minimum(ctx, case["window"])
    pairs = new * seen + (new * (new + 1) // 2)
    keys = np.where(new > 0, seen + new, 0)
    return {"bytes": int(keys.sum()) * h * d * 4 + total * h * g * (4 * d + 4),
            "flops": int(pairs.sum()) * h * g * 4 * d}


# ------------------------------------------------------------------ the inputs

def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def _normal(seed, *shape, dtype):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)


def _frequencies(case):
    """Angle per position of every pair (radians, float64) and the factor on cos and sin."""
    half = case["rot"] // 2
    inv = 10000.0 ** (-np.arange(half, dtype=np.float64) / half)
    if not case["scaled"]:
        return inv, 1.0
    # slow pairs are stretched by 32, fast ones kept, in between a ramp over their turns in 32768 tokens
    turns = 32768 * inv / (2 * math.pi)
    keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
    return inv * (keep + (1 - keep) / 32.0), 0.1 * math.log(32.0) + 1.0


def prepare(case, seed):
    """What a program has before the call: the cache, the step's rows, the plan's arrays."""
    s = {"case": case}
    op, page = case["op"], case["page"]
    if op == "rotary":
        dt = DTYPES[case["dtype"]]
        t, h, g, d = case["tokens"], case["kv_heads"], case["q_per_kv"], case["head_dim"]
        r = np.random.default_rng([seed, 3])
        s["qkv"] = _normal(seed, t, (h * g + 2 * h) * d, dtype=dt)
        s["pos"] = _dev(r.integers(0, case["far"], t))
        pool = t if case["step_rows"] else -(-t // page) + 2
        s["slots"] = None if case["step_rows"] else _dev(r.permutation(pool * page)[:t])
        s["k"], s["v"] = (torch.zeros(1, pool, h, page, d, dtype=dt, device="cuda") for _ in "kv")
        inv, s["mag"] = _frequencies(case)
        s["inv"] = torch.from_numpy(inv).cuda()
        s["q_out"] = torch.empty(t, h * g, d, device="cuda",
                                 dtype=torch.float32 if case["step_rows"] else dt)
        s["tables"] = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
        s["lens"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["free"] = torch.zeros(pool, dtype=torch.int32, device="cuda")
        s["count"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    else:
        ctx, new = _lengths(case)
        n, total = len(ctx), int(new.sum())
        width, pool = _pages(case, ctx, new)
        r = np.random.default_rng([seed, 4])
        ids = r.permutation(pool)
        held = -(-(ctx + (0 if op == "plan" else new)) // page)
        tables = np.zeros((n, width), np.int64)
        grid = np.arange(width)[None, :] < held[:, None]
        tables[grid] = ids[:int(held.sum())]
        left = ids[int(held.sum()):]
        free = np.zeros(pool, np.int64)
        free[:len(left)] = left
        s["tables"], s["lens"], s["free"] = _dev(tables), _dev(ctx), _dev(free)
        s["count"] = _dev(np.array([len(left)]))
        s["count_out"], s["lens_out"] = torch.zeros_like(s["count"]), torch.zeros_like(s["lens"])
        s["new"] = _dev(new)
        s["total"], s["most"] = total, int(new.max())
        s["mask"] = _dev(_trees(case, new, seed), torch.int64) if case["tree"] else None
        if op == "plan":
            s["room"] = total + 5  # the arrays of a step are sized for more tokens than it has
            s["first"] = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
            s["slots"], s["pos"] = (torch.zeros(s["room"], dtype=torch.int32, device="cuda") for _ in "sp")
            s["k"] = s["v"] = torch.zeros(1, pool, 1, page, 8, dtype=torch.bfloat16, device="cuda")
        else:
            dt = DTYPES[case["dtype"]]
            h, d = case["kv_heads"], case["head_dim"]
            s["first"] = _dev(np.concatenate([[0], np.cumsum(new)]))
            s["k"] = _normal(seed, case.get("layers", 1), pool, h, page, d, dtype=dt)
            s["v"] = _normal(seed + (1 << 40), case.get("layers", 1), pool, h, page, d, dtype=dt)
            if op == "keep":
                keep = _kept(case, new)
                s["keep"], s["path"] = _dev(keep), _dev(_paths(case, new, keep))
            else:
                g = case["q_per_kv"]
                s["q"] = _normal(seed + 7, total, h * g, d, dtype=dt)
                s["out"] = torch.empty_like(s["q"])
                s["lse"] = torch.empty(total, h * g, dtype=torch.float32, device="cuda")
                s["slopes"] = (2.0 ** (-8.0 * torch.arange(1, h * g + 1, device="cuda") / (h * g))
                               if case["slopes"] else None)
    if own:
        from decode_serving_gb300 import paged
        s["cache"] = paged.PagedCache(s["k"], s["v"], s["tables"], s["lens"], s["free"], s["count"])
        if op == "rotary":
            scaling = dict(factor=32.0, low_turns=1.0, high_turns=32.0, original=32768) if case["scaled"] else {}
            s["freq"] = paged.rotary_frequencies(case["rot"], base=10000.0, **scaling).cuda()
        if op == "attend":
            s["work"] = s["cache"].attention_workspace(case["q_per_kv"], s["most"])
    return s


# ------------------------------------------------------------------ the passes

def run(s):
    op = s["case"]["op"]
    if own:
        return {"plan": _own_plan, "rotary": _own_rotary, "attend": _own_attend,
                "keep": _own_keep}[op](s)
    return {"plan": _plain_plan, "rotary": _plain_rotary, "attend": _plain_attend,
            "keep": _plain_keep}[op](s)


def _own_plan(s):
    s["cache"].plan(s["new"], s["first"], s["slots"], s["pos"], mask=s["mask"],
                    free_count_out=s["count_out"])
    return {"first": s["first"], "slots": s["slots"], "pos": s["pos"], "tables": s["tables"],
            "count": s["count_out"]}


def _own_rotary(s):
    c = s["case"]
    h, g, d = c["kv_heads"], c["q_per_kv"], c["head_dim"]
    q, k, v = s["qkv"].split((h * g * d, h * d, h * d), 1)
    s["cache"].rotary(q, k, v, s["pos"], s["slots"], s["freq"], s["q_out"], rot_offset=c["offset"],
                      interleaved=c["interleaved"], magnitude=s["mag"],
                      tokens_per_request=max(1, c["step_rows"]))
    return {"q": s["q_out"], "k": s["k"], "v": s["v"]}


def _own_attend(s):
    c = s["case"]
    s["cache"].attend(s["q"], s["first"], s["out"], s["most"], s["work"], mask=s["mask"],
                      lse=s["lse"], softcap=c["cap"], window=c["window"], slopes=s["slopes"])
    return {"out": s["out"], "lse": s["lse"]}


def _own_keep(s):
    s["cache"].keep(s["first"], s["path"], s["keep"], lens_out=s["lens_out"],
                    free_count_out=s["count_out"])
    return {"k": s["k"], "v": s["v"], "lens": s["lens_out"], "free": s["free"],
            "count": s["count_out"]}


def _popcount(x):
    """Set bits of 64-bit words."""
    shifts = torch.arange(64, device=x.device)
    return ((x[..., None] >> shifts) & 1).sum(-1)


def _plain_plan(s):
    page, room = s["case"]["page"], s["room"]
    lens, new, tables = s["lens"].long(), s["new"].long(), s["tables"].long()
    ends = new.cumsum(0)
    first = torch.cat([ends.new_zeros(1), ends])
    held, need = (lens + page - 1) // page, (lens + new + page - 1) // page
    extra = need - held
    base = extra.cumsum(0) - extra
    x = torch.arange(tables.shape[1], device=lens.device)[None, :]
    taken = (x >= held[:, None]) & (x < need[:, None])
    at = (s["count"].long() - 1 - (base[:, None] + x - held[:, None])).clamp(0, s["free"].numel() - 1)
    tables = torch.where(taken, s["free"].long()[at], tables)
    t = torch.arange(room, device=lens.device)
    req = torch.searchsorted(ends, t, right=True).clamp(max=len(lens) - 1)
    i = t - first[req]
    p = lens[req] + i
    slot = tables[req, (p // page).clamp(max=tables.shape[1] - 1)] * page + p % page
    pos = p
    if s["mask"] is not None:
        words = torch.cat([s["mask"], s["mask"].new_zeros(room - s["total"])])
        pos = torch.where(words != 0, lens[req] + _popcount(words) - 1, p)
    live = t < first[-1]
    s["tables"].copy_(tables)
    return {"first": first.int(), "slots": torch.where(live, slot, -1).int(),
            "pos": torch.where(live, pos, 0).int(), "tables": s["tables"],
            "count": (s["count"] - extra.sum()).int()}


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
    angle = s["pos"].double()[:, None, None] * s["inv"]
    cos, sin = ((f(angle) * s["mag"]).float() for f in (torch.cos, torch.sin))
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


def _plain_attend(s):
    c = s["case"]
    h, g, d, page = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["page"]
    first, lens, most = s["first"].long(), s["lens"].long(), s["most"]
    n = len(lens)
    new = first[1:] - first[:-1]
    rows = lambda x: x[0][s["tables"].long()].transpose(1, 2).reshape(n, h, -1, d).float()  # noqa: E731
    k, v = rows(s["k"]), rows(s["v"])
    i = torch.arange(most, device=k.device)
    at = (first[:-1, None] + i).clamp(max=s["total"] - 1)
    q = s["q"][at].float().reshape(n, most, h, g, d).permute(0, 2, 1, 3, 4).reshape(n, h, most * g, d)
    score = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).reshape(n, h, most, g, -1)
    if c["cap"]:
        score = torch.tanh(score / c["cap"]) * c["cap"]
    j = torch.arange(k.shape[2], device=k.device)
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
    score = score.masked_fill(~see[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(score - top)
    sums = p.sum(-1, keepdim=True)
    out = (p.reshape(n, h, most * g, -1) @ v).reshape(n, h, most, g, d) / torch.where(sums == 0, 1.0, sums)
    lse = (top + torch.log(sums))[..., 0]
    t = torch.arange(s["total"], device=k.device)
    req = torch.searchsorted(first[1:], t, right=True)
    at = t - first[req]
    out = out.permute(0, 2, 1, 3, 4).reshape(n, most, h * g, d)[req, at]
    lse = lse.permute(0, 2, 1, 3).reshape(n, most, h * g)[req, at]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _plain_keep(s):
    c = s["case"]
    page, top = c["page"], c["keep_hi"]
    first, lens, keep, tables = (s[x].long() for x in ("first", "lens", "keep", "tables"))
    new = first[1:] - first[:-1]
    i = torch.arange(top, device=lens.device)
    live = i < keep[:, None]
    to = lens[:, None] + i
    path = s["path"].long()[(first[:-1, None] + i).clamp(max=s["total"] - 1)]
    src = torch.where(live, lens[:, None] + path, to)
    width = tables.shape[1]
    slot = lambda p: (tables.gather(1, (p // page).clamp(max=width - 1)), p % page)  # noqa: E731
    (fp, fo), (tp, to_) = slot(src), slot(to)
    # places that nothing is kept in write a spare row that no request holds
    spare = s["free"].long()[0]
    fp, tp = torch.where(live, fp, spare), torch.where(live, tp, spare)
    fo, to_ = torch.where(live, fo, 0), torch.where(live, to_, 0)
    for x in (s["k"], s["v"]):
        x[:, tp, :, to_] = x[:, fp, :, fo]
    after = torch.where(keep < 0, 0, lens + keep)
    a, b = (after + page - 1) // page, (lens + new + page - 1) // page
    x = torch.arange(width, device=lens.device)[None, :]
    back = ((x >= a[:, None]) & (x < b[:, None])).flatten()
    order = back.long().cumsum(0) - 1
    count, m = s["count"].long(), back.sum()
    free = torch.cat([s["free"].long(), s["free"].new_zeros(1).long()])
    at = torch.where(back, count + m - 1 - order, len(free) - 1)
    free[at] = tables.flatten()
    s["free"].copy_(free[:-1])
    return {"k": s["k"], "v": s["v"], "lens": after.int(), "free": s["free"],
            "count": (s["count"] + m).int()}


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """The definitions, request by request, in 64 bits."""
    if case["op"] == "plan":
        return None
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "attend": _exact_attend, "keep": _exact_keep}[case["op"]](case, s)


def _exact_rotary(c, s):
    h, g, d, t = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["tokens"]
    x = s["qkv"].double().reshape(t, h * g + 2 * h, d)
    half = c["rot"] // 2
    lo = torch.arange(half, device=x.device)
    lo, hi = (2 * lo, 2 * lo + 1) if c["interleaved"] else (lo, lo + half)
    lo, hi = lo + c["offset"], hi + c["offset"]
    z = torch.polar(torch.full((t, 1, half), float(s["mag"]), dtype=torch.float64, device=x.device),
                    s["pos"].double()[:, None, None] * s["inv"])
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


def _exact_attend(c, s):
    h, g, d, page = c["kv_heads"], c["q_per_kv"], c["head_dim"], c["page"]
    ctx, new = _lengths(c)
    if int((new * (ctx + new)).sum()) * h * g * d > 1 << 40:
        return None
    words = None if s["mask"] is None else s["mask"].tolist()
    out = torch.zeros(s["total"], h * g, d, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["total"], h * g, dtype=torch.float64, device="cuda")
    at = 0
    for r, (L, n) in enumerate(zip(ctx.tolist(), new.tolist())):
        if n == 0:
            continue
        ids = s["tables"][r, :-(-(L + n) // page)].long()
        k, v = (x[0, ids].transpose(0, 1).reshape(h, -1, d)[:, :L + n] for x in (s["k"], s["v"]))
        pos = torch.arange(L + n, device="cuda")
        see = torch.ones(n, L + n, dtype=torch.bool, device="cuda")
        if words is None:
            see[:, L:] = torch.tril(see[:, L:])
        else:
            w = words[at:at + n]
            see[:, L:] = torch.tensor([[(w[a] >> b) & 1 for b in range(n)] for a in range(n)],
                                      dtype=torch.bool, device="cuda")
            count = see[:, L:].sum(1)
            pos[L:] = torch.where(count > 0, L + count - 1, pos[L:])
        far = pos[L:, None] - pos[None, :]
        if c["window"]:
            see &= far < c["window"]
        for a in range(h):
            kd, vd = k[a].double(), v[a].double()
            for b in range(g):
                z = s["q"][at:at + n, a * g + b].double() @ kd.T / math.sqrt(d)
                if c["cap"]:
                    z = c["cap"] * torch.tanh(z / c["cap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][a * g + b].double() * far
                z[~see] = -math.inf
                lse[at:at + n, a * g + b] = torch.logsumexp(z, 1)
                out[at:at + n, a * g + b] = torch.nan_to_num(torch.softmax(z, 1)) @ vd
        at += n
    return {"out": out, "lse": lse}


def _exact_keep(c, s):
    ctx, new = _lengths(c)
    keep, page = _kept(c, new), c["page"]
    path, tables = s["path"].tolist(), s["tables"].tolist()
    k, v = s["k"].double(), s["v"].double()
    at, dst, src = 0, [], []
    for r, (L, n, m) in enumerate(zip(ctx.tolist(), new.tolist(), keep.tolist())):
        for i in range(max(m, 0)):
            for where, p in ((dst, L + i), (src, L + path[at + i])):
                where.append((tables[r][p // page], p % page))
        at += n
    if dst:
        (a, b), (e, f) = (torch.tensor(x, device="cuda").T for x in (dst, src))
        for x in (k, v):
            x[:, a, :, b] = x[:, e, :, f]
    return {"k": k, "v": v, "lens": None, "free": None, "count": None}
