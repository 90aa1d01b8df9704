"""Plain definitions of the operators of shared pages in numpy, request by
request (include/avsg.h); pages are arrays [L, P, H, pt, D]."""
import numpy as np


def fork(lens, parent, tables, free, count, shares, page, pages):
    """(lens, tables, free, count, shares) afterwards; the pages are changed in place."""
    n = len(lens)
    new_lens, new_tables, free, shares = lens.copy(), tables.copy(), free.copy(), shares.copy()
    held = [-(-int(x) // page) for x in lens]
    holders = {}
    for r in range(n):
        for x in range(held[r]):
            holders.setdefault(int(tables[r, x]), []).append(r)
    now = {i: 0 for i in holders}
    keeps = {r for r in range(n) if parent[r] == r}  # rows whose last page somebody goes on with
    for r in range(n):
        q = int(parent[r])
        new_lens[r] = 0 if q < 0 else lens[q]
        if q < 0:
            continue
        full, fill = divmod(int(lens[q]), page)
        if q != r:
            new_tables[r, :held[q]] = tables[q, :held[q]]
            if fill:
                if q in keeps:
                    count -= 1
                    to = int(free[count])
                    new_tables[r, full] = to
                    for a in pages:
                        a[:, to, :, :fill] = a[:, int(tables[q, full]), :, :fill]
                keeps.add(q)
        for x in range(held[r] if q == r else held[q]):
            i = int(tables[q, x])
            if x < full or int(new_tables[r, x]) == i:
                now[i] += 1
    back = []
    for r in range(n):
        for x in range(held[r]):
            i = int(tables[r, x])
            if now[i] == 0 and max(holders[i]) == r:
                back.append(i)
    for i, k in now.items():
        shares[i] = max(0, shares[i] + k - len(holders[i]))
    for i in reversed(back):
        free[count] = i
        count += 1
    return new_lens, new_tables, free, count, shares


def compact(lens, tables, free, count, shares, page, pages):
    """(tables, free, shares, map) afterwards; the pages are changed in place."""
    pool = len(free)
    live = pool - count
    stack = set(free[:count].tolist())
    where = {i: i for i in range(live) if i not in stack}
    movers, holes = [i for i in range(live, pool) if i not in stack], [i for i in range(live) if i in stack]
    assert len(movers) == len(holes)
    for a, b in zip(movers, holes):
        where[a] = b
        for x in pages:
            x[:, b] = x[:, a]
    tables, free, new_shares = tables.copy(), free.copy(), np.zeros_like(shares)
    for r, n in enumerate(lens.tolist()):
        for x in range(-(-n // page)):
            tables[r, x] = where[int(tables[r, x])]
    for a, b in where.items():
        new_shares[b] = shares[a]
    free[:count] = [pool - 1 - i for i in range(count)]
    return tables, free, new_shares, np.array([where.get(i, -1) for i in range(pool)], np.int32)


def find(lens, tables, first, page, least, capacity):
    """(leader, shared, group_first, token, request)."""
    n = len(lens)
    groups = {}
    for r in range(n):
        if first[r + 1] > first[r] and lens[r] >= page:
            groups.setdefault(int(tables[r, 0]), []).append(r)
    leader, shared = np.arange(n, dtype=np.int32), np.zeros(n, np.int32)
    members = {r: [] for r in range(n)}
    for of in groups.values():
        common = 0
        while all(lens[r] // page > common and tables[r, common] == tables[of[0], common] for r in of):
            common += 1
        if len(of) > 1 and common * page >= least:
            for r in of:
                leader[r], shared[r] = of[0], common * page
            members[of[0]] = of
    token, request, group_first = [], [], [0]
    for r in range(n):
        for m in members[r]:
            token += range(first[m], first[m + 1])
            request += [m] * int(first[m + 1] - first[m])
        group_first.append(len(token))
    pad = [-1] * (capacity - len(token))
    return leader, shared, *(np.array(x, np.int32) for x in (group_first, token + pad, request + pad))
