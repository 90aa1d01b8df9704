"""Plain definitions of the paged-cache operators in numpy and 64 bits, request
by request; shared by the tests of include/avsg.h's paged entry points."""
import math

import numpy as np


def popcount(x):
    return bin(int(x) & (2**64 - 1)).count("1")


def plan(lens, new, tables, free, count, page, capacity, mask=None):
    """(first, slots, pos, tables, count) after taking pages from the stack."""
    tables = tables.copy()
    first = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots, pos = np.full(capacity, -1, np.int32), np.zeros(capacity, np.int32)
    for r, (length, n) in enumerate(zip(lens.tolist(), new.tolist())):
        for x in range(-(-length // page), -(-(length + n) // page)):
            count -= 1
            tables[r, x] = free[count]
        for i in range(n):
            t, p = first[r] + i, length + i
            slots[t] = tables[r, p // page] * page + p % page
            bits = 0 if mask is None else popcount(mask[t])
            pos[t] = length + bits - 1 if bits else p
    return first, slots, pos, tables, count


def keep(lens, first, path, kept, tables, free, count, page, pages):
    """(lens, free, count) afterwards; every array of pages [L, P, H, pt, D] is
    changed in place."""
    lens, free, back = lens.copy(), free.copy(), []
    for r in range(len(lens)):
        n, k, old = int(first[r + 1] - first[r]), int(kept[r]), int(lens[r])
        at = lambda p: (int(tables[r, p // page]), p % page)  # noqa: E731
        for x in pages:
            src = [at(old + (int(path[first[r] + i]) if path is not None else i)) for i in range(max(k, 0))]
            rows = [x[:, a, :, b].copy() for a, b in src]
            for i, row in enumerate(rows):
                a, b = at(old + i)
                x[:, a, :, b] = row
        lens[r] = 0 if k < 0 else old + k
        back += [int(tables[r, x]) for x in range(-(-int(lens[r]) // page), -(-(old + n) // page))]
    for page_id in reversed(back):
        free[count] = page_id
        count += 1
    return lens, free, count


def rotate(x, turns, rot, offset, interleaved, magnitude):
    """x [T, heads, D] float64, turns [T, rot / 2] float64 in whole turns."""
    y = x.copy()
    half = rot // 2
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, s = (f(2 * math.pi * turns)[:, None, :] * magnitude for f in (np.cos, np.sin))
    xa, xb = x[..., offset + a], x[..., offset + b]
    y[..., offset + a] = xa * c - xb * s
    y[..., offset + b] = xa * s + xb * c
    return y


def turns_of(pos, freq):
    """Fractions of a turn, from the table's 64-bit words (exact integers)."""
    return np.array([[((int(p) * int(f)) % 2**64) / 2.0**64 for f in freq] for p in pos])


def attention(q, k, v, length, mask=None, scale=None, cap=0.0, window=0, slopes=None):
    """One request and one kv-head: q [n, G, D], k and v [length + n, D] float64,
    mask n words or None (a chain), slopes [G].  Returns out [n, G, D], lse [n, G] and
    the sums of weights times |v| (what a rounding of the weights scales with)."""
    n, groups, dim = q.shape
    scale = dim ** -0.5 if scale is None else scale
    out, lse, size = np.zeros_like(q), np.full((n, groups), -math.inf), np.zeros_like(q)
    depth = np.arange(n)
    if mask is not None:
        bits = np.array([popcount(m) for m in mask])
        depth = np.where(bits > 0, bits - 1, depth)
    k_pos = np.concatenate([np.arange(length), length + depth])
    for t in range(n):
        see = np.ones(length + n, bool)
        for j in range(n):
            see[length + j] = j <= t if mask is None else (int(mask[t]) >> j) & 1
        far = length + depth[t] - k_pos
        if window:
            see &= far < window
        if not see.any():
            continue
        for g in range(groups):
            s = scale * (k[see] @ q[t, g])
            if cap:
                s = cap * np.tanh(s / cap)
            if slopes is not None:
                s = s - slopes[g] * far[see]
            m = s.max()
            e = np.exp(s - m)
            lse[t, g] = m + math.log(e.sum())
            out[t, g] = (e / e.sum()) @ v[see]
            size[t, g] = (e / e.sum()) @ np.abs(v[see])
    return out, lse, size
