"""avsg_page_fork, avsg_page_compact, avsg_tree_keep_shared and avsg_prefix_find against their
plain definitions (tests/share_reference.py), and avsg_rotary_write_axes against 64 bits."""
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
import share_reference as want_of
from test_gpu_paged import BF16, F16, dev, host

pytestmark = pytest.mark.gpu


class Pool:
    """A cache whose requests share pages, in mid-run, and the same on the host."""

    def __init__(self, lens, page, groups=(), seed=0, spare=9, layers=1, heads=1, dim=8, dtype=BF16, room=1):
        """groups: (members, pages): the members' first pages are the first member's."""
        from decode_serving_gb300.paged import PagedCache
        r = np.random.default_rng(seed)
        self.lens, self.page = np.array(lens, np.int32), page
        held = -(-self.lens.astype(np.int64) // page)
        common = np.zeros(len(lens), np.int64)
        lead = np.arange(len(lens))
        for members, pages in groups:
            for m in members[1:]:
                common[m], lead[m] = pages, members[0]
        pool = int((held - common).sum()) + spare
        ids = r.permutation(pool)
        self.tables = r.integers(-5, 5, (len(lens), max(1, int(held.max()) + room))).astype(np.int32)
        at = 0
        self.shares = np.zeros(pool, np.int32)
        for i, n in enumerate(held):
            mine = int(n - common[i])
            self.tables[i, :common[i]] = self.tables[lead[i], :common[i]]
            self.tables[i, common[i]:n] = ids[at:at + mine]
            at += mine
            self.shares[self.tables[i, :common[i]]] += 1
        self.free = np.full(pool, -9, np.int32)
        self.free[:pool - at] = ids[at:]
        self.count = pool - at
        gen = torch.Generator("cuda").manual_seed(seed)
        self.k, self.v = (torch.randn(layers, pool, heads, page, dim, generator=gen, device="cuda").to(dtype)
                          for _ in "kv")
        self.cache = PagedCache(self.k, self.v, dev(self.tables), dev(self.lens), dev(self.free),
                                dev(np.array([self.count])), shares=dev(self.shares))
        self.pages = [x.view(torch.int16).cpu().numpy() for x in (self.k, self.v)]

    def fork(self, parent, work=None):
        work = self.cache.fork_workspace() if work is None else work
        self.cache.fork(dev(np.array(parent)), work)
        self.lens, self.tables, self.free, self.count, self.shares = want_of.fork(
            self.lens, np.array(parent), self.tables, self.free, self.count, self.shares, self.page, self.pages)

    def grow(self, new):
        """Plans and commits new tokens."""
        r, total = len(self.lens), int(np.sum(new))
        i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
        first, slots, pos = i32(r + 1), i32(max(1, total)), i32(max(1, total))
        self.cache.plan(dev(np.array(new)), first, slots, pos)
        self.cache.keep(first, None, dev(np.array(new)))
        _, _, _, self.tables, self.count = ref.plan(self.lens, np.array(new), self.tables, self.free, self.count,
                                                    self.page, max(1, total))
        self.lens = (self.lens + np.array(new)).astype(np.int32)

    def check(self):
        c = self.cache
        assert c.error()[0] == 0
        for name, g, w in (("lens", c.lens, self.lens), ("tables", c.tables, self.tables), ("free", c.free, self.free),
                           ("count", c.free_count, [self.count]), ("shares", c.shares, self.shares)):
            assert (host(g) == w).all(), name
        for name, g, w in zip("kv", (self.k, self.v), self.pages):
            assert (g.view(torch.int16).cpu().numpy() == w).all(), name


@pytest.mark.parametrize("lens,parent,page,groups", [
    ([5], [0], 4, ()),                                     # nothing happens
    ([5], [-1], 4, ()),                                    # it ends
    ([0, 0], [1, 0], 4, ()),                               # empty rows change places
    ([37, 0, 0, 0], [0, 0, 0, 0], 16, ()),                 # samples of a prompt
    ([32, 0, 9], [0, 0, 0], 16, ()),                       # a prompt that fills its pages; one that ends for it
    ([1, 0], [0, 0], 1, ()),                               # pages of one token
    ([255, 256, 257, 0], [3, 0, 1, 2], 256, ()),           # a cycle: every row moves, none is copied
    ([20, 21, 22], [1, 1, 0], 4, ()),                      # a parent that becomes a copy of another
    ([20, 21, 22], [1, 2, 2], 4, ()),                      # the heir is the lowest child
    ([21, 22, 23, 24], [3, 3, 3, 0], 4, ()),               # the last stays nobody's; its page goes to the lowest
    ([17, 18, 19, 30], [0, 0, -1, 1], 8, [((0, 1, 2, 3), 2)]),  # holders come and go at once
    ([17, 18, 19, 30], [-1, -1, -1, -1], 8, [((0, 1, 2, 3), 2)]),
    ([64, 64, 64], [2, -1, 2], 8, [((0, 1), 8), ((0, 2), 3)]),
])
@pytest.mark.parametrize("layers,heads,dim,dtype", [(1, 1, 8, BF16), (3, 2, 40, F16)])
def test_fork(lens, parent, page, groups, layers, heads, dim, dtype):
    p = Pool(lens, page, groups, layers=layers, heads=heads, dim=dim, dtype=dtype)
    p.fork(parent)
    p.check()


@pytest.mark.parametrize("requests,page,dim,steps", [(1, 4, 8, 4), (7, 4, 128, 12), (40, 1, 16, 8), (150, 16, 8, 8),
                                                     (33, 64, 256, 5)])
def test_forks_in_a_run(requests, page, dim, steps):
    """Random samples, beams, cycles and ends between steps that commit tokens, with one workspace;
    every page is accounted for at each."""
    r = np.random.default_rng(requests)
    p = Pool(r.integers(0, 5 * page, requests), page, seed=requests, spare=requests * 30, layers=2, heads=2,
             dim=dim, room=40)
    work = p.cache.fork_workspace()
    work.fill_(255)                                        # any contents
    for step in range(steps):
        parent = np.where(r.random(requests) < 0.5, np.arange(requests), r.integers(-1, requests, requests))
        if step == 3:
            parent = r.permutation(requests)
        p.fork(parent, work)
        p.check()
        holders = np.zeros(len(p.free), np.int64)
        for i, n in enumerate(p.lens.tolist()):
            np.add.at(holders, p.tables[i, :-(-n // page)], 1)
        assert ((holders > 0) == ~np.isin(np.arange(len(p.free)), p.free[:p.count])).all()
        assert (p.shares == np.maximum(holders - 1, 0)).all()
        p.grow(r.integers(0, 2 * page, requests))
        p.check()


def test_fork_of_thousands_of_requests_and_of_long_rows():
    r = np.random.default_rng(3)
    p = Pool(r.integers(0, 12, 8192), 4, spare=9000)
    p.fork(np.where(r.random(8192) < 0.3, r.integers(-1, 8192, 8192), np.arange(8192)))
    p.check()
    p = Pool([70001, 3, 70003, 0], 1, room=0, groups=[((0, 2), 50000)])
    p.fork([0, 0, -1, 2])
    p.check()


@pytest.mark.parametrize("what,code", [("parent", -4), ("low parent", -4), ("length", -4), ("columns", -2), ("page", -4),
                                       ("free page", -4), ("few", -2), ("count", -4), ("many", -2)])
def test_fork_errors_change_nothing_and_stay(what, code):
    p = Pool([37, 0, 20, 18], 16, groups=[((2, 3), 1)])
    c, parent = p.cache, [0, 0, -1, 3]
    if what == "parent":
        parent[1] = 4
    elif what == "low parent":
        parent[2] = -2
    elif what == "length":
        c.lens[3] = -1
    elif what == "columns":
        c.lens[3] = 16 * c.max_pages + 1
    elif what == "page":
        c.tables[0, 1] = c.pages
    elif what == "free page":
        c.free[p.count - 1] = -1
    elif what == "few":
        c.free_count[0] = 0
    elif what == "count":
        c.free_count[0] = c.pages + 1
    elif what == "many":                                   # a page that comes back is on the stack already
        c.free[:] = torch.arange(c.pages)
        c.free_count[0] = c.pages
        parent = [0, 1, -1, -1]
    before = [x.clone() for x in (c.lens, c.tables, c.free, c.free_count, c.shares, p.k, p.v)]
    work = c.fork_workspace()
    c.fork(dev(np.array(parent)), work)
    assert c.error()[0] == code
    c.fork(dev(np.array([0, 0, 0, 0])), work)              # latched: nothing happens
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (c.lens, c.tables, c.free, c.free_count, c.shares, p.k, p.v)))


def test_a_request_with_shared_pages_does_not_end_by_keep():
    p = Pool([20, 20, 9], 8, groups=[((0, 1), 2)])
    first = torch.zeros(4, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in (p.cache.lens, p.cache.free, p.cache.free_count)]
    p.cache.keep(first, None, dev(np.array([-1, 0, 0])))
    assert p.cache.error()[0] == -4
    assert all(torch.equal(a, b) for a, b in zip(before, (p.cache.lens, p.cache.free, p.cache.free_count)))
    p.cache.clear_error()
    p.cache.keep(first, None, dev(np.array([0, 0, -1])))   # one that shares nothing does
    assert p.cache.error()[0] == 0 and host(p.cache.lens).tolist() == [20, 20, 0]
    assert host(p.cache.free_count)[0] == p.count + 2


@pytest.mark.parametrize("lens,page,spare,layers,heads,dim", [
    ([5], 4, 0, 1, 1, 8),                                  # no page is free
    ([0, 0], 4, 5, 1, 1, 8),                               # all are
    ([9, 0, 30], 4, 30, 2, 2, 40),
    ([100, 7], 1, 3, 1, 1, 64),
    ([300, 255, 1, 90], 16, 31, 3, 2, 128),                # several pieces of a page, 32 ids a word
    (list(range(0, 400, 3)), 8, 700, 1, 1, 16),
    ([2000, 33], 256, 17, 2, 1, 256),
    ([50000, 0, 15000], 1, 536, 1, 1, 8),                  # 65536 pages, and more than a CTA's bitmap holds
    ([50000, 0, 15000], 1, 537, 1, 1, 8),
    ([60000, 9, 70000], 1, 60001, 1, 1, 8),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(lens, page, spare, layers, heads, dim, in_place):
    groups = [((0, len(lens) - 1), min(lens[0], lens[-1]) // page)] if min(lens[0], lens[-1]) >= page and len(lens) > 1 else []
    p = Pool(lens, page, groups, seed=len(lens), spare=spare, layers=layers, heads=heads, dim=dim)
    c = p.cache
    tables, free, shares, where = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, page, p.pages)
    page_map = torch.full((c.pages,), 77, dtype=torch.int32, device="cuda")
    work = c.compact_workspace()
    work.fill_(255)
    out = [c.tables, c.free, c.shares] if in_place else [torch.full_like(x, 99) for x in (c.tables, c.free, c.shares)]
    c.compact(page_map, work, *([] if in_place else out))
    assert (host(page_map) == where).all()
    for name, g, w in zip(("tables", "free", "shares"), out, (tables, free, shares)):
        assert (host(g) == w).all(), name
    if not in_place:                                       # the inputs stay
        p.check()
        c.compact(page_map, work)
    p.tables, p.free, p.shares = tables, free, shares
    p.check()
    c.compact(page_map, work)                              # once more: nothing moves
    p.check()
    n = c.pages - p.count
    assert (host(page_map) == np.where(np.arange(c.pages) < n, np.arange(c.pages), -1)).all()


def test_compact_without_shares():
    from decode_serving_gb300.paged import PagedCache
    p = Pool([40, 9], 8, spare=12)
    c = PagedCache(p.k, p.v, p.cache.tables, p.cache.lens, p.cache.free, p.cache.free_count)
    tables, free, _, where = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, 8, p.pages)
    page_map = torch.zeros(c.pages, dtype=torch.int32, device="cuda")
    c.compact(page_map, c.compact_workspace())
    p.tables, p.free = tables, free
    p.check()
    assert (host(page_map) == where).all()
    with pytest.raises(ValueError):
        c.compact(page_map, c.compact_workspace(), shares_out=p.cache.shares)
    with pytest.raises(ValueError):
        c.fork(dev(np.array([0, 1])), c.compact_workspace())


@pytest.mark.parametrize("what,code", [("twice", -4), ("range", -4), ("count", -4), ("free page", -4), ("page", -4),
                                       ("length", -4), ("columns", -2)])
@pytest.mark.parametrize("spare", [12, 70000])
def test_compact_errors_change_nothing(what, code, spare):
    p = Pool([40, 9, 100], 8, spare=spare)
    c = p.cache
    if what == "twice":
        c.free[1] = c.free[0]
    elif what == "range":
        c.free[2] = c.pages
    elif what == "count":
        c.free_count[0] = -1
    elif what == "free page":
        c.tables[2, 3] = c.free[0]
    elif what == "page":
        c.tables[0, 0] = -1
    elif what == "length":
        c.lens[1] = -1
    elif what == "columns":
        c.lens[1] = 8 * c.max_pages + 1
    page_map = torch.full((c.pages,), 77, dtype=torch.int32, device="cuda")
    before = [x.clone() for x in (c.tables, c.free, c.shares, page_map, p.k, p.v)]
    c.compact(page_map, c.compact_workspace())
    assert c.error()[0] == code
    assert all(torch.equal(a, b) for a, b in zip(before, (c.tables, c.free, c.shares, page_map, p.k, p.v)))


@pytest.mark.parametrize("lens,new,page,groups,least", [
    ([40], [1], 8, [], 1),
    ([40, 41], [1, 1], 8, [((0, 1), 5)], 1),
    ([40, 41], [1, 1], 8, [((0, 1), 5)], 41),              # too short a prefix
    ([40, 41], [1, 0], 8, [((0, 1), 5)], 1),               # only one with new tokens
    ([7, 5], [1, 1], 8, [], 1),                            # no full page
    ([40, 100, 17, 60, 41, 3], [3, 1, 2, 0, 70, 1], 8, [((0, 2, 4), 2), ((1, 3), 7)], 16),
    ([100, 90, 80, 70], [1, 2, 3, 4], 16, [((0, 1), 5), ((0, 2), 3), ((0, 3), 1)], 16),  # the least that all share
    ([9000, 9000, 8000], [1, 1, 1], 1, [((0, 1), 9000), ((0, 2), 7999)], 1),             # rows of several pieces
    ([i * 3 + 20 for i in range(700)], [i % 4 for i in range(700)], 4,
     [(tuple(range(k, 700, 7)), 3 + k // 2) for k in range(6)], 12),
    ([20] * 8192, [1] * 8192, 8, [(tuple(range(0, 8192, 2)), 2)], 1),
])
@pytest.mark.parametrize("extra", [0, 5])
def test_find(lens, new, page, groups, least, extra):
    p = Pool(lens, page, groups, seed=7)
    first = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    total = int(first[-1]) + extra
    want = want_of.find(p.lens, p.tables, first, page, least, total)
    x = p.cache.prefix_arrays(total)
    work = p.cache.prefix_workspace()
    work.fill_(255)
    for _ in range(2):
        p.cache.find_prefixes(dev(first), x, work, min_tokens=least)
        for name, g, w in zip(("leader", "shared", "first", "token", "request"),
                              (x.leader, x.shared, x.first, x.token, x.request), want):
            assert (host(g) == w).all(), name
    p.check()


@pytest.mark.parametrize("what,code", [("length", -4), ("page", -4), ("order", -4), ("begin", -4), ("columns", -2),
                                       ("tokens", -4)])
def test_find_errors_change_nothing(what, code):
    p = Pool([40, 41, 9], 8, [((0, 1), 5)])
    first, tokens = np.array([0, 1, 2, 4]), 4
    if what == "length":
        p.cache.lens[2] = -1
    elif what == "page":
        p.cache.tables[1, 0] = p.cache.pages
    elif what == "order":
        first[1] = 3
    elif what == "begin":
        first[0] = 1
    elif what == "columns":
        p.cache.lens[2] = 8 * p.cache.max_pages + 8
    elif what == "tokens":
        tokens = 3
    x = p.cache.prefix_arrays(tokens)
    before = [t.clone() for t in (x.leader, x.shared, x.first, x.token, x.request)]
    p.cache.find_prefixes(dev(first), x, p.cache.prefix_workspace())
    assert p.cache.error()[0] == code
    assert all(torch.equal(a, b) for a, b in zip(before, (x.leader, x.shared, x.first, x.token, x.request)))


@pytest.mark.parametrize("tokens,heads,groups,dim,rot,offset,interleaved,axes,dealt,page,step,dtype", [
    (1, 1, 1, 64, 64, 0, False, 3, False, 16, 0, BF16),
    (5, 2, 4, 128, 128, 0, True, 3, True, 8, 0, F16),
    (33, 2, 3, 128, 48, 80, False, 2, False, 1, 0, BF16),
    (12, 2, 4, 64, 32, 3, True, 4, True, 1, 3, F16),
    (3000, 1, 2, 256, 256, 0, False, 3, False, 16, 0, BF16),   # several tokens a CTA
    (7, 1, 1, 64, 2, 0, False, 1, False, 4, 0, BF16),          # one pair, one axis
])
def test_rotary_axes(tokens, heads, groups, dim, rot, offset, interleaved, axes, dealt, page, step, dtype):
    from decode_serving_gb300.paged import PagedCache, rotary_axes, rotary_frequencies
    r = np.random.default_rng(tokens)
    pool = tokens if step else -(-tokens // page) + 1
    c = PagedCache.allocate(1, 1, pool, heads, page, dim, dtype=dtype)
    gen = torch.Generator("cuda").manual_seed(tokens)
    qkv = torch.randn(tokens, (heads * groups + 2 * heads) * dim, generator=gen, device="cuda").to(dtype)
    q, k, v = qkv.split((heads * groups * dim, heads * dim, heads * dim), 1)
    pos = r.integers(-5, 1 << 20, (axes, tokens)).astype(np.int32)
    sections = [rot // 2 // axes] * (axes - 1)
    sections.append(rot // 2 - sum(sections))
    axis = rotary_axes(sections, dealt=dealt)
    assert len(axis) == rot // 2
    freq = rotary_frequencies(rot)
    slots = r.permutation(pool * page)[:tokens]
    out = torch.empty(tokens, heads * groups, dim, device="cuda", dtype=torch.float32 if step else dtype)
    c.rotary(q, k, v, dev(pos), None if step else dev(slots), freq.cuda(), out, rot_offset=offset,
             interleaved=interleaved, tokens_per_request=max(1, step), axes=axis.cuda())
    assert c.error()[0] == 0
    words = freq.numpy().view(np.uint64)
    turns = np.stack([ref.turns_of(pos[a], words[i:i + 1])[:, 0] for i, a in enumerate(axis.tolist())], 1)
    as64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    x = as64(qkv).reshape(tokens, -1, dim)
    want = ref.rotate(x[:, :heads * (groups + 1)], turns, rot, offset, interleaved, 1.0)
    w_q, w_k = want[:, :heads * groups], want[:, heads * groups:]
    if step:
        w_q = w_q.reshape(tokens // step, step, heads, groups, dim).transpose(0, 2, 1, 3, 4).reshape(tokens, -1, dim)
        slots = np.arange(tokens)
    at = torch.from_numpy(slots // page).cuda(), torch.from_numpy(slots % page).cuda()
    g_k, g_v = (as64(y[0][at[0], :, at[1]]) for y in (c.k, c.v))
    assert (g_v == x[:, heads * (groups + 1):]).all()
    # an angle off by 2^-25 turns and sincospi's own error (2 steps) act on two values each, then
    # two products and a sum in fp32: 6e-7 of the pair; the result is rounded once
    pair = 6e-7 * 2 * np.abs(x).max()
    for got, w, t in ((as64(out), w_q, out.dtype), (g_k, w_k, dtype)):
        assert (np.abs(got - w) <= pair + torch.finfo(t).eps / 2 * np.abs(w) + torch.finfo(t).smallest_normal).all()


def test_rotary_of_one_axis_is_the_plain_one():
    from decode_serving_gb300.paged import PagedCache, rotary_axes, rotary_frequencies
    got = []
    for axes in (None, rotary_axes([0, 64]).cuda()):
        c = PagedCache.allocate(1, 1, 4, 2, 16, 128)
        qkv = torch.randn(20, 8 * 128, generator=torch.Generator("cuda").manual_seed(1), device="cuda").to(BF16)
        q, k, v = qkv.split((512, 256, 256), 1)
        pos = dev(np.arange(20) * 1000)
        out = torch.empty(20, 4, 128, dtype=BF16, device="cuda")
        c.rotary(q, k, v, pos if axes is None else torch.stack([pos - 7, pos]), dev(np.arange(20)),
                 rotary_frequencies(128).cuda(), out, axes=axes)
        got.append((out, c.k, c.v))
    assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("bad", [-1, 2, 1 << 30])
def test_a_bad_axis_is_latched_and_nothing_written(bad):
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    c = PagedCache.allocate(1, 1, 300, 1, 16, 64)
    rows = torch.ones(4500, 64, dtype=BF16, device="cuda")
    axes = torch.zeros(32, dtype=torch.int32, device="cuda")
    axes[31] = bad
    out = torch.zeros(4500, 64, dtype=BF16, device="cuda")
    c.rotary(rows, rows, rows, torch.zeros(2, 4500, dtype=torch.int32, device="cuda"), dev(np.arange(4500)),
             rotary_frequencies(64).cuda(), out, axes=axes)
    assert c.error() == (-4, -1, 31)
    assert not out.any() and not c.k.any() and not c.v.any()


def test_refusals():
    from decode_serving_gb300.avsg import AvsgError
    from decode_serving_gb300.paged import Prefixes, rotary_axes, rotary_frequencies
    p = Pool([40, 41], 8, [((0, 1), 5)])
    c = p.cache
    parent, first = dev(np.array([0, 0])), dev(np.array([0, 1, 2]))
    work, pack, find = c.fork_workspace(), c.compact_workspace(), c.prefix_workspace()
    page_map, x = torch.zeros_like(c.free), c.prefix_arrays(2)
    for call in (lambda: c.fork(parent.long(), work), lambda: c.fork(parent[:1], work), lambda: c.fork(parent, work[::2]),
                 lambda: c.compact(page_map[1:], pack), lambda: c.compact(page_map, pack, tables_out=c.tables[:1]),
                 lambda: c.compact(page_map, pack, free_out=c.free.long()), lambda: c.compact(page_map, pack.int()),
                 lambda: c.compact(page_map, pack, shares_out=c.shares.cpu()),
                 lambda: c.find_prefixes(first[:2], x, find), lambda: c.find_prefixes(first, x, find, min_tokens=1 << 40),
                 lambda: Prefixes(x.leader, x.shared, x.shared, x.token, x.request),
                 lambda: Prefixes(x.leader.long(), x.shared, x.first, x.token, x.request),
                 lambda: c.find_prefixes(first, Pool([1], 8).cache.prefix_arrays(2), find),
                 lambda: rotary_axes([]), lambda: rotary_axes([3, -1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.fork(parent, work[:-256]), lambda: c.fork(parent, work[1:]),
                 lambda: c.compact(page_map, pack[:-256]), lambda: c.compact(page_map, pack[1:]),
                 lambda: c.find_prefixes(first, x, find[:-256]), lambda: c.find_prefixes(first, x, find[1:]),
                 lambda: c.find_prefixes(first, x, find, min_tokens=-1)):
        with pytest.raises(AvsgError):
            call()
    rows, out = torch.zeros(2, 8, dtype=BF16, device="cuda"), torch.zeros(2, 8, dtype=BF16, device="cuda")
    freq, axes = rotary_frequencies(8).cuda(), rotary_axes([2, 2]).cuda()
    rotary = lambda pos, axes: c.rotary(rows, rows, rows, pos, dev(np.array([0, 1])), freq, out, axes=axes)  # noqa: E731
    pos = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    for args in ((pos[0], axes), (pos[:, :1].contiguous(), axes), (pos, axes[:3]), (pos, axes.long()), (pos.long(), axes)):
        with pytest.raises(ValueError):
            rotary(*args)
    p.check()                                              # no refused call did anything
    rotary(pos, axes)
    assert c.error()[0] == 0
    assert math.isfinite(float(out.float().sum()))


def test_forks_in_a_row_do_not_reach_into_one_another():
    """Nothing is waited for between forks (their copies run beside their tables), compactions among them."""
    r = np.random.default_rng(11)
    p = Pool([100, 37, 0, 90, 5, 64] * 8, 16, spare=2500, layers=3, heads=2, dim=128, room=2)
    fork, pack = p.cache.fork_workspace(), p.cache.compact_workspace()
    page_map = torch.zeros(p.cache.pages, dtype=torch.int32, device="cuda")
    parents = [np.where(r.random(48) < 0.4, np.arange(48), r.integers(-1 if k == 20 else 0, 48, 48)) for k in range(30)]
    on_device = [dev(x) for x in parents]
    torch.cuda.synchronize()
    for k, x in enumerate(on_device):
        p.cache.fork(x, fork)
        if k % 10 == 5:
            p.cache.compact(page_map, pack)
    torch.cuda.synchronize()
    for k, x in enumerate(parents):
        p.lens, p.tables, p.free, p.count, p.shares = want_of.fork(p.lens, x, p.tables, p.free, p.count, p.shares, 16,
                                                                   p.pages)
        if k % 10 == 5:
            p.tables, p.free, p.shares, _ = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, 16, p.pages)
    p.check()


def test_the_binding_s_functions_beside_the_methods():
    from decode_serving_gb300 import avsg
    p = Pool([100, 37, 0, 90], 16, groups=[((0, 3), 4)], layers=2)
    c, pages, parent = p.cache, p.cache._pages, dev(np.array([0, 0, 3, -1]))
    n = avsg.avsg_page_fork_workspace(pages)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    avsg.avsg_page_fork(pages, parent.data_ptr(), c.shares.data_ptr(), work.data_ptr(), n)
    torch.cuda.synchronize()
    p.lens, p.tables, p.free, p.count, p.shares = want_of.fork(p.lens, host(parent), p.tables, p.free, p.count, p.shares,
                                                               16, p.pages)
    p.check()
    n = avsg.avsg_page_compact_workspace(pages)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    page_map = torch.zeros_like(c.free)
    avsg.avsg_page_compact(pages, c.shares.data_ptr(), c.shares.data_ptr(), c.tables.data_ptr(), c.free.data_ptr(),
                           page_map.data_ptr(), work.data_ptr(), n)
    torch.cuda.synchronize()
    p.tables, p.free, p.shares, where = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, 16, p.pages)
    p.check()
    assert (host(page_map) == where).all()
    first = torch.zeros(5, dtype=torch.int32, device="cuda")
    keep = dev(np.array([0, 0, 0, 0]))
    avsg.avsg_tree_keep_shared(pages, c.shares.data_ptr(), first.data_ptr(), 0, 0, keep.data_ptr(), c.lens.data_ptr(),
                               c.free_count.data_ptr())
    torch.cuda.synchronize()
    p.check()
