"""avsg_page_fork and avsg_page_compact beside calls of another cache that latch errors in the same words."""
import numpy as np
import pytest
import torch

import share_reference as want_of
from test_gpu_paged import dev, host
from test_gpu_share import Pool

pytestmark = pytest.mark.gpu


class Beside:
    """A cache, its state before a call, and another cache on another stream that latches an error of its own in
    the same error words, sooner or later while the call runs."""

    def __init__(self, p):
        self.p, self.c = p, p.cache
        self.other = Pool([40, 41], 8, seed=3)
        self.other.cache._pages.d_error = self.c._error.data_ptr()
        self.x, self.work = self.other.cache.prefix_arrays(2), self.other.cache.prefix_workspace()
        self.bad = dev(np.array([0, 2, 1]))
        self.streams = [torch.cuda.Stream() for _ in range(2)]
        c = self.c
        self.state = [c.lens, c.tables, c.free, c.free_count, c.shares, p.k, p.v]
        self.before = [t.clone() for t in self.state]

    def run(self, call, after, rounds=80):
        """Every call leaves the state before it or the one after it, whole."""
        for k in range(rounds):
            for t, b in zip(self.state, self.before):
                t.copy_(b)
            torch.cuda.synchronize()
            a, b = self.streams
            with torch.cuda.stream(b):
                torch.cuda._sleep(1 + k * 1000)            # up to 40 us and more, bounded
                self.other.cache.find_prefixes(self.bad, self.x, self.work)
            with torch.cuda.stream(a):
                call()
            torch.cuda.synchronize()
            assert self.c.error()[0] == -4
            self.c.clear_error()
            same = lambda want: [torch.equal(t, w) for t, w in zip(self.state, want)]  # noqa: E731
            assert all(same(self.before)) or all(same(after)), (k, same(self.before), same(after))
        for t, b in zip(self.state, self.before):
            t.copy_(b)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        assert self.c.error()[0] == 0 and all(torch.equal(t, w) for t, w in zip(self.state, after))


def on_device(p):
    pages = [torch.from_numpy(x).view(p.k.dtype).cuda() for x in p.pages]
    return [dev(x) for x in (p.lens, p.tables, p.free, np.array([p.count]), p.shares)] + pages


@pytest.mark.parametrize("page,requests", [(16, 48), (1, 300)])
def test_a_fork_is_whole_beside_errors_of_another_cache(page, requests):
    r = np.random.default_rng(5)
    p = Pool(r.integers(0, 6 * page, requests), page, spare=400, layers=3, heads=2, dim=64, room=2)
    parent = np.where(r.random(requests) < 0.4, np.arange(requests), r.integers(-1, requests, requests))
    b, work, at = Beside(p), p.cache.fork_workspace(), dev(parent)
    work.fill_(255)                                        # any contents
    p.lens, p.tables, p.free, p.count, p.shares = want_of.fork(p.lens, parent, p.tables, p.free, p.count, p.shares, page,
                                                               p.pages)
    b.run(lambda: p.cache.fork(at, work), on_device(p))


def test_a_fork_that_the_check_refuses_with_a_workspace_of_a_good_one():
    """The check's word of the call before is not taken for this one's."""
    p = Pool([37, 0, 20, 18], 16, groups=[((2, 3), 1)], spare=40)
    c, work = p.cache, p.cache.fork_workspace()
    p.fork([0, 0, 2, 3], work)
    p.check()
    for what in ("parent", "page", "free page", "latched"):
        state = [c.lens, c.tables, c.free, c.free_count, c.shares, p.k, p.v]
        parent = [0, 0, 2, 2]
        if what == "parent":
            parent[3] = 9
        elif what == "page":
            c.tables[2, 1] = c.pages
        elif what == "free page":
            c.free[p.count - 1] = -1
        before = [t.clone() for t in state]
        c.fork(dev(np.array(parent)), work)
        if what == "latched":
            assert c.error()[0] == 0                       # (a good one, and a bad one behind it)
            before = [t.clone() for t in state]
            c.fork(dev(np.array([9, 0, 0, 0])), work)
            c.fork(dev(np.array([0, 0, 0, 0])), work)
        assert c.error()[0] == -4
        assert all(torch.equal(t, b) for t, b in zip(state, before)), what
        c.clear_error()
        if what in ("page", "free page"):
            c.tables.copy_(dev(p.tables)), c.free.copy_(dev(p.free))
    assert host(c.lens).tolist() == [37, 37, 20, 20]


@pytest.mark.parametrize("lens,page,spare", [(list(range(1, 400, 3)), 8, 3000), (list(range(2000)), 16, 90000),
                                             ([300, 255, 1, 90] * 300, 4, 700)])
def test_a_compaction_is_whole_beside_errors_of_another_cache(lens, page, spare):
    """A pool whose lists are one cluster's work among them, and requests for many CTAs of the other kernel."""
    p = Pool(lens, page, seed=2, spare=spare)
    page_map, work = torch.zeros_like(p.cache.free), p.cache.compact_workspace()
    work.fill_(255)                                        # any contents
    b = Beside(p)
    b.state.append(page_map)
    b.before.append(page_map.clone())
    p.tables, p.free, p.shares, where = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, page, p.pages)
    b.run(lambda: p.cache.compact(page_map, work), on_device(p) + [dev(where)], rounds=60)


@pytest.mark.parametrize("requests,spare", [(3, 40), (1100, 40), (3, 70000), (1100, 70000)])
def test_a_compaction_that_is_refused_with_a_workspace_of_a_good_one(requests, spare):
    """What the checks of the call before found is not taken for this one's, of the last request too."""
    p = Pool([9 + i % 30 for i in range(requests)], 8, spare=spare)
    c, work = p.cache, p.cache.compact_workspace()
    page_map = torch.zeros_like(c.free)
    p.tables, p.free, p.shares, _ = want_of.compact(p.lens, p.tables, p.free, p.count, p.shares, 8, p.pages)
    c.compact(page_map, work)
    p.check()
    at = p.count // 2                                      # a page in use high up, so that something would move
    high, low = int(p.free[0]), int(p.tables[0, 0])
    p.free[0], p.tables[0, 0] = low, high
    for a in p.pages:
        a[:, high] = a[:, low]
    for what in ("page", "free page", "twice", "length"):
        for t, a in zip((c.lens, c.tables, c.free, c.k, c.v), (p.lens, p.tables, p.free, *p.pages)):
            t.copy_(torch.from_numpy(a).cuda().view(t.dtype) if t.dim() == 5 else dev(a))
        if what == "page":
            c.tables[requests - 1, 0] = -1
        elif what == "free page":
            c.tables[requests - 1, 0] = c.free[at]
        elif what == "twice":
            c.free[at] = c.free[1]
        elif what == "length":
            c.lens[requests - 1] = -1
        state = [c.lens, c.tables, c.free, c.free_count, c.shares, page_map, p.k, p.v]
        before = [t.clone() for t in state]
        c.compact(page_map, work)
        assert c.error()[0] == -4
        assert all(torch.equal(t, b) for t, b in zip(state, before)), what
        c.compact(page_map, work)                          # latched: nothing happens
        torch.cuda.synchronize()
        assert all(torch.equal(t, b) for t, b in zip(state, before)), what
        c.clear_error()


@pytest.mark.parametrize("spare", [60, 70000])
def test_what_a_compaction_does_with_pages_of_planned_tokens(spare):
    """They are in use and move, whole; what names them (entries behind the committed tokens, slots) does not follow."""
    p = Pool([20, 37], 8, spare=spare, layers=2, room=4)
    c = p.cache
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")  # noqa: E731
    first, slots, pos, page_map = i32(3), i32(16), i32(16), torch.zeros_like(c.free)
    c.plan(dev(np.array([9, 7])), first, slots, pos)
    planned, was = host(c.tables), host(slots)
    pages = [c.k.clone(), c.v.clone()]
    c.compact(page_map, c.compact_workspace())
    assert c.error()[0] == 0
    where, now = host(page_map), host(c.tables)
    for r, (length, new) in enumerate(((20, 9), (37, 7))):
        held, need = -(-length // 8), -(-(length + new) // 8)
        assert need > held
        assert (now[r, :held] == where[planned[r, :held]]).all()
        assert (now[r, held:] == planned[r, held:]).all()
        for x in planned[r, :need]:                        # (where the map says, whole)
            assert 0 <= where[x] < c.pages - int(c.free_count)
            assert all(torch.equal(new[:, int(where[x])], old[:, int(x)]) for new, old in zip((c.k, c.v), pages))
    assert (host(slots) == was).all()
