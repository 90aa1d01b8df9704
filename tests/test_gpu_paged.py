"""avsg_page_plan, avsg_rotary_write and avsg_tree_keep against their plain
definitions in 64 bits (tests/paged_reference.py)."""
import numpy as np
import pytest
import torch

import paged_reference as ref

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype).cuda()


def host(t):
    return t.cpu().numpy()


class Batch:
    """A cache in mid-run: requests with contexts, their pages held."""

    def __init__(self, lens, page, seed=0, spare=7, layers=1, heads=2, dim=8, dtype=BF16, room=0,
                 shift=0):
        from decode_serving_gb300.paged import PagedCache
        r = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        held = -(-(self.lens.astype(np.int64)) // page)
        width = max(1, int(held.max()) + room)
        pool = int(held.sum()) + spare
        ids = r.permutation(pool) + shift
        self.tables = r.integers(-5, 5, (len(lens), width)).astype(np.int32)  # stale entries
        at = 0
        for i, n in enumerate(held):
            self.tables[i, :n] = ids[at:at + n]
            at += int(n)
        self.free = np.full(pool, -9, np.int32)
        self.free[:pool - at] = ids[at:]
        self.count, self.page = pool - at, page
        gen = torch.Generator("cuda").manual_seed(seed)
        self.k, self.v = (torch.randn(layers, pool, heads, page, dim, generator=gen, device="cuda").to(dtype)
                          for _ in "kv")
        self.cache = PagedCache(self.k, self.v, dev(self.tables), dev(self.lens), dev(self.free),
                                dev(np.array([self.count])))

    def plan(self, new, capacity, mask=None, **kw):
        c = capacity
        self.first = torch.full((len(self.lens) + 1,), -77, dtype=torch.int32, device="cuda")
        self.slots, self.pos = (torch.full((c,), -77, dtype=torch.int32, device="cuda") for _ in "sp")
        self.cache.plan(dev(np.array(new)), self.first, self.slots, self.pos,
                        mask=None if mask is None else dev(mask, torch.int64), **kw)


def trees(new, seed):
    """Random ancestor masks, zero words for requests of more than 64 tokens."""
    r = np.random.default_rng(seed)
    out = []
    for n in new:
        words = []
        for i in range(n):
            if n > 64:
                words.append(0)
            elif i == 0:
                words.append(1)
            else:
                words.append(words[int(r.integers(max(0, i - 5), i))] | (1 << i))
        out += words
    return np.array(out, np.uint64).view(np.int64)


@pytest.mark.parametrize("lens,new,page,extra,tree", [
    ([0], [1], 16, 0, False),
    ([0], [0], 16, 3, False),
    ([15, 16, 17, 0, 31], [1, 1, 1, 33, 0], 16, 5, False),
    ([5, 9, 0], [64, 3, 1], 1, 2, True),
    ([255, 256, 1], [300, 1, 64], 256, 9, True),
    (list(range(0, 1026, 2)), [(i * 7) % 5 for i in range(513)], 8, 100, True),
    ([3, 700], [5000, 4096], 16, 1, False),
    ([0] * 8192, [1] * 8192, 2, 0, False),
])
def test_plan(lens, new, page, extra, tree):
    total = sum(new)
    b = Batch(lens, page, seed=len(lens), spare=total // page + len(lens) + 4, room=max(new) // page + 2)
    mask = trees(new, 5) if tree else None
    b.plan(new, total + extra, mask)
    want = ref.plan(b.lens, np.array(new), b.tables, b.free, b.count, page, total + extra, mask)
    got = (b.first, b.slots, b.pos, b.cache.tables, b.cache.free_count)
    for name, g, w in zip(("first", "slots", "pos", "tables", "count"), got, want):
        assert (host(g) == w).all(), name
    assert b.cache.error()[0] == 0
    # the context of each request and the stack are as they were
    assert (host(b.cache.lens) == b.lens).all() and (host(b.cache.free) == b.free).all()


def test_plan_leaves_the_count_alone_when_given_another():
    b = Batch([3, 40], 16)
    out = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.plan([20, 1], 21, free_count_out=out)
    assert host(out)[0] == b.count - 1 and host(b.cache.free_count)[0] == b.count


@pytest.mark.parametrize("what,code,request_", [
    ("pages", -2, -1), ("columns", -2, 1), ("entries", -2, -1), ("length", -4, 0), ("new", -4, 1),
    ("held page", -4, 0), ("free page", -4, -1), ("count", -4, -1), ("overflow", -2, 0),
])
def test_plan_errors_change_nothing_and_stay(what, code, request_):
    b = Batch([3, 40], 16, room=2, spare=4)
    new, cap = [20, 30], 64
    if what == "pages":
        new = [20, 33]
        b.cache.free_count.fill_(1)
    elif what == "columns":
        new = [1, 16 * 5]
    elif what == "entries":
        cap = 49
    elif what == "length":
        b.cache.lens[0] = -3
    elif what == "new":
        new = [1, -1]
    elif what == "held page":
        b.cache.tables[0, 0] = b.cache.free.numel()
    elif what == "free page":
        b.cache.free[b.count - 1] = -1
    elif what == "count":
        b.cache.free_count.fill_(b.cache.free.numel() + 1)
    elif what == "overflow":
        new = [2**31 - 1, 2**31 - 1]
    before = [host(x).copy() for x in (b.cache.tables, b.cache.free, b.cache.free_count)]
    b.plan(new, cap)
    assert b.cache.error()[:2] == (code, request_)
    for x in (b.first, b.slots, b.pos):
        assert (host(x) == -77).all()
    for x, y in zip((b.cache.tables, b.cache.free, b.cache.free_count), before):
        assert (host(x) == y).all()
    # latched: a good step does nothing until the error is cleared
    b = b if what in ("pages", "columns", "entries", "new", "overflow") else None
    if b is not None:
        b.cache.free_count.fill_(b.count)
        b.plan([1, 1], 2)
        assert (host(b.slots) == -77).all() and b.cache.error()[0] == code
        b.cache.clear_error()
        b.plan([1, 1], 2)
        assert b.cache.error()[0] == 0 and (host(b.slots) >= 0).all()


def test_plan_and_keep_refuse_short_masks_and_paths():
    b = Batch([3, 40], 16, room=2, spare=6)
    b.plan([5, 6], 11, mask=trees([5, 5], 1))                  # 10 words for 11 tokens
    assert b.cache.error()[0] == -2 and (host(b.slots) == -77).all()
    b.cache.clear_error()
    b.plan([5, 6], 11)
    b.cache.keep(b.first, dev(np.arange(10)), dev(np.array([1, 1])))
    assert b.cache.error()[:2] == (-2, 1) and (host(b.cache.lens) == b.lens).all()


def random_paths(new, kept, seed):
    r = np.random.default_rng(seed)
    out = []
    for n, k in zip(new, kept):
        row = list(range(n))
        row[:max(k, 0)] = sorted(r.choice(n, max(k, 0), replace=False).tolist()) if n else []
        out += row
    return np.array(out, np.int32)


@pytest.mark.parametrize("lens,new,kept,page,layers,heads,dim,dtype", [
    ([0], [1], [1], 16, 1, 1, 8, BF16),
    ([7], [64], [64], 16, 1, 2, 64, BF16),
    ([15, 3, 0, 20], [9, 64, 5, 0], [4, 17, 0, 0], 16, 3, 2, 64, F16),
    ([5, 6, 7], [30, 30, 30], [-1, 29, -1], 4, 2, 3, 24, BF16),
    ([100, 0, 9], [200, 1, 64], [150, -1, 1], 1, 2, 1, 128, F16),
    ([1] * 700, [3] * 700, [i % 5 - 1 if i % 5 < 5 else 0 for i in range(700)], 8, 1, 1, 8, BF16),
])
@pytest.mark.parametrize("in_place", [True, False])
def test_plan_then_keep(lens, new, kept, page, layers, heads, dim, dtype, in_place):
    total = sum(new)
    b = Batch(lens, page, seed=7, spare=total // page + len(lens) + 4, room=max(new) // page + 2,
              layers=layers, heads=heads, dim=dim, dtype=dtype)
    b.plan(new, total)
    lens0, first, tables, free = (host(x).copy() for x in (b.cache.lens, b.first, b.cache.tables, b.cache.free))
    count = int(host(b.cache.free_count)[0])
    bits = [host(x.view(torch.int16)).copy() for x in (b.k, b.v)]
    path = random_paths(new, kept, 3)
    out = {} if in_place else dict(lens_out=torch.empty_like(b.cache.lens),
                                   free_count_out=torch.empty_like(b.cache.free_count))
    b.cache.keep(b.first, dev(path), dev(np.array(kept)), **out)
    w_lens, w_free, w_count = ref.keep(lens0, first, path, kept, tables, free, count, page, bits)
    g_lens = out.get("lens_out", b.cache.lens)
    g_count = out.get("free_count_out", b.cache.free_count)
    assert b.cache.error()[0] == 0
    assert (host(g_lens) == w_lens).all() and int(host(g_count)[0]) == w_count
    assert (host(b.cache.free) == w_free).all()
    for x, w in zip((b.k, b.v), bits):
        assert (host(x.view(torch.int16)) == w).all()
    if not in_place:
        assert (host(b.cache.lens) == lens0).all() and int(host(b.cache.free_count)[0]) == count


def test_a_rejected_step_gives_the_stack_back():
    b = Batch([3, 40, 0], 16, spare=30, room=8)
    free = host(b.cache.free).copy()
    b.plan([64, 17, 33], 114)
    b.cache.keep(b.first, None, dev(np.zeros(3)))
    assert (host(b.cache.free) == free).all() and int(host(b.cache.free_count)[0]) == b.count
    assert (host(b.cache.lens) == b.lens).all()


@pytest.mark.parametrize("what", ["same twice", "decreasing", "behind", "negative", "too many", "below -1",
                                  "page", "count"])
def test_keep_errors_change_nothing(what):
    b = Batch([3, 40], 16, room=3, spare=9, layers=2)
    b.plan([20, 8], 28)
    path, kept = np.arange(28, dtype=np.int32), np.array([3, 4])
    path[20:28] = np.arange(8)
    path[20:24] = [0, 2, 5, 7]
    if what == "same twice":
        path[20:24] = [0, 2, 2, 7]
    elif what == "decreasing":
        path[20:24] = [0, 5, 2, 7]
    elif what == "behind":
        path[23] = 8
    elif what == "negative":
        path[20] = -1
    elif what == "too many":
        kept[1] = 9
    elif what == "below -1":
        kept[0] = -2
    elif what == "page":
        b.cache.tables[0, 1] = 1 << 20
    elif what == "count":
        b.cache.free_count.fill_(b.cache.free.numel())
    before = [host(x).copy() for x in (b.cache.lens, b.cache.free, b.cache.free_count,
                                       b.k.view(torch.int16), b.v.view(torch.int16))]
    b.cache.keep(b.first, dev(path), dev(kept))
    assert b.cache.error()[0] == (-2 if what == "count" else -4)
    for x, y in zip((b.cache.lens, b.cache.free, b.cache.free_count, b.k.view(torch.int16),
                     b.v.view(torch.int16)), before):
        assert (host(x) == y).all()


# Rotary.  fp32 error before the final rounding, relative to |a| + |b| times the magnitude: the
# angle (at most half a turn) rounded to fp32, pi * 2^-24 = 1.9e-7; sincospif, 2 ulp, 1.2e-7; the
# factor's, two products' and the sum's roundings, 4 * 2^-24 = 2.4e-7.  Together below 6e-7.
FP32 = 6e-7


def rotary_bound(x, y, rot, magnitude, dtype):
    """Allowed |difference| from the exact y: fp32 arithmetic, then half a step of the type
    (or half the smallest subnormal step)."""
    parts = 2 * np.abs(x).max(-1, keepdims=True) * magnitude * FP32
    f = torch.finfo(dtype)
    return parts + f.eps / 2 * (np.abs(y) + parts) + f.smallest_normal * f.eps / 2


@pytest.mark.parametrize("tokens,heads,groups,dim,rot,offset,interleaved,dtype,page,out32,far", [
    (1, 1, 1, 8, 8, 0, False, BF16, 1, False, 100),
    (8, 8, 4, 128, 128, 0, False, BF16, 16, False, 65536),
    (7, 2, 3, 64, 32, 32, True, F16, 8, False, 1 << 20),
    (5, 1, 5, 96, 24, 8, False, F16, 4, True, 1 << 20),       # half of 12: 8-byte chunks
    (5, 2, 1, 40, 6, 3, True, BF16, 2, False, 4096),          # odd offset: single values
    (3, 2, 2, 256, 0, 0, False, BF16, 32, True, 64),          # nothing rotated
    (2600, 2, 2, 64, 64, 0, False, F16, 16, False, 1 << 20),  # several tokens per CTA
    (2431, 1, 3, 72, 40, 16, True, BF16, 64, False, 1 << 20),
])
def test_rotary(tokens, heads, groups, dim, rot, offset, interleaved, dtype, page, out32, far):
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    r = np.random.default_rng(tokens + dim)
    pool = -(-tokens // page) + 2
    cache = PagedCache.allocate(1, 1, pool, heads, page, dim, layers=2, dtype=dtype)
    cache.k.fill_(7.0)
    cache.v.fill_(7.0)
    hq = heads * groups
    # one projection's rows: q, k and v lie beside each other, with something else between
    wide = torch.randn(tokens, (hq + 2 * heads) * dim + 24, device="cuda",
                       generator=torch.Generator("cuda").manual_seed(dim)).to(dtype)
    q, k = wide[:, :hq * dim], wide[:, hq * dim:(hq + heads) * dim]
    v = wide[:, (hq + heads) * dim + 24:]
    pos = r.integers(0, far, tokens).astype(np.int32)
    slots = r.permutation(pool * page)[:tokens].astype(np.int32)
    if tokens > 2:
        slots[tokens // 2] = -1
    freq = rotary_frequencies(rot, factor=2.0).cuda() if rot else torch.zeros(0, dtype=torch.int64, device="cuda")
    out = torch.full((tokens, hq, dim), 5.0, dtype=torch.float32 if out32 else dtype, device="cuda")
    cache.rotary(q, k, v, dev(pos), dev(slots), freq, out, layer=1, rot_offset=offset,
                 interleaved=interleaved, magnitude=1.25)
    assert cache.error()[0] == 0
    inv = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(rot, 1)) / 2.0
    turns = pos[:, None].astype(np.float64) * inv / (2 * np.pi)
    live = slots >= 0
    as64 = lambda t, h: t.double().cpu().numpy().reshape(tokens, h, dim)  # noqa: E731
    xq = as64(q, hq)
    yq = ref.rotate(xq, turns, rot, offset, interleaved, 1.25)
    gq = as64(out, hq)
    bound = rotary_bound(xq, yq, rot, 1.25, torch.float32 if out32 else dtype)
    assert (np.abs(gq - yq) <= bound)[live].all()
    assert (gq[~live] == 5.0).all()                            # padding: left as it was
    xk = as64(k, heads)
    yk = ref.rotate(xk, turns, rot, offset, interleaved, 1.25)
    rows = lambda x: x[1].transpose(1, 2).reshape(pool * page, heads, dim)  # noqa: E731
    gk, gv = (rows(x).double().cpu().numpy() for x in (cache.k, cache.v))
    assert (np.abs(gk[slots[live]] - yk[live]) <= rotary_bound(xk, yk, rot, 1.25, dtype)[live]).all()
    assert (gv[slots[live]] == as64(v, heads)[live]).all()
    rest = np.setdiff1d(np.arange(pool * page), slots[live])
    assert (gk[rest] == 7.0).all() and (gv[rest] == 7.0).all()
    assert (cache.k[0] == 7.0).all() and (cache.v[0] == 7.0).all()   # the other layer


def test_rotary_angles_are_exact_at_the_ends_of_int32():
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    pos = np.array([0, 1, 2**31 - 1, -1, -2**31, 123456789], np.int32)
    cache = PagedCache.allocate(1, 1, len(pos), 1, 1, 64)
    freq = rotary_frequencies(64)
    x = torch.randn(len(pos), 64, device="cuda").to(BF16)
    out = torch.empty(len(pos), 64, dtype=torch.float32, device="cuda")
    cache.rotary(x, x, x, dev(pos), None, freq.cuda(), out)
    x64 = x.double().cpu().numpy()[:, None]
    want = ref.rotate(x64, ref.turns_of(pos, freq.numpy().view(np.uint64)), 64, 0, False, 1.0)
    bound = rotary_bound(x64, want, 64, 1.0, torch.float32)
    assert (np.abs(out.double().cpu().numpy()[:, None] - want) <= bound).all()


def test_rotary_in_place_and_the_step_layout():
    """q in place equals q elsewhere; three tokens per request give avsg_step's layout."""
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    tokens, heads, groups, dim = 12, 2, 4, 64
    cache = PagedCache.allocate(1, 1, tokens, heads, 1, dim)
    freq = rotary_frequencies(dim).cuda()
    q = torch.randn(tokens, heads * groups, dim, device="cuda").to(BF16)
    k, v = (torch.randn(tokens, heads * dim, device="cuda").to(BF16) for _ in "kv")
    pos = dev(np.arange(tokens) * 1001)
    flat, step = (torch.empty(tokens, heads * groups, dim, dtype=torch.float32, device="cuda") for _ in "ab")
    cache.rotary(q, k, v, pos, None, freq, flat)
    cache.rotary(q, k, v, pos, None, freq, step, tokens_per_request=3)
    want = flat.reshape(4, 3, heads, groups, dim).transpose(1, 2).contiguous()
    assert torch.equal(step.reshape(want.shape), want)
    cache.rotary(q, k, v, pos, None, freq, q)
    assert torch.equal(q, flat.to(BF16))


def test_rotary_skips_and_latches_a_slot_past_the_pool():
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    cache = PagedCache.allocate(1, 1, 2, 1, 4, 64)
    freq = rotary_frequencies(64).cuda()
    x = torch.randn(3, 64, device="cuda").to(BF16)
    out = torch.zeros(3, 64, dtype=BF16, device="cuda")
    cache.rotary(x, x, x, dev(np.arange(3)), dev(np.array([1, 8, 2])), freq, out)
    assert cache.error() == (-4, -1, 1)
    assert (out[1] == 0).all()                                 # the others: written or not
    rows = cache.v[0, :, 0].reshape(8, 64)
    assert all((rows[i] == 0).all() for i in (0, 3, 4, 5, 6, 7))
    out.zero_()
    cache.rotary(x, x, x, dev(np.arange(3)), dev(np.array([1, 3, 2])), freq, out)
    assert (out == 0).all()                                    # latched
    cache.clear_error()
    cache.rotary(x, x, x, dev(np.arange(3)), dev(np.array([1, 3, 2])), freq, out)
    assert cache.error()[0] == 0 and (out[1] != 0).any()


def test_refusals_of_the_cache():
    from decode_serving_gb300.avsg import AvsgError
    from decode_serving_gb300.paged import PagedCache
    c = PagedCache.allocate(2, 4, 8, 2, 16, 64)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    f = torch.zeros(32, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError):
        c.plan(i(3), i(3), i(2), i(2))
    with pytest.raises(ValueError):
        c.plan(i(2).cpu(), i(3), i(2), i(2))
    with pytest.raises(ValueError):
        c.plan(i(2).long(), i(3), i(2), i(2))
    with pytest.raises(ValueError):
        c.plan(i(2), i(3), i(4)[::2], i(2))
    with pytest.raises(ValueError):
        c.keep(i(3), None, i(3))
    with pytest.raises(ValueError):
        c.rotary(x.half(), x, x, i(2), i(2), f, x)
    with pytest.raises(ValueError):
        c.rotary(x[:, ::2], x, x, i(2), i(2), f, x)
    with pytest.raises(ValueError):
        c.rotary(x, x[:1], x, i(2), i(2), f, x)
    with pytest.raises(ValueError):
        c.rotary(x, x, x, i(2), i(2), f, x[:1])
    with pytest.raises(AvsgError):
        c.rotary(x, x, x, i(2), i(2), f, x, layer=1)
    with pytest.raises(AvsgError):
        c.rotary(x, x, x, i(2), i(2), f, x, rot_offset=2)
    with pytest.raises(ValueError):
        PagedCache(c.k, c.v, c.tables, c.lens, c.free[:4], c.free_count)


@pytest.mark.parametrize("page_of,path", [
    (2, [0, 2, 5, 7]),                                 # the page of both the rows and their places
    (2, [0, 1, 8, 11]),                                # of the places alone: the rows lie in the next one
    (3, [0, 1, 8, 11, 12, 13, 14, 15, 16, 17]),        # of rows and, in part, places; a page is returned behind it
])
def test_keep_checks_the_pages_that_stay_before_it_changes_anything(page_of, path):
    b = Batch([3, 40], 16, room=3, spare=9, layers=2)
    b.plan([20, 26], 46)
    paths = np.zeros(46, np.int32)
    paths[:3] = [0, 5, 9]                              # request 0 moves rows of its own
    paths[20:20 + len(path)] = path
    b.cache.tables[1, page_of] = 1 << 20
    state = (b.cache.lens, b.cache.free, b.cache.free_count, b.k.view(torch.int16), b.v.view(torch.int16))
    before = [host(x).copy() for x in state]
    b.cache.keep(b.first, dev(paths), dev(np.array([3, len(path)])))
    assert b.cache.error()[:2] == (-4, 1)
    for x, y in zip(state, before):
        assert (host(x) == y).all()


def test_keep_reads_no_page_whose_rows_stay():
    """A path that keeps its rows where they are asks nothing of the pages that stay."""
    b = Batch([3, 40], 16, room=3, spare=9)
    b.plan([20, 8], 28)
    b.cache.tables[1, 2] = 1 << 20
    b.cache.keep(b.first, dev(np.concatenate([np.arange(20), np.arange(8)])), dev(np.array([3, 4])))
    assert b.cache.error()[0] == 0 and host(b.cache.lens).tolist() == [6, 44]


def test_error_waits_for_every_stream():
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    cache = PagedCache.allocate(1, 1, 2, 1, 4, 64)
    freq = rotary_frequencies(64).cuda()
    x = torch.randn(3, 64, device="cuda").to(BF16)
    out = torch.zeros(3, 64, dtype=BF16, device="cuda")
    pos, slots = dev(np.arange(3)), dev(np.array([1, 8, 2]))      # slot 8 is past the pool
    side = torch.cuda.Stream()
    cache.rotary(x, x, x, pos, dev(np.arange(3)), freq, out)      # (the first launch loads the kernel)
    with torch.cuda.stream(side):
        torch.cuda._sleep(1000)
    torch.cuda.synchronize()
    assert cache.error()[0] == 0
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)                            # about 0.1 s
    cache.rotary(x, x, x, pos, slots, freq, out, stream=side.cuda_stream)
    assert cache.error() == (-4, -1, 1)


def test_a_new_cache_serves_any_stream():
    """Its error word is zero for calls on every stream, not only behind the stream it was made on."""
    from decode_serving_gb300.paged import PagedCache
    old = PagedCache.allocate(1, 2, 2, 1, 16, 64)
    i32 = lambda n: torch.full((n,), -7, dtype=torch.int32, device="cuda")  # noqa: E731
    new, first, slots, pos = dev(np.array([3])), i32(2), i32(3), i32(3)
    old.plan(new, first, slots, pos)                   # (loads the kernel)
    side = torch.cuda.Stream()
    keep = [torch.full((4,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]
    slots.fill_(-7)
    torch.cuda.synchronize()
    del keep                                           # (memory of such words is given out again)
    torch.cuda._sleep(200_000_000)
    cache = PagedCache(old.k, old.v, old.tables, old.lens, old.free, old.free_count)
    cache.plan(new, first, slots, pos, stream=side.cuda_stream)
    assert cache.error()[0] == 0 and host(slots).tolist() == [16, 17, 18]


def test_the_binding_functions_make_the_same_calls():
    """avsg.py's functions, which take structures and addresses, beside the cache's methods."""
    from decode_serving_gb300 import avsg as C
    from decode_serving_gb300.paged import PagedCache, rotary_frequencies
    requests, heads, groups, dim = 3, 2, 4, 64
    new, kept = dev(np.array([3, 1, 5])), dev(np.array([2, 0, 3]))
    mask, path = dev(trees([3, 1, 5], 2), torch.int64), dev(np.array([0, 2, 0, 0, 0, 2, 4, 0, 0]))
    gen = torch.Generator("cuda").manual_seed(4)
    qkv = torch.randn(9, (groups + 2) * heads * dim, generator=gen, device="cuda").to(BF16)
    freq = rotary_frequencies(dim).cuda()
    a, b = groups * heads * dim, heads * dim
    q, k, v = qkv.split((a, b, b), 1)
    states = []
    for how in ("methods", "functions"):
        c = PagedCache.allocate(requests, 4, 8, heads, 8, dim)
        first, slots, pos = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (4, 9, 9))
        q_rot = torch.zeros(9, groups * heads, dim, dtype=BF16, device="cuda")
        out, work = torch.zeros_like(q_rot), c.attention_workspace(groups, 5)
        lse = torch.zeros(9, groups * heads, device="cuda")
        if how == "methods":
            c.plan(new, first, slots, pos, mask=mask)
            c.rotary(q, k, v, pos, slots, freq, q_rot)
            c.attend(q_rot, first, out, 5, work, mask=mask, lse=lse, softcap=20.0)
            c.keep(first, path, kept)
        else:
            error = torch.zeros(4, dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()
            p = C.avsg_pages(requests, 1, 8, heads, 8, dim, 4, C.AVSG_BF16, c.k.data_ptr(), c.v.data_ptr(),
                             c.tables.data_ptr(), c.lens.data_ptr(), c.free.data_ptr(), c.free_count.data_ptr(),
                             error.data_ptr())
            C.avsg_page_plan(p, new.data_ptr(), mask.data_ptr(), 9, 9, first.data_ptr(), slots.data_ptr(),
                             pos.data_ptr(), c.free_count.data_ptr())
            width = qkv.shape[1]
            C.avsg_rotary_write(p, C.avsg_rotary(
                num_tokens=9, num_q_heads=groups * heads, rot_dim=dim, tokens_per_request=1, q_stride=width,
                k_stride=width, v_stride=width, magnitude=1.0, d_q=q.data_ptr(), d_k=k.data_ptr(), d_v=v.data_ptr(),
                d_freq=freq.data_ptr(), d_pos=pos.data_ptr(), d_slot=slots.data_ptr(), d_q_out=q_rot.data_ptr()))
            assert C.avsg_tree_attention_workspace(p, groups, 5) == work.numel()
            C.avsg_tree_attention(p, C.avsg_tree(
                num_tokens=9, q_per_kv=groups, max_new=5, softcap=20.0, q_stride=a, d_q=q_rot.data_ptr(),
                d_first=first.data_ptr(), d_mask=mask.data_ptr(), d_out=out.data_ptr(), d_lse=lse.data_ptr(),
                d_work=work.data_ptr(), work_bytes=work.numel()))
            C.avsg_tree_keep(p, first.data_ptr(), path.data_ptr(), 9, kept.data_ptr(), c.lens.data_ptr(),
                             c.free_count.data_ptr())
            with pytest.raises(C.AvsgError):
                C.avsg_tree_keep(p, 0, path.data_ptr(), 9, kept.data_ptr(), c.lens.data_ptr(), c.free_count.data_ptr())
            assert host(error)[0] == 0
        states.append([x.clone() for x in (first, slots, pos, q_rot, out, lse, c.k, c.v, c.tables, c.lens, c.free,
                                           c.free_count)])
        assert host(c.lens).tolist() == [2, 0, 3]
    assert all(torch.equal(x, y) for x, y in zip(*states))


def test_shapes_and_numbers_that_do_not_fit_are_refused_as_such():
    """ValueError for shapes and whole numbers, AvsgError for what the library refuses: not whatever
    error a bad shape or a number too large would run into."""
    from decode_serving_gb300.avsg import AvsgError
    from decode_serving_gb300.paged import PagedCache
    c = PagedCache.allocate(2, 4, 8, 2, 16, 64)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros(2, 128, dtype=BF16, device="cuda")
    f = torch.zeros(32, dtype=torch.int64, device="cuda")
    work = c.attention_workspace(1, 1)
    for bad in (x[0], x[0, 0], x.reshape(2, 2, 32, 2), x[:, :65]):
        with pytest.raises(ValueError):
            c.rotary(bad, x, x, i(2), i(2), f, x)
        with pytest.raises(ValueError):
            c.rotary(x, bad, x, i(2), i(2), f, torch.empty_like(x))
        with pytest.raises(ValueError):
            c.attend(bad, i(3), torch.empty_like(x), 1, work)
    for kw in (dict(layer=1 << 40), dict(rot_offset=-(1 << 40)), dict(tokens_per_request=1 << 31)):
        with pytest.raises(ValueError):
            c.rotary(x, x, x, i(2), i(2), f, torch.empty_like(x), **kw)
    for kw in (dict(layer=1 << 40), dict(window=1 << 31)):
        with pytest.raises(ValueError):
            c.attend(x, i(3), torch.empty_like(x), 1, work, **kw)
    with pytest.raises(ValueError):
        c.attend(x, i(3), torch.empty_like(x), 1 << 31, work)
    for kw in (dict(softcap=1e39), dict(scale=1e39), dict(scale=float("nan"))):
        with pytest.raises(AvsgError):
            c.attend(x, i(3), torch.empty_like(x), 1, work, **kw)
    with pytest.raises(AvsgError):
        c.rotary(x, x, x, i(2), i(2), f, torch.empty_like(x), magnitude=float("nan"))
    with pytest.raises(ValueError):
        PagedCache(c.k, c.v, c.tables, c.lens[0], c.free, c.free_count)
    assert c.error()[0] == 0


def test_a_cache_made_in_a_capture():
    """Its error word is zeroed by each replay, behind which the graph's calls run."""
    from decode_serving_gb300.paged import PagedCache
    old = PagedCache.allocate(1, 2, 2, 1, 16, 64)
    first, slots, pos = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (2, 3, 3))
    new, count = dev(np.array([3])), torch.zeros(1, dtype=torch.int32, device="cuda")
    old.plan(new, first, slots, pos, free_count_out=count)
    want = host(slots).copy()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        cache = PagedCache(old.k, old.v, old.tables, old.lens, old.free, old.free_count)
        cache.plan(new, first, slots, pos, free_count_out=count)
    for _ in range(2):
        slots.zero_()
        graph.replay()
        assert cache.error()[0] == 0 and (host(slots) == want).all()
