"""avsg_prefix_attention against its definition in 64 bits (that of the tree
attention: the groups change no result), alone and in steps of requests that
share pages."""
import math

import numpy as np
import pytest
import torch

import share_reference as want_of
from test_gpu_paged import BF16, F16, dev, host, trees
from test_gpu_tree_attention import Step

pytestmark = pytest.mark.gpu


class Shared(Step):
    """A planned step of requests that share prefixes: groups of (members, pages)."""

    def __init__(self, lens, new, page, heads, groups, dim, dtype, tree, share, pool=0, least=1, **kw):
        super().__init__(lens, new, page, heads, groups, dim, dtype, tree, **kw)
        if pool:                                           # room that makes contexts look long
            from decode_serving_gb300.paged import PagedCache
            old, c = self.k, self.cache
            self.k, self.v = (torch.cat([x, torch.zeros(x.shape[0], pool, *x.shape[2:], dtype=dtype, device="cuda")], 1)
                              for x in (self.k, self.v))
            free = torch.zeros(self.k.shape[1], dtype=torch.int32, device="cuda")
            free[:old.shape[1]] = c.free
            self.cache = PagedCache(self.k, self.v, c.tables, c.lens, free, c.free_count)
        t = self.cache.tables
        for members, pages in share:
            for m in members[1:]:
                t[m, :pages] = t[members[0], :pages]
        self.x = self.cache.prefix_arrays(max(1, self.total))
        self.find(least)

    def find(self, least=1):
        self.cache.find_prefixes(self.first, self.x, self.cache.prefix_workspace(), min_tokens=least)

    def attend(self, work=None, most=None, q=None, **kw):
        most = max(max(self.new), 1) if most is None else most
        if work is None:
            work = self.cache.attend_prefixes_workspace(self.groups, most, len(self.q))
        self.cache.attend_prefixes(self.q if q is None else q, self.first, self.x, self.out, most, work,
                                   mask=self.dmask, lse=self.lse, layer=self.layer, **kw)


@pytest.mark.parametrize("lens,new,page,heads,groups,dim,dtype,tree,share", [
    ([16], [1], 16, 1, 1, 128, BF16, False, []),                                  # nobody shares
    ([16, 16], [1, 1], 16, 1, 1, 128, BF16, False, [((0, 1), 1)]),                # a prefix of one page, nothing after it
    ([17, 40], [1, 1], 1, 1, 1, 64, F16, False, [((0, 1), 17)]),                  # pages of one token
    ([127, 128, 129, 300], [1, 1, 1, 1], 1, 2, 4, 128, BF16, False, [((0, 1, 2, 3), 127)]),
    ([1000, 1010, 1999, 1000], [1, 1, 1, 1], 16, 1, 4, 128, BF16, False, [((0, 1, 2, 3), 62)]),
    ([300, 31, 305, 0, 299, 64], [3, 1, 4, 2, 0, 9], 8, 2, 3, 128, F16, True, [((0, 2, 4), 37), ((1, 5), 3)]),
    ([700, 640, 20, 900], [29, 64, 5, 40], 32, 2, 5, 64, F16, True, [((0, 1, 3), 20)]),   # several m-tiles
    ([100, 257, 260], [11, 2, 30], 32, 1, 16, 256, BF16, True, [((1, 2), 8)]),
    ([77, 80], [9, 9], 1, 2, 3, 256, F16, True, [((0, 1), 70)]),
    ([256, 10, 333, 512], [300, 129, 70, 1], 64, 1, 2, 128, F16, False, [((0, 2, 3), 4)]),  # prompt chunks behind a prompt
    ([600, 512], [70, 12], 256, 1, 64, 64, BF16, True, [((0, 1), 2)]),                      # a chain beside a tree
    ([40 + i for i in range(150)], [1 + i % 3 for i in range(150)], 16, 1, 2, 64, BF16, False,
     [(tuple(range(i, 150, 5)), 1 + i % 2) for i in range(4)]),
])
@pytest.mark.parametrize("pool", [0, 9000])
def test_attention(lens, new, page, heads, groups, dim, dtype, tree, share, pool):
    """On either kernel: a large pool makes few rows take the tensor cores too."""
    pool = pool * len(lens) // page if page >= 8 else 0
    s = Shared(lens, new, page, heads, groups, dim, dtype, tree, share, pool=pool, layers=2, extra=2)
    shared = host(s.x.shared)
    assert all((shared[list(m)] > 0).any() for m, _ in share)
    s.attend()
    s.check()
    assert (s.out[s.total:] == 3.0).all() and (s.lse[s.total:] == 3.0).all()


@pytest.mark.parametrize("dim,dtype,page", [(64, F16, 16), (128, BF16, 16), (256, BF16, 16), (128, F16, 4)])
@pytest.mark.parametrize("kw", [
    dict(cap=30.0), dict(window=100), dict(slopes=True), dict(window=1), dict(window=400), dict(scale=0.3),
    dict(cap=5.0, window=270, slopes=True, scale=0.2),
])
@pytest.mark.parametrize("tree", [True, False])
def test_caps_windows_and_slopes(dim, dtype, page, kw, tree):
    """Positions are each row's own, wherever its group's rows lie."""
    heads, groups = 2, 4
    s = Shared([256, 500, 366, 390, 129], [12, 9, 70 if not tree else 30, 1, 3], page, heads, groups, dim, dtype, tree,
               [((0, 1, 3), 256 // page), ((2, 4), 128 // page)])
    kw = dict(kw)
    slopes = None
    if kw.pop("slopes", False):
        slopes = (2.0 ** (-np.arange(1, heads * groups + 1) / 2.0)).astype(np.float32)
    s.attend(scale=kw.get("scale", 0.0), softcap=kw.get("cap", 0.0), window=kw.get("window", 0),
             slopes=None if slopes is None else dev(slopes, torch.float32))
    s.check(slopes=slopes, **kw)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("groups,most,window", [(1, 8, 50), (4, 8, 50), (8, 16, 50), (16, 16, 30), (4, 8, 0)])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, groups, most, window, cap):
    """NaN and infinities in prefixes out of the window of some rows, in drafts of other branches
    and behind the last token; rows that see nothing of their own."""
    s = Shared([40, 0, 75, 47], [most, 7, 3, 5], 16, 2, groups, 64, dtype, True, [((0, 2, 3), 2)])
    s.mask[most] = 0                                   # request 1 has no context: its first row is empty
    s.mask[most + 3] = -2**63                          # a bit past its new tokens
    s.dmask = dev(s.mask, torch.int64)
    tables = host(s.cache.tables)
    for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new)):
        for p in range(length + n, -(-(length + n) // 16) * 16):
            for x in (s.k, s.v):
                x[0, int(tables[r, p // 16]), :, p % 16] = math.nan
    page = lambda r, p: (0, int(tables[r, p // 16]), slice(None), p % 16)  # noqa: E731
    s.v[page(0, 42)] = math.inf                        # draft 2 of request 0: seen by its branch only
    s.k[page(0, 43)] = math.nan                        # draft 3
    if window:
        s.v[page(2, 3)] = math.nan                     # of the prefix: in some members' windows
        s.v[page(2, 20)] = -math.inf
    s.attend(window=window, softcap=cap)
    s.check(window=window, cap=cap)


def test_a_prefix_whose_values_are_not_finite_reaches_its_rows():
    s = Shared([200, 190, 60], [2, 5, 1], 16, 1, 4, 128, BF16, True, [((0, 1), 11)])
    s.v[0, int(host(s.cache.tables)[0, 2]), 0, 5, 7] = math.inf
    s.attend()
    s.check()


def test_rows_of_any_stride_and_reused_workspace():
    s = Shared([300, 290], [5, 8], 16, 2, 4, 128, BF16, True, [((0, 1), 16)])
    wide = torch.zeros(s.total, 8 * 128 + 66, dtype=BF16, device="cuda")
    wide[:, 66:] = s.q.reshape(s.total, -1)
    work = s.cache.attend_prefixes_workspace(4, 8, s.total)
    work.fill_(255)                                    # any contents
    s.attend(work=work, q=wide[:, 66:])
    s.check()
    a, b = s.out.clone(), s.lse.clone()
    s.out.fill_(0)
    s.attend(work=work)
    assert torch.equal(a, s.out) and torch.equal(b, s.lse)   # the same bits again


@pytest.mark.parametrize("dim,dtype,requests,new,pages", [
    (128, BF16, 70, 1, 300), (128, F16, 20, 16, 130), (64, F16, 33, 9, 200), (256, BF16, 40, 3, 70),
])
def test_groups_of_many_rows(dim, dtype, requests, new, pages):
    """Several m-tiles of 256 rows over a prefix that many CTAs share, beside requests alone."""
    r = np.random.default_rng(requests)
    lens = [pages * 16 + int(x) for x in r.integers(0, 400, requests)] + [5, 1700, 130]
    order = r.permutation(requests)
    s = Shared(lens, [new] * len(lens), 16, 2, 8, dim, dtype, new > 1, [(tuple(sorted(order[: requests - 5])), pages)])
    s.attend()
    s.check(only=set(range(0, requests, 9)) | {requests, requests + 1, requests + 2})


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, BF16)])
def test_many_groups_of_short_prefixes(dim, dtype):
    """Many units in a CTA's share: whole ones beside ones that cross CTAs."""
    n = 600
    lens = [48 + (i * 37) % 200 for i in range(n)]
    s = Shared(lens, [1 + i % 5 for i in range(n)], 16, 1, 8, dim, dtype, True,
               [((i, i + 1, i + 200), 3) for i in range(0, 200, 2)])
    s.attend()
    s.check(only=set(range(0, n, 31)) | {n - 1})


def test_it_gives_what_the_tree_attention_gives_for_requests_alone():
    """Without groups every row has the pieces that avsg_tree_attention cuts; only the order in which
    up to 40 of them are added differs."""
    s = Shared([300, 31, 1000], [4, 64, 1], 16, 2, 4, 128, BF16, True, [])
    s.attend()
    s.check()
    out, lse = torch.zeros_like(s.out), torch.zeros_like(s.lse)
    s.cache.attend(s.q, s.first, out, 64, s.cache.attention_workspace(4, 64), mask=s.dmask, lse=lse)
    # 39 additions of values of one sign, half a step of fp32 (2^-24) each in either order: the sums are
    # 2 * 39 * 2^-24 apart at most, relatively, and so are their logarithms absolutely; log and the product
    # and sum behind it are off by a step each (2^-23 of at most 8)
    order = 2 * 39 * 2.0**-24
    assert (lse - s.lse).abs().max() <= order + 2 * 3 * 8 * 2.0**-23
    # the outputs' sums too, of terms below 6 in all, divided by the sums; then each is rounded to bf16
    far = (out.float() - s.out.float()).abs()
    assert (far <= 2 * order * 6 + 2 * 2.0**-8 * 1.01 * torch.maximum(out.float().abs(), s.out.float().abs())).all()


def test_offsets_past_32_bits():
    from decode_serving_gb300.paged import PagedCache
    heads, page, dim = 8, 16, 128
    pool = (1 << 32) // (heads * page * dim) + 40      # values of K alone pass 2^32
    s = Shared([100, 90], [4, 2], page, heads, 4, dim, BF16, True, [((0, 1), 5)])
    k, v = (torch.zeros(1, pool, heads, page, dim, dtype=BF16, device="cuda") for _ in "kv")
    small = s.k.shape[1]
    k[:, pool - small:], v[:, pool - small:] = s.k, s.v
    s.cache = PagedCache(k, v, s.cache.tables + (pool - small), s.cache.lens,
                         torch.zeros(pool, dtype=torch.int32, device="cuda"), s.cache.free_count)
    s.k, s.v = k, v
    s.find()
    s.attend()
    s.check()
    # a fork copies rows there, a compaction moves them down
    free = torch.arange(pool, dtype=torch.int32, device="cuda")
    held = torch.unique(s.cache.tables[torch.arange(s.cache.max_pages, device="cuda")[None] <
                                       torch.tensor([[7], [6]], device="cuda")].long())
    used = torch.zeros(pool, dtype=torch.bool, device="cuda")
    used[held] = True
    stack = free[~used]
    free[:len(stack)] = stack
    c = PagedCache(k, v, s.cache.tables, s.cache.lens, free, torch.full_like(s.cache.free_count, len(stack)),
                   shares=torch.zeros(pool, dtype=torch.int32, device="cuda"))
    c.shares[s.cache.tables[0, :5].long()] = 1
    rows = [k[0, int(c.tables[0, 6]), :, :4].clone(), v[0, int(c.tables[0, 0])].clone()]
    c.fork(dev(np.array([0, 0])), c.fork_workspace())
    assert c.error()[0] == 0 and c.tables[0, 6] != c.tables[1, 6] and c.tables[1, 6] == stack[-1]
    assert torch.equal(k[0, int(c.tables[1, 6]), :, :4], rows[0])
    c.compact(torch.zeros_like(free), c.compact_workspace())
    assert c.error()[0] == 0 and int(c.tables[:, :6].max()) < 8
    assert torch.equal(k[0, int(c.tables[1, 6]), :, :4], rows[0]) and torch.equal(v[0, int(c.tables[0, 0])], rows[1])


@pytest.mark.parametrize("what,code", [("page", -4), ("shared", -4), ("ragged", -4), ("first", -4), ("order", -4),
                                       ("token", -4), ("low token", -4), ("request", -4), ("unlisted", -4),
                                       ("length", -4), ("rows", -4), ("most", -2), ("columns", -2)])
def test_bad_inputs_are_latched(what, code):
    s = Shared([100, 90], [4, 2], 16, 2, 4, 64, BF16, True, [((0, 1), 5)])
    work = s.cache.attend_prefixes_workspace(4, 4, s.total)
    work.fill_(255)
    most, kw = None, {}
    if what == "page":
        s.cache.tables[0, 3] = s.k.shape[1]
    elif what == "shared":
        s.x.shared[1] = 96
    elif what == "ragged":
        s.x.shared[0] = 72
    elif what == "first":
        s.x.first[1:] = 7
    elif what == "order":
        s.x.first[0] = -1
    elif what == "token":
        s.x.token[2] = s.total
    elif what == "low token":
        s.x.token[2] = -1
    elif what == "request":
        s.x.request[1] = 2
        kw = dict(window=50)
    elif what == "unlisted":
        s.x.first.zero_()
    elif what == "length":
        s.cache.lens[0] = -1
    elif what == "rows":
        s.first[2] = 7
    elif what == "most":
        most = 3
    elif what == "columns":
        s.cache.lens[1] = 16 * s.cache.tables.shape[1]
    s.attend(work=work, most=most, **kw)
    assert s.cache.error()[0] == code
    s.out.fill_(9.0)
    s.attend()                                          # latched: nothing is written
    assert (s.out == 9.0).all()


@pytest.mark.parametrize("shared", [2 ** 31 - 16, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("dim,new", [(64, 1), (64, 40), (256, 2)])
def test_the_most_tokens_that_an_int_holds_are_no_prefix(shared, dim, new):
    s = Shared([100, 90], [new, new], 16, 2, 4, dim, BF16, False, [((0, 1), 5)])
    s.x.shared[0] = shared
    s.out.fill_(9.0)
    s.attend()
    assert s.cache.error()[0] == -4


def test_refusals():
    from decode_serving_gb300.avsg import AvsgError
    s = Shared([100, 90], [2, 2], 16, 2, 2, 64, BF16, True, [((0, 1), 5)])
    work = s.cache.attend_prefixes_workspace(2, 2, 4)
    call = lambda **kw: s.cache.attend_prefixes(**{**dict(q=s.q, first=s.first, prefixes=s.x, out=s.out, max_new=2,  # noqa: E731
                                                          work=work), **kw})
    other = Shared([100], [2], 16, 2, 2, 64, BF16, True, [])
    for kw in (dict(q=s.q.half()), dict(out=s.out[:1]), dict(first=s.first[:1]), dict(mask=s.dmask.int()),
               dict(lse=s.lse[:, :1].contiguous()), dict(prefixes=other.x), dict(work=work[::2])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(work=work[:-256]), dict(work=work[1:]), dict(layer=1), dict(window=-1), dict(softcap=-1.0),
               dict(max_new=0)):
        with pytest.raises(AvsgError):
            call(**kw)
    with pytest.raises(AvsgError):
        s.cache.attend_prefixes_workspace(2, 2, -1)
    call(q=s.q[:0], out=s.out[:0])                      # no rows: no work
    assert s.cache.error()[0] == 0


def test_two_streams_with_a_workspace_each():
    steps = [Shared([4000, 3900, 17], [5, 8, 1], 16, 2, 4, 128, BF16, True, [((0, 1), 200)], seed=k) for k in (1, 2)]
    alone = []
    for s in steps:
        s.attend()
        alone.append(s.out.clone())
    streams = [torch.cuda.Stream() for _ in steps]
    works = [s.cache.attend_prefixes_workspace(4, 8, s.total) for s in steps]
    for s in steps:
        s.out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, st, w in zip(steps, streams, works):
            s.attend(work=w, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for s, a in zip(steps, alone):
        assert s.cache.error()[0] == 0 and torch.equal(s.out, a)


def test_two_graphs_share_a_workspace_in_turn():
    s = Shared([2000, 1990], [6, 8], 16, 2, 4, 128, F16, True, [((0, 1), 100)])
    few = Shared([900, 901, 902], [1, 1, 1], 16, 2, 4, 128, F16, False, [((0, 1, 2), 50)])
    work = s.cache.attend_prefixes_workspace(4, 8, 14)
    graphs = []
    s.attend(work=work)
    few.attend(work=work, most=8)
    torch.cuda.synchronize()
    want = s.out.clone(), few.out.clone()
    side = torch.cuda.Stream()
    for x in (s, few):
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                x.attend(work=work, most=8)
        graphs.append(g)
    s.out.zero_(), few.out.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out, want[0]) and torch.equal(few.out, want[1])


class Sampler:
    """Steps of a model's attention layers for requests that share pages: fork, plan, groups, rotary
    positions of two axes and attention in two layers, keep; a compaction now and then."""

    def __init__(self, dtype):
        from decode_serving_gb300.paged import PagedCache, rotary_axes, rotary_frequencies
        self.R, self.H, self.G, self.D, self.cap = 6, 2, 4, 64, 240
        self.cache = PagedCache.allocate(self.R, 40, 120, self.H, 8, self.D, layers=2, dtype=dtype, sharing=True)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.new, self.first, self.slots, self.pos = i32(self.R), i32(self.R + 1), i32(self.cap), i32(self.cap)
        self.parent, self.kept, self.map = i32(self.R), i32(self.R), i32(120)
        width = (self.H * self.G + 2 * self.H) * self.D
        self.qkv = torch.zeros(2, self.cap, width, dtype=dtype, device="cuda")
        self.q = torch.zeros(2, self.cap, self.H * self.G, self.D, dtype=dtype, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.freq, self.axes = rotary_frequencies(self.D).cuda(), rotary_axes([20, 12]).cuda()
        c = self.cache
        self.x = c.prefix_arrays(self.cap)
        self.work = [c.fork_workspace(), c.prefix_workspace(), c.attend_prefixes_workspace(self.G, 200, self.cap),
                     c.compact_workspace()]

    def step(self, plain=None):
        c = self.cache
        c.fork(self.parent, self.work[0])
        c.compact(self.map, self.work[3])
        c.plan(self.new, self.first, self.slots, self.pos)
        c.find_prefixes(self.first, self.x, self.work[1], min_tokens=8)
        pos = torch.stack([self.pos, self.pos * 3 + 1])
        for layer in range(2):
            a, b = self.H * self.G * self.D, self.H * self.D
            q, k, v = self.qkv[layer].split((a, b, b), 1)
            c.rotary(q, k, v, pos, self.slots, self.freq, self.q[layer], layer=layer, axes=self.axes)
            c.attend_prefixes(self.q[layer], self.first, self.x, self.out[layer], 200, self.work[2], layer=layer,
                              softcap=20.0)
            if plain is not None:
                c.attend(self.q[layer], self.first, plain[layer], 200, c.attention_workspace(self.G, 200), layer=layer,
                         softcap=20.0)
        c.keep(self.first, None, self.kept)

    def inputs(self, t):
        new, parent = [1] * 6, list(range(6))
        if t == 0:
            new = [100, 0, 50, 0, 0, 0]                    # two prompts
        elif t == 1:
            parent = [0, 0, 2, 2, 0, 2]                    # samples of them
        elif t == 3:
            parent, new = [1, 1, 2, -1, 4, 0], [2, 1, 9, 40, 1, 3]  # beams, an end and a new prompt
        elif t == 4:
            parent = [5, 4, 3, 2, 1, 0]
        for a, b in ((self.new, new), (self.kept, new), (self.parent, parent)):
            a.copy_(dev(np.array(b)))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=torch.Generator("cuda").manual_seed(t),
                                   device="cuda").to(self.qkv.dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_steps_eager_captured_and_on_a_side_stream(dtype):
    """Six steps with forks, ends, a compaction each: eager, replayed from one captured graph and on
    another stream they give the same state and outputs, and what the tree attention gives without groups."""
    runs = []
    for how in ("eager", "graph", "stream"):
        d = Sampler(dtype)
        side = torch.cuda.Stream()
        if how == "graph":
            with torch.cuda.stream(side):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    d.step()
        state = []
        for t in range(6):
            d.inputs(t)
            d.out.zero_()
            torch.cuda.synchronize()
            plain = torch.zeros_like(d.out) if how == "eager" else None
            if how == "graph":
                graph.replay()
            elif how == "stream":
                with torch.cuda.stream(side):
                    d.step()
            else:
                d.step(plain)
            torch.cuda.synchronize()
            assert d.cache.error()[0] == 0
            if plain is not None:
                # either rounds its weights and its result to the type: outputs are means of values within 6
                half = torch.finfo(dtype).eps / 2
                assert (plain.float() - d.out.float()).abs().max() <= 2 * 6 * 2 * half * 1.01
                if t in (1, 2):
                    assert host(d.x.shared).tolist() == [96, 96, 48, 48, 96, 48]
            c = d.cache
            state.append([x.clone() for x in (d.out, c.lens, c.tables, c.free_count, c.free, c.shares, d.slots, d.map)])
        runs.append((d, state))
    for _, state in runs[1:]:
        for a, b in zip(runs[0][1], state):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    c = runs[0][0].cache
    holders = np.zeros(120, np.int64)
    for row, n in zip(host(c.tables), c.lens.tolist()):
        np.add.at(holders, row[:-(-n // 8)], 1)
    assert (host(c.shares) == np.maximum(holders - 1, 0)).all()
    stack = host(c.free)[:int(c.free_count)]
    assert sorted(np.concatenate([stack, np.nonzero(holders)[0]]).tolist()) == list(range(120))


@pytest.mark.parametrize("dim,dtype", [(128, BF16), (64, F16), (256, BF16)])
def test_a_late_maximum_in_either_part(dim, dtype):
    """Scores that grow along the keys of the prefix, and of the requests' own."""
    s = Shared([900, 1240], [40, 3], 16, 1, 6, dim, dtype, True, [((0, 1), 50)])
    first, tables = host(s.first), host(s.cache.tables)
    for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new)):
        q = s.q[first[r], 0].float()
        for p in range(0 if r == 0 else 800, length + n, 3):
            at = (0, int(tables[r, p // 16]), 0, p % 16)
            s.k[at] = (q * (8.0 * p / (length + n)) / q.norm() * dim ** 0.25).to(dtype)
    s.attend(scale=1.0)
    s.check(scale=1.0)


def test_find_and_attention_follow_the_reference_groups():
    s = Shared([300, 31, 305, 0, 299, 64], [3, 1, 4, 2, 1, 9], 8, 2, 3, 128, F16, True, [((0, 2, 4), 37), ((1, 5), 3)],
               least=25)
    want = want_of.find(s.lens, host(s.cache.tables), host(s.first), 8, 25, s.total)
    for g, w in zip((s.x.leader, s.x.shared, s.x.first, s.x.token, s.x.request), want):
        assert (host(g) == w).all()
    assert host(s.x.shared).tolist() == [296, 0, 296, 0, 296, 0]
    s.attend()
    s.check()


@pytest.mark.parametrize("groups", [2, 9])
def test_thousands_of_requests(groups):
    lens = [16 + (i * 37) % 150 for i in range(3000)]
    new = [(i * 5) % 4 for i in range(3000)]
    s = Shared(lens, new, 16, 1, groups, 64, BF16, True, [(tuple(range(k, 3000, 16)), 1) for k in range(8)])
    s.attend()
    s.check(only=set(range(0, 3000, 97)) | {2999})


def test_masks_of_long_requests_are_not_looked_at():
    """A request of more than 64 new tokens is a chain in either part."""
    s = Shared([64, 70, 64], [70, 12, 3], 16, 1, 4, 128, BF16, True, [((0, 1, 2), 4)])
    s.mask[:70] = trees([64], 1).tolist() + [5] * 6
    s.dmask = dev(s.mask, torch.int64)
    s.attend(window=100)
    s.check(window=100)


def test_calls_in_a_row_do_not_reach_into_one_another():
    """Two batches in turn with one workspace and nothing waited for in between: long prefixes beside
    short own keys, and the other way round."""
    a = Shared([6000, 6100, 6050, 40], [1, 1, 1, 1], 16, 2, 4, 128, BF16, False, [((0, 1, 2), 370)], seed=1)
    b = Shared([9000, 300, 290, 700], [16, 3, 8, 1], 16, 2, 4, 128, BF16, True, [((1, 2), 17)], seed=2)
    work = a.cache.attend_prefixes_workspace(4, 16, 28)
    want = []
    for s in (a, b):
        s.attend(work=work, most=16)
        torch.cuda.synchronize()
        s.check()
        want.append((s.out.clone(), s.lse.clone()))
    got = []
    for k in range(40):
        s = (a, b)[k % 2]
        s.out.zero_()
        s.attend(work=work, most=16)
        got.append((s.out.clone(), s.lse.clone()))
    torch.cuda.synchronize()
    for k, g in enumerate(got):
        assert all(torch.equal(x, y) for x, y in zip(g, want[k % 2])), k


def test_groups_that_change_between_replays():
    """One captured attention, with other groups, lengths and first tokens at each replay."""
    cases = [([400, 410, 420, 30], [((0, 1, 2), 25)]), ([400, 410, 420, 410], [((0, 2), 20), ((1, 3), 3)]),
             ([17, 300, 5, 290], [((1, 3), 18)]), ([50, 60, 70, 80], [])]
    base = Shared([420] * 4, [3, 1, 2, 4], 16, 2, 4, 128, F16, True, [], seed=3)
    work, find = base.cache.attend_prefixes_workspace(4, 4, base.total), base.cache.prefix_workspace()

    def step():
        base.cache.find_prefixes(base.first, base.x, find, min_tokens=16)
        base.attend(work=work, most=4)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
    for lens, share in cases:
        s = Shared(lens, [3, 1, 2, 4], 16, 2, 4, 128, F16, True, share, seed=3, least=16)
        base.lens = np.array(lens, np.int32)
        base.cache.lens.copy_(dev(base.lens))
        base.cache.tables.zero_()
        base.cache.tables[:, :s.cache.max_pages].copy_(s.cache.tables)
        base.k[:, :s.k.shape[1]].copy_(s.k)
        base.v[:, :s.v.shape[1]].copy_(s.v)
        base.q.copy_(s.q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(base.x.shared, s.x.shared)
        base.check()


def test_the_binding_s_functions_beside_the_methods():
    from decode_serving_gb300 import avsg
    s = Shared([300, 290, 60], [2, 5, 1], 16, 2, 4, 128, BF16, True, [((0, 1), 16)])
    s.attend()
    torch.cuda.synchronize()
    x = s.cache.prefix_arrays(s.total)
    args = avsg.avsg_prefixes(num_tokens=s.total, d_leader=x.leader.data_ptr(), d_shared=x.shared.data_ptr(),
                              d_first=x.first.data_ptr(), d_token=x.token.data_ptr(), d_request=x.request.data_ptr())
    pages = s.cache._pages
    n = avsg.avsg_prefix_find_workspace(pages)
    work = torch.empty(n, dtype=torch.uint8, device="cuda")
    avsg.avsg_prefix_find(pages, s.first.data_ptr(), 1, args, work.data_ptr(), n)
    n = avsg.avsg_prefix_attention_workspace(pages, 4, 5, s.total)
    work2 = torch.empty(n, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(s.out), torch.zeros_like(s.lse)
    t = avsg.avsg_tree(num_tokens=s.total, q_per_kv=4, max_new=5, layer=0, q_stride=8 * 128, d_q=s.q.data_ptr(),
                       d_first=s.first.data_ptr(), d_mask=s.dmask.data_ptr(), d_out=out.data_ptr(),
                       d_lse=lse.data_ptr(), d_work=work2.data_ptr(), work_bytes=n)
    avsg.avsg_prefix_attention(pages, t, args)
    torch.cuda.synchronize()
    assert s.cache.error()[0] == 0 and torch.equal(out, s.out) and torch.equal(lse, s.lse)
    assert all(torch.equal(a, b) for a, b in zip((x.leader, x.shared, x.first, x.token, x.request),
                                                 (s.x.leader, s.x.shared, s.x.first, s.x.token, s.x.request)))
