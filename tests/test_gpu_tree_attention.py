"""avsg_tree_attention against its definition in 64 bits, alone and as part of
a step (plan, rotary write, attention, keep), eager and captured."""
import math

import numpy as np
import pytest
import torch

import paged_reference as ref
from test_gpu_paged import BF16, F16, Batch, dev, host, trees

pytestmark = pytest.mark.gpu


def bound(q, k, size, out, scale, cap, slopes, reach, dtype):
    """Allowed |difference| of out and of lse, by counting roundings.

    A score is a sum of D products in fp32 (each addition at most 2^-24 of the
    sum of |q k|), scaled, capped and biased (a step of 2^-23 of its size each;
    the cap's quotient 2^-21); exp2 and the sums of the weights 2^-20 in all.
    A score's error d changes a weight by a factor of exp(+-2d).  The weights
    are rounded to the cache's type (half a step) before the second product,
    the result once more."""
    dim = q.shape[-1]
    terms = scale * np.abs(q).max(0) @ np.abs(k).max(0) if len(k) else 0.0
    score = (dim + 8) * 2.0**-24 * terms + 2.0**-22 * terms + cap * 2.0**-21
    if slopes is not None:
        score += 3 * 2.0**-24 * np.abs(slopes).max() * reach
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).smallest_normal * half
    e = 2 * score + 2.0**-20
    return size * (half + e) * 1.01 + half * np.abs(out) + tiny, score + 2.0**-20


class Step(Batch):
    """A planned step with q for every new token; K and V as the pages hold them."""

    def __init__(self, lens, new, page, heads, groups, dim, dtype, tree, seed=1, layers=1, extra=0):
        total = sum(new)
        super().__init__(lens, page, seed=seed, spare=total // page + len(lens) + 4,
                         room=max(new) // page + 2, layers=layers, heads=heads, dim=dim, dtype=dtype)
        self.new, self.groups, self.total, self.layer = new, groups, total, layers - 1
        self.mask = trees(new, seed) if tree else None
        self.plan(new, total + extra, self.mask)
        gen = torch.Generator("cuda").manual_seed(seed + 9)
        self.q = torch.randn(total + extra, heads * groups, dim, generator=gen, device="cuda").to(dtype)
        self.out = torch.full_like(self.q, 3.0)
        self.lse = torch.full((total + extra, heads * groups), 3.0, device="cuda")
        self.dmask = None if self.mask is None else dev(np.pad(self.mask, (0, extra)), torch.int64)

    def row(self, r, p):
        """(page, row) of token p of request r."""
        return int(self.htables[r, p // self.page]), p % self.page

    def attend(self, work=None, most=None, q=None, **kw):
        most = max(max(self.new), 1) if most is None else most
        work = self.cache.attention_workspace(self.groups, most) if work is None else work
        self.cache.attend(self.q if q is None else q, self.first, self.out, most, work, mask=self.dmask,
                          lse=self.lse, layer=self.layer, **kw)

    def check(self, scale=0.0, cap=0.0, window=0, slopes=None, only=None):
        assert self.cache.error()[0] == 0
        self.htables = host(self.cache.tables)
        as64 = lambda t: t.double().cpu().numpy()  # noqa: E731
        first, heads, groups = host(self.first), self.k.shape[2], self.groups
        out, lse, q = as64(self.out), as64(self.lse), as64(self.q)
        dim = q.shape[-1]
        scale = scale or dim ** -0.5
        for r, (length, n) in enumerate(zip(self.lens.tolist(), self.new)):
            if n == 0 or (only is not None and r not in only):
                continue
            ids = torch.from_numpy(self.htables[r, :-(-(length + n) // self.page)].astype(np.int64)).cuda()
            rows = slice(first[r], first[r] + n)
            mask = None if self.mask is None or n > 64 else self.mask[rows].view(np.uint64)
            for h in range(heads):
                k, v = (as64(x[self.layer, ids, h]).reshape(-1, dim)[:length + n] for x in (self.k, self.v))
                hs = slice(h * groups, (h + 1) * groups)
                sl = None if slopes is None else slopes[hs].astype(np.float64)
                with np.errstate(invalid="ignore"):
                    w_out, w_lse, size = ref.attention(q[rows, hs], k, v, length, mask, scale, cap,
                                                       window, sl)
                fine = np.isfinite(k).all(1)
                b_out, b_lse = bound(q[rows, hs].reshape(-1, dim), k[fine], size, w_out, scale, cap, sl,
                                     length + n, self.q.dtype)
                g_out, g_lse = out[rows, hs], lse[rows, hs]
                nan = np.isnan(w_out)
                assert (np.isnan(g_out) == nan).all(), f"request {r} head {h}: NaN elsewhere"
                inf = np.isinf(w_out)
                assert (g_out[inf] == w_out[inf]).all(), f"request {r} head {h}: infinities"
                ok = ~nan & ~inf
                assert (np.abs(g_out[ok] - w_out[ok]) <= b_out[ok]).all(), f"request {r} head {h}: out"
                none = np.isneginf(w_lse)
                assert (np.isneginf(g_lse) == none).all(), f"request {r} head {h}: empty rows"
                assert (g_out[none] == 0).all()
                ok = ~none & ~np.isnan(w_lse)
                assert (np.abs(g_lse[ok] - w_lse[ok]) <= b_lse + 2.0**-22 * np.abs(w_lse[ok])).all(), \
                    f"request {r} head {h}: lse"


@pytest.mark.parametrize("lens,new,page,heads,groups,dim,dtype,tree", [
    ([0], [1], 16, 1, 1, 128, BF16, False),                       # one token, nothing before it
    ([1], [1], 1, 1, 1, 64, F16, False),
    ([63, 64, 65, 0], [1, 1, 1, 1], 16, 2, 4, 128, BF16, False),   # a tile's border
    ([3000], [1], 16, 1, 8, 128, F16, False),                      # one unit over many CTAs
    ([4095, 5, 0, 700, 64], [3, 1, 4, 0, 2], 8, 2, 4, 128, BF16, False),
    ([200, 31, 1], [64, 17, 1], 16, 2, 4, 128, BF16, True),        # several m-tiles
    ([130, 0, 500], [29, 64, 5], 8, 3, 5, 64, F16, True),
    ([100, 257], [11, 2], 32, 1, 16, 256, BF16, True),
    ([77], [9], 1, 2, 3, 256, F16, True),
    ([10, 0, 333], [300, 129, 1], 64, 1, 2, 128, F16, False),      # prompt chunks
    ([5, 40], [70, 12], 256, 1, 64, 64, BF16, True),               # a chain beside a tree, 64 heads
    ([i * 3 for i in range(150)], [1 + i % 3 for i in range(150)], 16, 1, 2, 64, BF16, False),
])
def test_attention(lens, new, page, heads, groups, dim, dtype, tree):
    s = Step(lens, new, page, heads, groups, dim, dtype, tree, layers=2, extra=2)
    s.attend()
    s.check()
    assert (s.out[s.total:] == 3.0).all() and (s.lse[s.total:] == 3.0).all()


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16)])
@pytest.mark.parametrize("kw", [
    dict(cap=30.0), dict(window=100), dict(slopes=True), dict(window=1), dict(scale=0.3),
    dict(cap=5.0, window=70, slopes=True, scale=0.2),
])
@pytest.mark.parametrize("tree", [True, False])
def test_caps_windows_and_slopes(dim, dtype, kw, tree):
    heads, groups = 2, 4
    s = Step([0, 500, 66, 129], [12, 9, 30, 1], 16, heads, groups, dim, dtype, tree)
    kw = dict(kw)
    slopes = None
    if kw.pop("slopes", False):
        slopes = (2.0 ** (-np.arange(1, heads * groups + 1) / 2.0)).astype(np.float32)
    s.attend(scale=kw.get("scale", 0.0), softcap=kw.get("cap", 0.0), window=kw.get("window", 0),
             slopes=None if slopes is None else dev(slopes, torch.float32))
    s.check(slopes=slopes, **kw)


@pytest.mark.parametrize("dim,page,new", [(64, 4, 12), (128, 16, 12), (256, 4, 12), (256, 16, 12), (128, 16, 2)])
def test_a_cap_far_above_the_scores(dim, page, new):
    """It changes a score s by s (s / cap)^2 / 3: here, below 50, by less than 2^-24 of itself, so the
    result is held to the one without a cap."""
    s = Step([300, 40], [new, new], page, 2, 4, dim, F16, True)
    s.attend(softcap=1e6)
    s.check()
    s.attend(softcap=3.0, slopes=dev(np.full(8, 0.25, np.float32), torch.float32))
    s.check(cap=3.0, slopes=np.full(8, 0.25, np.float32))


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("groups,most", [(1, 8), (4, 8), (8, 16), (16, 16)])
def test_what_a_row_does_not_see_does_not_reach_it(dtype, groups, most, cap):
    """NaN and infinities behind the last token, in drafts of other branches and outside the window;
    rows that see nothing."""
    s = Step([40, 0, 75], [most, 7, 3], 16, 2, groups, 64, dtype, True)
    s.mask[most] = 0                                   # request 1 has no context: its first row is empty
    s.mask[most + 3] = -2**63                       # a bit past its new tokens
    s.dmask = dev(s.mask, torch.int64)
    tables = host(s.cache.tables)
    for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new)):
        for p in range(length + n, -(-(length + n) // 16) * 16):
            for x in (s.k, s.v):
                x[0, int(tables[r, p // 16]), :, p % 16] = math.nan
    page = lambda r, p: (0, int(tables[r, p // 16]), slice(None), p % 16)  # noqa: E731
    s.v[page(0, 42)] = math.inf                        # draft 2 of request 0: seen by its branch only
    s.k[page(0, 43)] = math.nan                        # draft 3
    s.v[page(2, 3)] = math.nan                         # outside the window
    s.k[page(2, 4)] = math.inf
    s.attend(window=50, softcap=cap)
    s.check(window=50, cap=cap)


def test_rows_of_any_stride_and_reused_workspace():
    s = Step([300, 20], [5, 8], 16, 2, 4, 128, BF16, True)
    wide = torch.zeros(s.total, 8 * 128 + 64, dtype=BF16, device="cuda")
    wide[:, 64:] = s.q.reshape(s.total, -1)
    work = s.cache.attention_workspace(4, 8)
    work.fill_(255)                                    # any contents
    s.attend(work=work, q=wide[:, 64:])
    s.check()
    a = s.out.clone()
    s.out.fill_(0)
    s.attend(work=work)
    assert torch.equal(a, s.out)                       # the same bits again


def test_offsets_past_32_bits():
    """Pages whose bytes and values lie past 2^32, at both ends of the pool."""
    from decode_serving_gb300.paged import PagedCache
    heads, page, dim = 8, 16, 128
    pool = (1 << 32) // (heads * page * dim) + 40      # values of K alone pass 2^32
    s = Step([100, 90], [4, 2], page, heads, 4, dim, BF16, True)
    k, v = (torch.empty(1, pool, heads, page, dim, dtype=BF16, device="cuda") for _ in "kv")
    small = s.k.shape[1]
    k[:, pool - small:], v[:, pool - small:] = s.k, s.v
    tables = s.cache.tables + (pool - small)
    free = torch.zeros(pool, dtype=torch.int32, device="cuda")
    s.cache = PagedCache(k, v, tables, s.cache.lens, free, s.cache.free_count)
    s.k, s.v = k, v
    s.attend()
    s.check()
    path = np.array([0, 2, 1, 3, 1, 0], np.int32)
    want = k[0, int(tables[0, 102 // 16]), :, 102 % 16].clone()
    s.cache.keep(s.first, dev(path), dev(np.array([2, 1])))
    assert s.cache.error()[0] == 0
    assert torch.equal(k[0, int(tables[0, 101 // 16]), :, 101 % 16], want)


@pytest.mark.parametrize("what,code", [("page", -4), ("held", -4), ("length", -4), ("rows", -4), ("most", -2),
                                       ("columns", -2)])
def test_bad_inputs_are_latched(what, code):
    s = Step([100, 90], [4, 2], 16, 2, 4, 64, BF16, True)
    most = None
    if what == "page":
        s.cache.tables[0, 3] = s.k.shape[1]
    elif what == "held":
        s.cache.tables[1, 0] = -1
    elif what == "length":
        s.cache.lens[0] = -1
    elif what == "rows":
        s.first[2] = 7
    elif what == "most":
        most = 3
    elif what == "columns":
        s.cache.lens[1] = 16 * s.cache.tables.shape[1]
    s.attend(most=most)
    assert s.cache.error()[0] == code
    s.out.fill_(9.0)
    s.attend()                                          # latched: nothing is written
    assert (s.out == 9.0).all()


def test_refusals():
    from decode_serving_gb300.avsg import AvsgError
    s = Step([10], [2], 16, 2, 2, 64, BF16, True)
    work = s.cache.attention_workspace(2, 2)
    call = lambda **kw: s.cache.attend(**{**dict(q=s.q, first=s.first, out=s.out, max_new=2, work=work), **kw})  # noqa: E731
    for kw in (dict(q=s.q.half()), dict(q=s.q[..., ::2]), dict(out=s.out[:1]), dict(first=s.first[:1]),
               dict(first=s.first.long()), dict(mask=s.dmask.int()), dict(mask=s.dmask[:1]), dict(lse=s.lse[:, :1].contiguous()),
               dict(slopes=torch.zeros(3, device="cuda")), dict(q=s.q[:, :3]), dict(out=s.out.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(work=work[:-256]), dict(work=work[1:]), dict(layer=1), dict(window=-1), dict(softcap=-1.0),
               dict(max_new=0)):
        with pytest.raises(AvsgError):
            call(**kw)
    with pytest.raises(ValueError):
        call(work=work[::2])


class Decoder:
    """A step of a model's attention layers with drafted trees: plan, rotary and attention in
    two layers, keep."""

    def __init__(self, dtype):
        from decode_serving_gb300.paged import PagedCache, rotary_frequencies
        self.R, self.H, self.G, self.D, self.cap = 3, 2, 4, 64, 24
        self.cache = PagedCache.allocate(self.R, 20, 40, self.H, 8, self.D, layers=2, dtype=dtype)
        i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.new, self.first, self.slots, self.pos = i32(self.R), i32(self.R + 1), i32(self.cap), i32(self.cap)
        self.path, self.kept = i32(self.cap), i32(self.R)
        self.mask = torch.zeros(self.cap, dtype=torch.int64, device="cuda")
        width = (self.H * self.G + 2 * self.H) * self.D
        self.qkv = torch.zeros(2, self.cap, width, dtype=dtype, device="cuda")
        self.q = torch.zeros(2, self.cap, self.H * self.G, self.D, dtype=dtype, device="cuda")
        self.out = torch.zeros_like(self.q)
        self.freq = rotary_frequencies(self.D).cuda()
        self.work = self.cache.attention_workspace(self.G, 8)

    def step(self, stream=0):
        c = self.cache
        c.plan(self.new, self.first, self.slots, self.pos, mask=self.mask, stream=stream)
        for layer in range(2):
            a, b = self.H * self.G * self.D, self.H * self.D
            q, k, v = self.qkv[layer].split((a, b, b), 1)
            c.rotary(q, k, v, self.pos, self.slots, self.freq, self.q[layer], layer=layer, stream=stream)
            c.attend(self.q[layer], self.first, self.out[layer], 8, self.work, mask=self.mask, layer=layer,
                     softcap=20.0, stream=stream)
        c.keep(self.first, self.path, self.kept, stream=stream)

    def inputs(self, seed, ends=False):
        r = np.random.default_rng(seed)
        new = r.integers(0, 9, self.R)
        kept = np.array([r.integers(0, n + 1) for n in new])
        if ends:
            kept[1] = -1
        self.new.copy_(dev(new))
        self.kept.copy_(dev(kept))
        path = np.zeros(self.cap, np.int32)
        mask = np.zeros(self.cap, np.int64)
        path[:new.sum()] = np.concatenate([np.pad(np.sort(r.choice(n, max(k, 0), replace=False)), (0, n - max(k, 0)))
                                           for n, k in zip(new, kept)])
        mask[:new.sum()] = trees(new.tolist(), seed)
        self.path.copy_(dev(path))
        self.mask.copy_(dev(mask, torch.int64))
        self.qkv.copy_(torch.randn(self.qkv.shape, generator=torch.Generator("cuda").manual_seed(seed),
                                   device="cuda").to(self.qkv.dtype))


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_steps_eager_captured_and_on_a_side_stream(dtype):
    """Six steps, one request ending on the way: eager, replayed from one captured graph, and on
    another stream give the same state and outputs; the last step's output is the definition's."""
    runs = []
    for how in ("eager", "graph", "stream"):
        d = Decoder(dtype)
        side = torch.cuda.Stream()
        graph = None
        if how == "graph":
            d.inputs(0)
            d.cache.free_count.fill_(40)
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=side):
                    d.step(torch.cuda.current_stream().cuda_stream)
                graph = g
            torch.cuda.synchronize()
        state = []
        for t in range(6):
            d.inputs(100 + t, ends=t == 3)
            d.out.zero_()
            torch.cuda.synchronize()
            if how == "eager":
                d.step()
            elif how == "graph":
                graph.replay()
            else:
                d.step(side.cuda_stream)
            torch.cuda.synchronize()
            assert d.cache.error()[0] == 0
            state.append([x.clone() for x in (d.out, d.cache.lens, d.cache.tables, d.cache.free_count, d.slots)])
        runs.append((d, state))
    for _, state in runs[1:]:
        for a, b in zip(runs[0][1], state):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    # all pages are accounted for, once each
    c = runs[0][0].cache
    held = sum(-(-int(n) // 8) for n in c.lens.tolist())
    assert held + int(c.free_count) == 40
    ids = [int(c.tables[r, x]) for r in range(3) for x in range(-(-int(c.lens[r]) // 8))]
    assert sorted(ids + c.free[:int(c.free_count)].tolist()) == list(range(40))


def test_a_step_gives_the_definition():
    """Plan, rotary write and attention of a step whose context an earlier step kept."""
    d = Decoder(BF16)
    d.inputs(3)
    d.new.copy_(dev(np.array([8, 5, 7])))
    d.mask.copy_(dev(np.pad(trees([8, 5, 7], 3), (0, 4)), torch.int64))
    d.kept.copy_(dev(np.array([3, 5, 0])))
    path = np.zeros(24, np.int32)
    path[0:3], path[8:13] = [0, 4, 7], range(5)
    d.path.copy_(dev(path))
    d.step()
    lens = host(d.cache.lens)
    assert lens.tolist() == [3, 5, 0]
    first_kv = host(d.cache.k.float())
    d.inputs(4)
    d.step()
    first, mask = host(d.first), host(d.mask).view(np.uint64)
    tables = host(d.cache.tables)
    as64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    # the pages before the keep moved rows: the kept context, then this step's rotated rows
    pos = host(d.pos)
    inv = 10000.0 ** (-np.arange(32) * 2.0 / 64)
    turns = pos[:, None] * inv / (2 * np.pi)
    for layer in range(2):
        q, k, v = as64(d.qkv[layer]).reshape(24, -1, 64)[:, :8], as64(d.qkv[layer]).reshape(24, -1, 64)[:, 8:10], \
            as64(d.qkv[layer]).reshape(24, -1, 64)[:, 10:]
        rounded = lambda x: torch.from_numpy(x).to(BF16).double().numpy()  # noqa: E731
        q, k = (rounded(ref.rotate(x, turns, 64, 0, False, 1.0)) for x in (q, k))
        for r in range(3):
            length, rows = int(lens[r]), slice(first[r], first[r + 1])
            if first[r] == first[r + 1]:
                continue
            for h in range(2):
                at = [(int(tables[r, p // 8]), p % 8) for p in range(length)]
                old_k = np.array([first_kv[layer, a, h, b] for a, b in at]).reshape(-1, 64)
                old_v = np.array([as64(d.cache.v[layer, a, h, b]) for a, b in at]).reshape(-1, 64)
                hs = slice(h * 4, h * 4 + 4)
                want, _, size = ref.attention(q[rows, hs], np.concatenate([old_k, k[rows, h]]),
                                              np.concatenate([old_v, v[rows, h]]), length, mask[rows], cap=20.0)
                # a rotated value may round to the neighbouring bf16 value: a step of 2^-8 relative in
                # single places of q and k, scores (below 20 in size) off by at most 2^-7 of their terms
                got = as64(d.out[layer])[rows, hs]
                all_k = np.concatenate([old_k, k[rows, h]])
                terms = 64 ** -0.5 * np.abs(q[rows, hs].reshape(-1, 64)).max(0) @ np.abs(all_k).max(0)
                assert (np.abs(got - want) <= size * (2 * 2.0**-7 * terms + 2.0**-8) + 2.0**-8 * np.abs(want)).all()


@pytest.mark.parametrize("spare", [0, 2000])
@pytest.mark.parametrize("lens,new,groups,dim,dtype", [
    ([0, 1, 127, 128, 129, 700], [1, 1, 1, 1, 1, 1], 4, 128, BF16),
    ([513, 0, 64], [2, 3, 1], 5, 64, F16),
    ([300, 31, 64, 1], [4, 8, 5, 1], 4, 128, F16),
    ([0, 63, 64, 65, 1500], [1, 2, 3, 1, 2], 3, 256, BF16),
    ([700, 0, 129], [8, 5, 1], 4, 256, F16),
])
def test_few_rows_with_a_small_and_a_large_pool(lens, new, groups, dim, dtype, spare):
    """Up to 32 rows per kv-head run on either kernel, by the pool's tokens per request."""
    s = Step(lens, new, 16, 2, groups, dim, dtype, False)
    if spare:
        from decode_serving_gb300.paged import PagedCache
        pool = s.k.shape[1] + spare * len(lens)
        k, v = (torch.zeros(1, pool, *s.k.shape[2:], dtype=dtype, device="cuda") for _ in "kv")
        k[:, :s.k.shape[1]], v[:, :s.k.shape[1]] = s.k, s.v
        s.cache = PagedCache(k, v, s.cache.tables, s.cache.lens,
                             torch.zeros(pool, dtype=torch.int32, device="cuda"), s.cache.free_count)
        s.k, s.v = k, v
    s.attend()
    s.check()


@pytest.mark.parametrize("groups,dim", [(2, 64), (6, 128), (3, 256)])
def test_rows_aligned_to_four_bytes_only(groups, dim):
    """q rows whose start and stride are even counts of values, and no more."""
    s = Step([70, 3], [4, 5], 8, 2, groups, dim, F16, True)
    width = 2 * groups * dim
    wide = torch.zeros(s.total, width + 6, dtype=F16, device="cuda")
    wide[:, 2:2 + width] = s.q.reshape(s.total, -1)
    s.attend(q=wide[:, 2:2 + width])
    s.check()


@pytest.mark.parametrize("groups", [2, 9])
def test_thousands_of_requests(groups):
    lens = [(i * 37) % 150 for i in range(3000)]
    s = Step(lens, [(i * 5) % 4 for i in range(3000)], 16, 1, groups, 64, BF16, True)
    s.attend()
    s.check(only=set(range(0, 3000, 97)) | {2999})


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, BF16)])
@pytest.mark.parametrize("most", [9, 150])
def test_many_short_units(dim, dtype, most):
    """Several units in a CTA's share, of one tile and of a few (of 40 rows and more: on tcgen05)."""
    lens = [(i * 37) % 200 for i in range(600 if most < 64 else 60)]
    s = Step(lens, [5 + i % 5 if most < 64 else most - i for i in range(len(lens))], 16, 1, 8, dim, dtype,
             most < 64)
    s.attend()
    s.check(only=set(range(0, len(lens), 31)) | {len(lens) - 1})


def test_two_streams_with_a_workspace_each():
    """Two caches' attention at the same time gives what each gives alone."""
    steps = [Step([4000, 17], [5, 8], 16, 2, 4, 128, BF16, True, seed=k) for k in (1, 2)]
    alone = []
    for s in steps:
        s.attend()
        alone.append(s.out.clone())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    works = [s.cache.attention_workspace(4, 8) for s in steps]
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
    s = Step([2000, 40], [6, 8], 16, 2, 4, 128, F16, True)
    few = Step([900], [1], 16, 2, 4, 128, F16, False)
    work = s.cache.attention_workspace(4, 8)
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
                x.attend(work=work, most=8, stream=torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    s.out.zero_(), few.out.zero_()
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert torch.equal(s.out, want[0]) and torch.equal(few.out, want[1])


@pytest.mark.parametrize("dim,dtype,window", [(128, BF16, 0), (64, F16, 0), (128, F16, 300),
                                              (256, BF16, 0), (256, F16, 300)])
def test_a_late_maximum(dim, dtype, window):
    """Scores that grow along the keys, so that the output is scaled again and again; and keys of
    large scores at the very end and the very beginning."""
    s = Step([900, 640], [40, 3], 16, 1, 6, dim, dtype, True)
    first, tables = host(s.first), host(s.cache.tables)
    for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new)):
        q = s.q[first[r], 0].float()
        for p in range(0, length + n, 3):
            at = (0, int(tables[r, p // 16]), 0, p % 16)
            s.k[at] = (q * (8.0 * p / (length + n)) / q.norm() * dim ** 0.25).to(dtype)
    s.attend(window=window, scale=1.0)
    s.check(window=window, scale=1.0)
