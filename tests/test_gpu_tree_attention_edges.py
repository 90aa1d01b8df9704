"""Tree attention where a result may depend on what it must not: values that a row does not see, the
place of a tile's border, words and bits that stand for nothing, the stream of a call."""
import math

import numpy as np
import pytest
import torch

from test_gpu_paged import BF16, F16, dev, host
from test_gpu_tree_attention import Decoder, Step

pytestmark = pytest.mark.gpu

# (groups, dim, page): few rows and pages of fewer than 8 tokens run on mma.sync, the others on tcgen05;
# 12 drafts of 4 heads are one stream's rows, of 16 heads two streams'.
KERNELS = [(1, 64, 16), (4, 64, 4), (4, 256, 4), (4, 64, 16), (16, 64, 16), (4, 128, 16), (16, 128, 16), (4, 256, 16)]


def unseen_places(s, window):
    """(page, row) of keys that no row sees: behind the last token, outside every window."""
    out = []
    for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new)):
        out += [(r, p) for p in range(max(0, length - window + 1))]
        out += [(r, p) for p in range(length + n, -(-(length + n) // s.page) * s.page)]
    return [s.row(r, p) for r, p in out]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_unseen_keys_leave_a_large_cap_alone(groups, dim, page, dtype):
    """A cap of 1e6 changes scores below 50 by less than 2^-24 of themselves, whatever the keys hold
    that a row does not see: no bit of the result may depend on them."""
    window, draft = 50, 2
    s = Step([40, 0, 75], [12, 7, 3], page, 2, groups, dim, dtype, True)
    s.htables = host(s.cache.tables)
    at = unseen_places(s, window)
    a, b = s.row(0, 40 + draft)                        # seen by its branch only
    blind = torch.from_numpy(np.array([not (int(m) >> draft) & 1 or t >= 12 for t, m in enumerate(s.mask)])).cuda()
    results = []
    for value in (0.0, math.inf, -3e4, math.nan):
        for x, y in at + [(a, b)]:
            s.k[0, x, :, y] = 0.0
            s.k[0, x, :, y, 3] = value                 # (its scores: infinities, large ones, NaN)
        s.attend(window=window, softcap=1e6)
        results.append((s.out[blind].clone(), s.lse[blind].clone()))
        if value == 0.0:
            s.check(window=window)                     # the definition without a cap
    assert s.cache.error()[0] == 0
    for out, lse in results[1:]:
        assert torch.equal(out, results[0][0]) and torch.equal(lse, results[0][1])


@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_a_row_is_capped_by_what_it_sees(groups, dim, page):
    """Scores beyond half of the cap, of one row or of all: the same bits whatever the other rows see,
    and for a large cap as near the definition as small scores are."""
    s = Step([200, 9], [12, 5], page, 2, groups, dim, BF16, True)
    s.htables = host(s.cache.tables)
    blind = torch.from_numpy(np.array([not (int(m) >> 2) & 1 or t >= 12 for t, m in enumerate(s.mask)])).cuda()
    for cap in (2.0, 30.0, 1e5):
        results = []
        for value in (0.0, 2.0**50):
            a, b = s.row(0, 202)                       # draft 2, seen by its branch only
            s.k[0, a, :, b] = 0.0
            s.k[0, a, :, b, 3] = value
            s.attend(softcap=cap)
            results.append((s.out[blind].clone(), s.lse[blind].clone()))
            if cap < 1e5 or value == 0.0:
                s.check(cap=cap)
        assert all(torch.equal(x, y) for x, y in zip(*results))
    # a seen score of -cap, which has no weight, leaves the small ones beside it as exact as one of
    # -512 / sqrt(dim) does, whose weight is below 1e-13
    a, b = s.row(0, 30)
    s.q[:, :, 3] = 1.0
    s.k[0, a, :, b] = 0.0
    results = []
    for value in (-512.0, -2.0**50):
        s.k[0, a, :, b, 3] = value
        s.attend(softcap=1e5)
        results.append((s.out.clone(), s.lse.clone()))
        s.check(cap=1e5)
    assert all(torch.equal(x, y) for x, y in zip(*results))


def step_without_streams(d):
    """A step's calls as the README prints them."""
    c = d.cache
    c.plan(d.new, d.first, d.slots, d.pos, mask=d.mask)
    for layer in range(2):
        a, b = d.H * d.G * d.D, d.H * d.D
        q, k, v = d.qkv[layer].split((a, b, b), 1)
        c.rotary(q, k, v, d.pos, d.slots, d.freq, d.q[layer], layer=layer)
        c.attend(d.q[layer], d.first, d.out[layer], 8, d.work, mask=d.mask, layer=layer)
    c.keep(d.first, d.path, d.kept)


@pytest.mark.parametrize("how", ["side stream", "graph"])
def test_calls_without_a_stream_follow_the_current_one(how):
    runs = []
    for where in ("default", how):
        d = Decoder(BF16)
        d.cache.free_count.fill_(40)
        side = torch.cuda.Stream()
        torch.cuda.synchronize()
        if where == "graph":
            d.inputs(0)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                step_without_streams(d)
        for t in range(3):
            if where == "side stream":
                d.inputs(50 + t)
                late = d.qkv.clone()
                d.qkv.zero_()
                torch.cuda.synchronize()
                with torch.cuda.stream(side):
                    torch.cuda._sleep(20_000_000)
                    d.qkv.copy_(late)
                    step_without_streams(d)
                side.synchronize()
            else:
                d.inputs(50 + t)
                g.replay() if where == "graph" else step_without_streams(d)
        assert d.cache.error()[0] == 0
        runs.append([x.clone() for x in (d.out, d.cache.lens, d.cache.tables, d.cache.free_count, d.cache.k)])
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("groups,dim,page", [(1, 64, 4), (4, 128, 16), (2, 256, 16)])
def test_long_requests_are_chains_whatever_their_words_hold(groups, dim, page):
    """More than 64 new tokens: the plan's positions and the attention's are those of a chain."""
    s = Step([10, 33], [70, 9], page, 2, groups, dim, BF16, True)
    s.mask[:70] = 5                                    # (Step made zeros; two bits for every token)
    s.dmask = dev(s.mask, torch.int64)
    s.cache.free_count.fill_(s.count)                  # the same pages again
    s.plan(s.new, s.total, s.mask)
    assert host(s.pos)[:70].tolist() == list(range(10, 80))
    s.attend(window=25)
    s.check(window=25)


@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_bits_past_the_new_tokens_count_for_the_position(groups, dim, page):
    """A mask word's bits past the request's tokens stand for no key, but a position is the number
    of bits: the window lies before that position."""
    s = Step([532, 70, 0], [3, 12, 5], page, 2, groups, dim, BF16, True)
    words = s.mask.view(np.uint64).copy()
    words[:3] |= np.uint64(2**64 - 8)
    words[3:15] |= np.uint64(2**64 - 2**40)
    s.mask = words.view(np.int64)
    s.dmask = dev(s.mask, torch.int64)
    slopes = np.full(2 * groups, 0.02, np.float32)
    for window in (200, 66, 30):
        s.attend(window=window)
        s.check(window=window)
    s.attend(window=200, slopes=dev(slopes, torch.float32))
    s.check(window=200, slopes=slopes)


@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_a_cap_far_below_the_scores(groups, dim, page):
    """Every score is the cap's value or its negative, next to nothing: all visible keys weigh the same."""
    s = Step([300, 40], [12, 5], page, 2, groups, dim, F16, True)
    for cap in (1e-30, 1e-37):
        s.attend(softcap=cap)
        s.check(cap=cap)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("groups,dim,page", KERNELS)
@pytest.mark.parametrize("length", [128, 150, 700, 1500])
def test_values_that_are_not_finite_reach_every_row_that_sees_them(groups, dim, page, dtype, length):
    """One key takes all of the weight, that of the others rounds to 0: wherever a tile's border lies, a
    row that sees an infinity or a NaN of V has a result that is not finite, and no other row has."""
    s = Step([length], [12], page, 1, groups, dim, dtype, True)
    s.htables = host(s.cache.tables)
    q = s.q[:, 0].float()
    s.q[:] = (q.mean(0) + 0.1 * q)[:, None].to(dtype)  # rows that agree on the largest key
    s.k *= 0.1
    a, b = s.row(0, length - 40)
    s.k[0, a, :, b] = (q.mean(0) * 30).to(dtype)
    for place, value in ((5, math.inf), (length - 33, math.nan), (length + 2, -math.inf), (length + 7, math.inf)):
        a, b = s.row(0, place)
        old = s.v[0, a, :, b, 3].clone()
        s.v[0, a, :, b, 3] = value
        s.attend(scale=40.0)
        sees = place < length or torch.from_numpy((s.mask >> (place - length)) & 1).bool().cuda()
        finite = torch.isfinite(s.out.float())
        assert torch.equal(~finite[..., 3], (torch.zeros_like(s.lse) > 1) | (
            sees if place < length else sees[:, None])), f"place {place}"
        assert finite[..., :3].all() and finite[..., 4:].all()
        s.v[0, a, :, b, 3] = old
    s.attend(scale=40.0)
    s.check(scale=40.0)


@pytest.mark.parametrize("groups,most,dim", [(4, 1, 128), (4, 8, 64), (2, 5, 256), (16, 9, 128)])
def test_a_workspace_fits_every_pool(groups, most, dim):
    """Its size depends on the heads and max_new alone: a small pool's serves a large one."""
    from decode_serving_gb300.paged import PagedCache
    caches = [PagedCache.allocate(2, 4, pages, 1, page, dim) for pages, page in ((8, 16), (2048, 16), (64, 4))]
    sizes = [c.attention_workspace(groups, most).numel() for c in caches]
    assert sizes[0] == sizes[1] == sizes[2]
    work = caches[0].attention_workspace(groups, most)
    q = torch.randn(2, groups, dim, device="cuda").to(BF16)
    for c in caches:
        out, first = torch.full_like(q, 3.0), dev(np.array([0, 1, 2]))
        c.plan(dev(np.array([1, 1])), first, dev(np.zeros(2)), dev(np.zeros(2)))
        c.attend(q, first, out, most, work)
        assert c.error()[0] == 0 and (out == 0).all()  # (V is zero)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("groups,dim,page", [k for k in KERNELS if k[1] > 64])
def test_unseen_values_with_wider_heads(groups, dim, page, dtype, cap):
    s = Step([40, 0, 175], [12, 7, 3], page, 2, groups, dim, dtype, True)
    s.mask[12] = 0                                     # request 1 has no context: its first row is empty
    s.mask[15] = -2**63                                # a bit past its new tokens
    s.dmask = dev(s.mask, torch.int64)
    s.htables = host(s.cache.tables)
    at = lambda r, p: (0, s.row(r, p)[0], slice(None), s.row(r, p)[1])  # noqa: E731
    for r, p in ((r, p) for r, (length, n) in enumerate(zip(s.lens.tolist(), s.new))
                 for p in range(length + n, -(-(length + n) // page) * page)):
        s.k[at(r, p)] = s.v[at(r, p)] = math.nan
    s.v[at(0, 42) + (dim - 1,)] = math.inf             # draft 2 of request 0: seen by its branch only
    s.v[at(0, 42) + (63,)] = -math.inf
    s.k[at(0, 43)] = math.nan                          # draft 3
    s.v[at(2, 3)] = math.nan                           # outside the window
    s.k[at(2, 4)] = math.inf
    s.attend(window=150, softcap=cap)
    s.check(window=150, cap=cap)


@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, BF16), (256, F16)])
@pytest.mark.parametrize("kw", [dict(slopes=True), dict(slopes=True, cap=6.0, window=90, scale=0.2),
                                dict(window=33), dict(cap=30.0)])
@pytest.mark.parametrize("tree", [True, False])
def test_two_streams_with_caps_windows_and_slopes(dim, dtype, kw, tree):
    """Units of more than 128 rows (two m-tiles for heads of 256)."""
    heads, groups = 2, 12
    s = Step([0, 500, 66, 129], [12, 19, 40, 1], 16, heads, groups, dim, dtype, tree)
    kw = dict(kw)
    slopes = (2.0 ** (-np.arange(1, heads * groups + 1) / 3.0)).astype(np.float32) if kw.pop("slopes", False) else None
    s.attend(scale=kw.get("scale", 0.0), softcap=kw.get("cap", 0.0), window=kw.get("window", 0),
             slopes=None if slopes is None else dev(slopes, torch.float32))
    s.check(slopes=slopes, **kw)


@pytest.mark.parametrize("dim,dtype,page", [(64, BF16, 16), (128, F16, 1), (256, BF16, 4)])
@pytest.mark.parametrize("kw", [dict(window=70), dict(window=1), dict(slopes=True),
                                dict(slopes=True, cap=5.0, window=100, scale=0.2)])
def test_chains_on_mma_sync_with_windows_and_slopes(dim, dtype, page, kw):
    heads, groups = 2, 3
    new = [1, 5, 9, 2] if page == 16 else [70, 9, 30, 1]
    s = Step([300, 0, 64, 1000], new, page, heads, groups, dim, dtype, False)
    kw = dict(kw)
    slopes = (2.0 ** (-np.arange(1, heads * groups + 1) / 2.0)).astype(np.float32) if kw.pop("slopes", False) else None
    s.attend(scale=kw.get("scale", 0.0), softcap=kw.get("cap", 0.0), window=kw.get("window", 0),
             slopes=None if slopes is None else dev(slopes, torch.float32))
    s.check(slopes=slopes, **kw)


@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_the_same_bits_from_call_to_call(groups, dim, page):
    s = Step([4000, 17, 900], [12, 1, 7], page, 2, groups, dim, BF16, True)
    s.attend(softcap=30.0)
    want = s.out.clone(), s.lse.clone()
    for _ in range(5):
        s.out.zero_(), s.lse.zero_()
        s.attend(softcap=30.0)
        assert torch.equal(s.out, want[0]) and torch.equal(s.lse, want[1])


@pytest.mark.parametrize("groups,dim,page", KERNELS)
def test_max_new_is_a_bound_alone(groups, dim, page):
    """The largest one there is gives what the right one does."""
    s = Step([400, 17, 0], [12, 1, 7], page, 2, groups, dim, BF16, True)
    s.attend(most=2**31 - 1)
    s.check()
