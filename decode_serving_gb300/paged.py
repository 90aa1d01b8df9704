"""A paged device cache for decoding with drafted tokens: marshalling around
avsg_page_plan, avsg_rotary_write, avsg_tree_attention and avsg_tree_keep, and
for requests that share pages avsg_page_fork, avsg_page_compact,
avsg_prefix_find and avsg_prefix_attention (include/avsg.h has the layouts and
the rules).

All tensors are the caller's, contiguous and on one CUDA device; shapes, types
and devices are checked here (``ValueError``), the rest by the library
(``AvsgError``).  Nothing synchronises except ``error``, ``clear_error`` and the making of a cache.
"""
from __future__ import annotations

import ctypes
import struct

import numpy as np
import torch

from . import avsg as C

_TYPES = {torch.bfloat16: C.AVSG_BF16, torch.float16: C.AVSG_F16}
# The argument structures as bytes: a third of the time that filling them field by field takes.
_ROTARY = struct.Struct("8i3qfi7P")
_TREE = struct.Struct("5i2fiq7PN")
_PREFIXES = struct.Struct("2i5P")
assert _PREFIXES.size == ctypes.sizeof(C.avsg_prefixes)
assert _ROTARY.size == ctypes.sizeof(C.avsg_rotary) and _TREE.size == ctypes.sizeof(C.avsg_tree)


def rotary_frequencies(rot_dim, base=10000.0, factor=1.0, low_turns=1.0, high_turns=32.0,
                       original=0) -> torch.Tensor:
    """The frequency table of ``PagedCache.rotary`` (a host tensor: 64-bit words as int64)."""
    t = C.avsg_rotary_frequencies(rot_dim, base, factor, low_turns, high_turns, original)
    return torch.from_numpy(t[:int(rot_dim) // 2].view(np.int64))


def rotary_axes(sections, dealt=False) -> torch.Tensor:
    """The ``axes`` of ``PagedCache.rotary`` (a host tensor, int32): sections[a] pairs of a head
    turn by axis a, one section after the other or, ``dealt``, a pair of each axis in turn as
    long as it has some left."""
    sections = [int(n) for n in sections]
    if not sections or min(sections) < 0:
        raise ValueError("sections: the number of pairs of each axis is wanted")
    out = [a for a, n in enumerate(sections) for _ in range(n)]
    if dealt:
        out = [a for i in range(max(sections)) for a, n in enumerate(sections) if i < n]
    return torch.tensor(out, dtype=torch.int32)


_P, _I32, _SIZE = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
_calls = {}


def _library():
    """The entry points by address and packed arguments (the binding's own take the structures)."""
    if not _calls:
        lib = C.load_library()
        for name, args in (("avsg_page_plan", [_P, _P, _P, _I32, _I32] + [_P] * 5), ("avsg_rotary_write", [_P] * 3),
                           ("avsg_tree_attention", [_P] * 3), ("avsg_tree_keep", [_P, _P, _P, _I32] + [_P] * 4),
                           ("avsg_rotary_write_axes", [_P, _P, _I32, _P, _P]),
                           ("avsg_page_fork", [_P] * 4 + [_SIZE, _P]),
                           ("avsg_tree_keep_shared", [_P] * 4 + [_I32] + [_P] * 4),
                           ("avsg_page_compact", [_P] * 7 + [_SIZE, _P]),
                           ("avsg_prefix_find", [_P, _P, _I32, _P, _P, _SIZE, _P]),
                           ("avsg_prefix_attention", [_P] * 4)):
            _calls[name] = ctypes.CFUNCTYPE(ctypes.c_int, *args)((name, lib))
    return _calls


def _int32(x):
    """x, if an int32 holds it (struct.error: it does not)."""
    return struct.unpack("i", struct.pack("i", x))[0]


class Prefixes:
    """Groups of requests with a common prefix, as ``PagedCache.find_prefixes`` writes them: leader
    and shared [requests], first [requests + 1], token and request [tokens], int32 (avsg_prefixes)."""

    def __init__(self, leader, shared, first, token, request):
        n, tokens = leader.numel(), token.numel()
        for name, t, count in (("leader", leader, n), ("shared", shared, n), ("first", first, n + 1),
                               ("token", token, tokens), ("request", request, tokens)):
            if t.dtype is not torch.int32 or t.device != leader.device or t.numel() != count or \
                    not t.is_contiguous():
                raise ValueError(f"{name}: a contiguous torch.int32 tensor of {count} values on "
                                 f"{leader.device} is wanted, not {t.dtype} {list(t.shape)} on {t.device}")
        self.leader, self.shared, self.first, self.token, self.request = leader, shared, first, token, request
        self.requests, self._index = n, leader.get_device()
        self._args = _PREFIXES.pack(tokens, 0, leader.data_ptr(), shared.data_ptr(), first.data_ptr(),
                                    token.data_ptr(), request.data_ptr())


class PagedCache:
    """Pages, block tables, lengths and free pages of a batch of requests.

    k, v [layers][num_pages][kv_heads][page_tokens][head_dim] bf16 or fp16;
    tables [requests][max_pages], lens [requests], free [num_pages] and
    free_count [1] int32; shares [num_pages] int32, or None where no page is
    shared: how many requests hold a page beyond the first (``fork``).  New tokens are ragged rows: request r owns rows
    first[r] .. first[r + 1] of every per-token tensor.

    Calls are enqueued on torch's current stream, so that they follow the
    tensors' own work and are captured with it; ``stream`` names another one by
    its handle (0: the default stream).
    """

    def __init__(self, k, v, tables, lens, free, free_count, shares=None):
        if k.dim() != 5 or v.shape != k.shape or k.dtype not in _TYPES or v.dtype != k.dtype:
            raise ValueError("k and v: [layers][num_pages][kv_heads][page_tokens][head_dim], "
                             "both bfloat16 or both float16")
        if k.device.type != "cuda":
            raise ValueError("the cache lives on a CUDA device")
        layers, pages, heads, page, dim = k.shape
        if lens.dim() != 1:
            raise ValueError("lens: [requests] is wanted")
        self.device, self.dtype, self._index = k.device, k.dtype, k.get_device()
        self.requests, self.kv_heads, self.head_dim = len(lens), heads, dim
        self.k, self.v, self.tables, self.lens = k, v, tables, lens
        self.free, self.free_count = free, free_count
        self._check("k", k, k.dtype, k.numel())
        self._check("v", v, k.dtype, k.numel())
        if tables.dim() != 2 or tables.shape[0] != len(lens):
            raise ValueError("tables: [requests][max_pages] is wanted")
        self._check("tables", tables, torch.int32, tables.numel())
        self._check("lens", lens, torch.int32, len(lens))
        self._check("free", free, torch.int32, pages)
        self._check("free_count", free_count, torch.int32, 1)
        self.shares, self.pages, self.max_pages = shares, pages, tables.shape[1]
        if shares is not None:
            self._check("shares", shares, torch.int32, pages)
        self._error = torch.zeros(4, dtype=torch.int32, device=k.device)
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(k.device).synchronize()  # (any stream may read it from here on)
        self._pages = C.avsg_pages(len(lens), layers, pages, heads, page, dim, tables.shape[1],
                                   _TYPES[k.dtype], k.data_ptr(), v.data_ptr(), tables.data_ptr(),
                                   lens.data_ptr(), free.data_ptr(), free_count.data_ptr(),
                                   self._error.data_ptr())
        self._at = ctypes.addressof(self._pages)
        calls = _library()
        self._plan, self._rotary = calls["avsg_page_plan"], calls["avsg_rotary_write"]
        self._attend, self._keep = calls["avsg_tree_attention"], calls["avsg_tree_keep"]
        self._calls = calls

    @classmethod
    def allocate(cls, requests, max_pages, num_pages, kv_heads, page_tokens, head_dim, layers=1,
                 dtype=torch.bfloat16, device="cuda", sharing=False) -> "PagedCache":
        """An empty cache: no tokens, every page free (taken from 0 upward); with ``sharing`` its
        requests can share pages."""
        shape = (layers, num_pages, kv_heads, page_tokens, head_dim)
        ints = dict(dtype=torch.int32, device=device)
        return cls(torch.zeros(shape, dtype=dtype, device=device),
                   torch.zeros(shape, dtype=dtype, device=device),
                   torch.zeros(requests, max_pages, **ints), torch.zeros(requests, **ints),
                   torch.arange(num_pages - 1, -1, -1, **ints), torch.full((1,), num_pages, **ints),
                   torch.zeros(num_pages, **ints) if sharing else None)

    def _check(self, name, t, dtype, count):
        """t: contiguous, of this type and this many values, on the cache's device."""
        if t.dtype is not dtype or t.get_device() != self._index or t.numel() != count or \
                not t.is_contiguous():
            raise ValueError(f"{name}: a contiguous {dtype} tensor of {count} values on {self.device} "
                             f"is wanted, not {t.dtype} {list(t.shape)} on {t.device}")

    def _rows(self, name, t, width):
        """Token rows of `width` consecutive values, any stride between tokens; the stride."""
        if t.dtype is not self.dtype or t.get_device() != self._index:
            raise ValueError(f"{name}: {self.dtype} rows on {self.device} are wanted, not {t.dtype} "
                             f"on {t.device}")
        shape, stride = t.shape, t.stride()
        if len(shape) == 2:
            ok = shape[1] == width and (stride[1] == 1 or width == 1)
        else:
            ok = len(shape) == 3 and shape[1] * shape[2] == width and stride[2] == 1 and (
                shape[1] == 1 or stride[1] == shape[2])
        if not ok:
            raise ValueError(f"{name}: rows of {width} consecutive values are wanted, not "
                             f"{list(shape)} with strides {list(stride)}")
        return stride[0] if shape[0] > 1 else width

    def _stream(self, stream):
        """The handle to launch on (the raw form of torch.cuda.current_stream, without its object)."""
        return (torch._C._cuda_getCurrentRawStream(self._index) if stream is None else stream) or None

    def _heads(self, t):
        """Heads of a row tensor [T][heads * head_dim] or [T][heads][head_dim]."""
        if not 2 <= t.dim() <= 3:
            raise ValueError(f"q: [tokens][heads * head_dim] or [tokens][heads][head_dim] is wanted, not "
                             f"{list(t.shape)}")
        return t.shape[1] if t.dim() == 3 else t.shape[1] // self.head_dim

    def plan(self, new, first, slots, positions, mask=None, free_count_out=None, stream=None):
        """Tables, slots and positions of the step's new tokens.  new [requests],
        first [requests + 1], slots and positions [capacity] int32; mask
        [tokens] int64 words of ancestor bits; free_count_out defaults to the
        cache's own count."""
        r, capacity = self.requests, slots.numel()
        out = self.free_count if free_count_out is None else free_count_out
        self._check("new", new, torch.int32, r)
        self._check("first", first, torch.int32, r + 1)
        self._check("slots", slots, torch.int32, capacity)
        self._check("positions", positions, torch.int32, capacity)
        self._check("free_count_out", out, torch.int32, 1)
        masks = 0
        if mask is not None:
            masks = mask.numel()
            self._check("mask", mask, torch.int64, masks)
        rc = self._plan(self._at, new.data_ptr(), None if mask is None else mask.data_ptr(), masks, capacity,
                        first.data_ptr(), slots.data_ptr(), positions.data_ptr(), out.data_ptr(),
                        self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_page_plan")

    def rotary(self, q, k, v, positions, slots, freq, q_out, layer=0, rot_offset=0,
               interleaved=False, magnitude=1.0, tokens_per_request=1, stream=None, axes=None):
        """Rotates q into q_out and k into the pages, stores v beside it.

        q [T][q_heads * head_dim] (or [T][q_heads][head_dim]), k and v like it
        with kv_heads, any stride between tokens; slots [T] or None (slot t for
        token t); freq from ``rotary_frequencies``, on the device; q_out
        contiguous, the cache's type or float32.  axes [pairs] int32
        (``rotary_axes``, on the device): positions are [axes][T], and a pair
        turns by the position on its axis."""
        heads, tokens, dim = self._heads(q), q.shape[0], self.head_dim
        kv = self.kv_heads * dim
        qs, ks, vs = self._rows("q", q, heads * dim), self._rows("k", k, kv), self._rows("v", v, kv)
        if k.shape[0] != tokens or v.shape[0] != tokens:
            raise ValueError("q, k and v have one row per token")
        f32 = q_out.dtype is torch.float32
        pairs = freq.numel()
        self._check("q_out", q_out, torch.float32 if f32 else self.dtype, tokens * heads * dim)
        if axes is None:
            self._check("positions", positions, torch.int32, tokens)
        else:
            if positions.dim() != 2 or positions.shape[0] < 1:
                raise ValueError("positions: [axes][tokens] is wanted")
            self._check("positions", positions, torch.int32, positions.shape[0] * tokens)
            self._check("axes", axes, torch.int32, pairs)
        self._check("freq", freq, torch.int64, pairs)
        if slots is not None:
            self._check("slots", slots, torch.int32, tokens)
        try:
            args = _ROTARY.pack(
                tokens, heads, 2 * pairs, rot_offset, interleaved, f32, tokens_per_request, layer, qs, ks, vs,
                magnitude, 0, q.data_ptr(), k.data_ptr(), v.data_ptr(), freq.data_ptr(), positions.data_ptr(),
                0 if slots is None else slots.data_ptr(), q_out.data_ptr())
        except struct.error as e:                      # a number that its field does not hold
            raise ValueError(str(e)) from None
        if axes is None:
            rc = self._rotary(self._at, args, self._stream(stream))
        else:
            rc = self._calls["avsg_rotary_write_axes"](self._at, args, positions.shape[0], axes.data_ptr(),
                                                       self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_rotary_write")

    def attention_workspace(self, q_per_kv, max_new) -> torch.Tensor:
        """Scratch of ``attend``; calls that may overlap need one each."""
        n = C.avsg_tree_attention_workspace(self._pages, q_per_kv, max_new)
        return torch.empty(n, dtype=torch.uint8, device=self.device)

    def attend(self, q, first, out, max_new, work, mask=None, lse=None, layer=0, scale=0.0,
               softcap=0.0, window=0, slopes=None, stream=None):
        """Attention of the step's new tokens over their requests' pages.

        q [T][q_heads][head_dim] (any stride between tokens), out like it and
        contiguous, lse [T][q_heads] float32 or None; first from ``plan``;
        max_new bounds every request's new tokens; mask [tokens] int64 words
        (None: chains); slopes [q_heads] float32 or None."""
        args = self._tree(q, first, out, max_new, work, mask, lse, layer, scale, softcap, window, slopes)
        rc = self._attend(self._at, args, self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_tree_attention")

    def _tree(self, q, first, out, max_new, work, mask, lse, layer, scale, softcap, window, slopes):
        """The packed arguments of an attention."""
        heads, tokens, dim = self._heads(q), q.shape[0], self.head_dim
        stride = self._rows("q", q, heads * dim)
        if heads % self.kv_heads:
            raise ValueError("q: a multiple of the cache's heads is wanted")
        self._check("out", out, self.dtype, tokens * heads * dim)
        self._check("first", first, torch.int32, self.requests + 1)
        size = work.numel()
        self._check("work", work, torch.uint8, size)
        if mask is not None:
            if mask.numel() < tokens:
                raise ValueError("mask: a word per row of q is wanted")
            self._check("mask", mask, torch.int64, mask.numel())
        if lse is not None:
            self._check("lse", lse, torch.float32, tokens * heads)
        if slopes is not None:
            self._check("slopes", slopes, torch.float32, heads)
        try:
            return _TREE.pack(
                tokens, heads // self.kv_heads, max_new, layer, window, scale, softcap, 0, stride, q.data_ptr(),
                first.data_ptr(), 0 if mask is None else mask.data_ptr(), 0 if slopes is None else slopes.data_ptr(),
                out.data_ptr(), 0 if lse is None else lse.data_ptr(), work.data_ptr(), size)
        except struct.error as e:                      # a number that its field does not hold
            raise ValueError(str(e)) from None

    def keep(self, first, path, keep, lens_out=None, free_count_out=None, stream=None):
        """Keeps the accepted drafts of every layer and frees the pages past the
        new lengths.  keep [requests] int32: kept tokens, or -1: the request
        ends (one that holds shared pages ends by ``fork``); path [tokens]
        int32 or None: the first keep[r] ones."""
        r = self.requests
        lens = self.lens if lens_out is None else lens_out
        count = self.free_count if free_count_out is None else free_count_out
        self._check("first", first, torch.int32, r + 1)
        self._check("keep", keep, torch.int32, r)
        self._check("lens_out", lens, torch.int32, r)
        self._check("free_count_out", count, torch.int32, 1)
        paths = 0
        if path is not None:
            paths = path.numel()
            self._check("path", path, torch.int32, paths)
        args = (first.data_ptr(), None if path is None else path.data_ptr(), paths, keep.data_ptr(),
                lens.data_ptr(), count.data_ptr(), self._stream(stream))
        if self.shares is None:
            rc = self._keep(self._at, *args)
        else:
            rc = self._calls["avsg_tree_keep_shared"](self._at, self.shares.data_ptr(), *args)
        if rc:
            raise C.AvsgError(rc, "avsg_tree_keep")

    def _workspace(self, size):
        return torch.empty(size, dtype=torch.uint8, device=self.device)

    def fork_workspace(self) -> torch.Tensor:
        """Scratch of ``fork``; calls that may overlap need one each."""
        return self._workspace(C.avsg_page_fork_workspace(self._pages))

    def fork(self, parent, work, stream=None):
        """Request r goes on as what request parent[r] was: itself, a copy of
        another that shares its full pages, or (-1) nothing.  parent
        [requests] int32.  Tables, lengths, shares and free pages change in
        place; between steps, when every token is committed."""
        if self.shares is None:
            raise ValueError("the cache has no shares: its requests cannot share pages")
        self._check("parent", parent, torch.int32, self.requests)
        size = work.numel()
        self._check("work", work, torch.uint8, size)
        rc = self._calls["avsg_page_fork"](self._at, parent.data_ptr(), self.shares.data_ptr(), work.data_ptr(),
                                           size, self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_page_fork")

    def compact_workspace(self) -> torch.Tensor:
        """Scratch of ``compact``; calls that may overlap need one each."""
        return self._workspace(C.avsg_page_compact_workspace(self._pages))

    def compact(self, page_map, work, tables_out=None, free_out=None, shares_out=None, stream=None):
        """Moves the pages in use to the front of the pool, whole and in all
        layers.  page_map [num_pages] int32 receives each page's new id, -1
        for a free one; tables, free pages and shares change in place unless
        others are given for them.  Between steps, when every token is
        committed: pages of planned tokens move too, but neither their table
        entries nor the step's slots follow."""
        tables = self.tables if tables_out is None else tables_out
        free = self.free if free_out is None else free_out
        shares = self.shares if shares_out is None else shares_out
        self._check("page_map", page_map, torch.int32, self.pages)
        self._check("tables_out", tables, torch.int32, self.requests * self.max_pages)
        self._check("free_out", free, torch.int32, self.pages)
        old, new = None, None
        if self.shares is not None:
            self._check("shares_out", shares, torch.int32, self.pages)
            old, new = self.shares.data_ptr(), shares.data_ptr()
        elif shares is not None:
            raise ValueError("shares_out: the cache has no shares")
        size = work.numel()
        self._check("work", work, torch.uint8, size)
        rc = self._calls["avsg_page_compact"](self._at, old, new, tables.data_ptr(), free.data_ptr(),
                                              page_map.data_ptr(), work.data_ptr(), size, self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_page_compact")

    def prefix_arrays(self, tokens) -> Prefixes:
        """Arrays for the groups of steps of up to so many new tokens (no groups yet)."""
        ints = dict(dtype=torch.int32, device=self.device)
        return Prefixes(torch.arange(self.requests, **ints), torch.zeros(self.requests, **ints),
                        torch.zeros(self.requests + 1, **ints), torch.full((tokens,), -1, **ints),
                        torch.full((tokens,), -1, **ints))

    def prefix_workspace(self) -> torch.Tensor:
        """Scratch of ``find_prefixes``; calls that may overlap need one each."""
        return self._workspace(C.avsg_prefix_find_workspace(self._pages))

    def _prefixes(self, prefixes):
        if prefixes.requests != self.requests or prefixes._index != self._index:
            raise ValueError(f"prefixes: arrays of {self.requests} requests on {self.device} are wanted")
        return prefixes._args

    def find_prefixes(self, first, prefixes, work, min_tokens=1024, stream=None):
        """Finds the groups of requests with new tokens whose tables begin
        with the same pages, at least min_tokens of committed tokens, and
        lists each group's new tokens; once per step, after ``plan``.  first
        from ``plan``.

        Below some length a prefix is read faster by every request for
        itself (8 kv-heads of 4, heads of 128, one new token, groups against
        requests alone: 64 requests behind 512 tokens 42 and 41 us, behind
        1024 40 and 56; 16 groups of 4 behind 1024 56 and 59; 32 pairs behind
        1024 71 and 60, behind 2048 85 and 97; 4 groups of 16 with trees of
        16 behind 2048 102 and 107)."""
        self._check("first", first, torch.int32, self.requests + 1)
        size = work.numel()
        self._check("work", work, torch.uint8, size)
        try:
            least = _int32(min_tokens)
        except struct.error as e:
            raise ValueError(str(e)) from None
        rc = self._calls["avsg_prefix_find"](self._at, first.data_ptr(), least, self._prefixes(prefixes),
                                             work.data_ptr(), size, self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_prefix_find")

    def attend_prefixes_workspace(self, q_per_kv, max_new, tokens) -> torch.Tensor:
        """Scratch of ``attend_prefixes`` for up to so many rows of q; calls that may overlap need one each."""
        return self._workspace(C.avsg_prefix_attention_workspace(self._pages, q_per_kv, max_new, tokens))

    def attend_prefixes(self, q, first, prefixes, out, max_new, work, mask=None, lse=None, layer=0, scale=0.0,
                        softcap=0.0, window=0, slopes=None, stream=None):
        """``attend`` with every group's prefix read and multiplied once for
        all of its members; prefixes from ``find_prefixes``, for the same
        tables, lengths and first.  A step without groups is 8 to 28 us faster
        by ``attend`` (64 requests: 42 and 32 us at 100 tokens, 206 and 178 at
        4000, 335 and 327 at 8000)."""
        args = self._tree(q, first, out, max_new, work, mask, lse, layer, scale, softcap, window, slopes)
        rc = self._calls["avsg_prefix_attention"](self._at, args, self._prefixes(prefixes), self._stream(stream))
        if rc:
            raise C.AvsgError(rc, "avsg_prefix_attention")

    def error(self):
        """(code, request, position) of the first latched device error, code 0
        for none; waits for the device (all of its streams)."""
        torch.cuda.synchronize(self.device)
        return tuple(self._error.tolist()[:3])

    def clear_error(self):
        """Waits for the device and drops a latched error."""
        torch.cuda.synchronize(self.device)
        self._error.zero_()
        torch.cuda.synchronize(self.device)
