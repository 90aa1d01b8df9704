"""The paged-cache entry points reject bad arguments on the host, before any
CUDA call, and the rotary frequency table is what its definition says."""
import ctypes
import math
import subprocess
import os
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT


def pages(**kw):
    """A well-formed avsg_pages whose pointers are host memory (never read)."""
    from decode_serving_gb300 import avsg
    buf = np.zeros(64, np.int64)
    at = (buf.ctypes.data + 63) // 64 * 64
    f = dict(num_requests=2, num_layers=2, num_pages=8, num_kv_heads=2, page_tokens=16, head_dim=64,
             max_pages=4, dtype=0, d_k=at, d_v=at, d_tables=at, d_len=at, d_free=at,
             d_free_count=at, d_error=at)
    f.update(kw)
    p = avsg.avsg_pages(**f)
    p.keep = buf
    return p, at


BAD_PAGES = [
    (dict(num_requests=0), -1), (dict(num_layers=0), -1), (dict(num_pages=0), -1),
    (dict(num_kv_heads=0), -1), (dict(page_tokens=0), -1), (dict(head_dim=0), -1),
    (dict(head_dim=12), -1), (dict(max_pages=0), -1), (dict(dtype=2), -1), (dict(d_k=None), -1),
    (dict(d_v=None), -1), (dict(d_tables=None), -1), (dict(d_len=None), -1), (dict(d_free=None), -1),
    (dict(d_free_count=None), -1), (dict(d_error=None), -1), (dict(d_k=8), -1),
    (dict(page_tokens=24), -7), (dict(page_tokens=512), -7),
    (dict(num_requests=8193), -2), (dict(num_pages=1 << 27), -2), (dict(max_pages=1 << 27), -2),
]


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_bad_pages(lib, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages(**kw)
    assert lib.avsg_page_plan(p, at, None, 0, 4, at, at, at, at, None) == code
    assert lib.avsg_tree_keep(p, at, at, 4, at, at, at, None) == code
    assert lib.avsg_rotary_write(p, avsg.avsg_rotary(), None) == code


def test_null_arguments_of_plan_and_keep(lib):
    p, at = pages()
    good = [at, None, 0, 4, at, at, at, at]
    for i in (0, 4, 5, 6, 7):
        assert lib.avsg_page_plan(p, *[None if j == i else x for j, x in enumerate(good)], None) == -1
    assert lib.avsg_page_plan(p, at, None, 0, -1, at, at, at, at, None) == -1
    assert lib.avsg_page_plan(p, at, None, -1, 4, at, at, at, at, None) == -1
    for i in (0, 3, 4, 5):
        args = [at, at, 4, at, at, at]
        args[i] = None
        assert lib.avsg_tree_keep(p, *args, None) == -1
    assert lib.avsg_tree_keep(p, at, at, -1, at, at, at, None) == -1
    assert lib.avsg_page_plan(None, at, None, 0, 4, at, at, at, at, None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(num_q_heads=0), -1), (dict(num_q_heads=3), -1),
    (dict(rot_dim=3), -1), (dict(rot_dim=-2), -1), (dict(rot_offset=-1), -1),
    (dict(rot_dim=64, rot_offset=2), -1), (dict(tokens_per_request=0), -1),
    (dict(tokens_per_request=5), -1), (dict(layer=-1), -1), (dict(layer=2), -1),
    (dict(reserved0=1), -1), (dict(magnitude=math.nan), -1), (dict(q_stride=255), -1),
    (dict(k_stride=127), -1), (dict(v_stride=127), -1), (dict(d_q=None), -1), (dict(d_k=None), -1),
    (dict(d_v=None), -1), (dict(d_freq=None), -1), (dict(d_pos=None), -1), (dict(d_q_out=None), -1),
    (dict(d_q=1), -1), (dict(d_slot=None, num_tokens=129), -2), (dict(num_q_heads=65536 * 2), -2),
])
def test_bad_rotary(lib, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages()
    f = dict(num_tokens=4, num_q_heads=4, rot_dim=64, rot_offset=0, interleaved=0, q_f32=0,
             tokens_per_request=1, layer=1, q_stride=1 << 24, k_stride=128, v_stride=128,
             magnitude=1.0, d_q=at, d_k=at, d_v=at, d_freq=at, d_pos=at, d_slot=at, d_q_out=at)
    f.update(kw)
    assert lib.avsg_rotary_write(p, avsg.avsg_rotary(**f), None) == code


@pytest.mark.parametrize("magnitude,code", [(math.inf, -1), (-math.inf, -1), (math.nan, -1), (-2.0, 0), (0.0, 0)])
def test_magnitudes_are_finite(lib, magnitude, code):
    from decode_serving_gb300 import avsg
    r = avsg.avsg_rotary(num_tokens=0, num_q_heads=4, rot_dim=64, tokens_per_request=1, magnitude=magnitude)
    assert lib.avsg_rotary_write(pages()[0], r, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(q_per_kv=0), -1), (dict(q_per_kv=65), -7), (dict(max_new=0), -1),
    (dict(layer=2), -1), (dict(layer=-1), -1), (dict(window=-1), -1), (dict(softmax_scale=-1.0), -1),
    (dict(softmax_scale=math.inf), -1), (dict(softcap=-1.0), -1), (dict(softcap=math.nan), -1),
    (dict(softcap=3e38), -1),
    (dict(reserved0=1), -1), (dict(q_stride=255), -1), (dict(q_stride=257), -1), (dict(d_q=None), -1),
    (dict(d_q=2), -1), (dict(d_first=None), -1), (dict(d_out=None), -1), (dict(d_out=8), -1),
    (dict(d_work=None), -1), (dict(d_work=128), -1),
])
def test_bad_attention(lib, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages()
    f = dict(num_tokens=4, q_per_kv=2, max_new=4, layer=1, q_stride=256, d_q=at, d_first=at, d_out=at,
             d_work=(at + 255) // 256 * 256, work_bytes=1 << 30)
    f.update(kw)
    assert lib.avsg_tree_attention(p, avsg.avsg_tree(**f), None) == code


@pytest.mark.parametrize("scale,cap,code", [
    (3e38, 0.0, -1), (0.0, 1e-40, -1), (1.0, 1e-39, -1), (1e30, 1e-9, -1), (1e38, 1e30, 0), (1e-38, 1e38, 0),
    (0.0, 1e-37, 0), (2e38, 0.0, 0),
])
def test_factors_of_scores_are_finite(lib, scale, cap, code):
    """What scores are multiplied by: the scale, and twice the scale by the cap, times log2(e)."""
    from decode_serving_gb300 import avsg
    p, at = pages()
    t = avsg.avsg_tree(num_tokens=0, q_per_kv=2, max_new=4, layer=1, softmax_scale=scale, softcap=cap)
    assert lib.avsg_tree_attention(p, t, None) == code


def test_attention_shapes(lib):
    from decode_serving_gb300 import avsg
    n = ctypes.c_size_t()
    assert lib.avsg_tree_attention_workspace(pages(head_dim=96)[0], 4, 1, ctypes.byref(n)) == -7
    assert lib.avsg_tree_attention_workspace(pages()[0], 0, 1, ctypes.byref(n)) == -1
    assert lib.avsg_tree_attention_workspace(pages()[0], 4, 0, ctypes.byref(n)) == -1
    assert lib.avsg_tree_attention_workspace(pages()[0], 4, 1, None) == -1
    assert lib.avsg_tree_attention(pages()[0], None, None) == -1
    assert lib.avsg_tree_attention(pages(page_tokens=3)[0], avsg.avsg_tree(q_per_kv=1, max_new=1), None) == -7
    assert lib.avsg_tree_attention(pages()[0], avsg.avsg_tree(q_per_kv=1, max_new=1), None) == 0


def test_no_tokens_is_no_work(lib):
    from decode_serving_gb300 import avsg
    p, _ = pages()
    assert lib.avsg_rotary_write(p, avsg.avsg_rotary(num_tokens=0, num_q_heads=4, rot_dim=64,
                                                     tokens_per_request=1, magnitude=1.0), None) == 0


def test_struct_layouts(tmp_path):
    from decode_serving_gb300 import avsg
    names = [("avsg_pages", "d_k"), ("avsg_pages", "d_error"), ("avsg_rotary", "q_stride"),
             ("avsg_rotary", "magnitude"), ("avsg_rotary", "d_q_out"), ("avsg_tree", "q_stride"),
             ("avsg_tree", "d_first"), ("avsg_tree", "work_bytes")]
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "avsg.h"\nint main(void){'
                   + "".join(f'printf("%zu %zu\\n", sizeof({s}), offsetof({s}, {f}));' for s, f in names)
                   + "return 0;}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    want = [x for s, f in names for x in (ctypes.sizeof(getattr(avsg, s)), getattr(getattr(avsg, s), f).offset)]
    assert [int(x) for x in got] == want


@pytest.mark.parametrize("rot,base,kw", [
    (2, 10000.0, {}), (128, 10000.0, {}), (64, 5e5, dict(factor=4.0)),
    (128, 10000.0, dict(factor=32.0, low_turns=1.0, high_turns=32.0, original=32768)),
    (24, 1e6, dict(factor=8.0, low_turns=1.0, high_turns=4.0, original=8192)),
])
def test_rotary_frequencies(lib, rot, base, kw):
    from decode_serving_gb300 import avsg
    got = avsg.avsg_rotary_frequencies(rot, base, **kw)
    two_pi = Fraction(6283185307179586476925286766559005768, 10**36)
    assert len(got) == rot // 2
    for i, word in enumerate(got):
        w = base ** (-2.0 * i / rot)
        factor = kw.get("factor", 1.0)
        if kw.get("original"):
            turns = kw["original"] * w / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - kw["low_turns"]) / (kw["high_turns"] - kw["low_turns"])))
            w *= keep + (1 - keep) / factor
        else:
            w /= factor
        want = Fraction(w) / two_pi * 2**64
        # powers, ramp and division in 64 bits: a few steps of 2^-53 each (a pow of at most 1 ulp
        # on either side included), 16 of them in all
        assert abs(Fraction(int(word)) - want) <= want * Fraction(16, 2**53) + 1


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=3), dict(base=1.0), dict(base=math.nan),
                                dict(factor=0.5), dict(original=-1.0),
                                dict(original=4096.0, low_turns=4.0, high_turns=4.0)])
def test_bad_frequencies(lib, kw):
    from decode_serving_gb300 import avsg
    f = dict(rot=64, base=10000.0, factor=1.0, low_turns=1.0, high_turns=32.0, original=0.0)
    f.update(kw)
    with pytest.raises(avsg.AvsgError):
        avsg.avsg_rotary_frequencies(f["rot"], f["base"], f["factor"], f["low_turns"],
                                     f["high_turns"], f["original"])


def test_the_cache_wants_cuda_tensors():
    import torch
    from decode_serving_gb300.paged import PagedCache
    z = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(1, 1, 1, 1, 8, dtype=torch.bfloat16),
                   torch.zeros(1, 1, 1, 1, 8, dtype=torch.bfloat16), z[None], z, z, z)
    with pytest.raises(ValueError):
        PagedCache(torch.zeros(1, 1, 1, 1, 8), torch.zeros(1, 1, 1, 1, 8), z[None], z, z, z)
