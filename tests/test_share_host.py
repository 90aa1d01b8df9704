"""The entry points of shared pages reject bad arguments on the host, before any
CUDA call; the plain definitions that the GPU tests hold them to keep every page's count."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import share_reference as ref
from conftest import ROOT
from test_paged_host import BAD_PAGES, pages


def prefixes(at, **kw):
    from decode_serving_gb300 import avsg
    f = dict(num_tokens=4, reserved0=0, d_leader=at, d_shared=at, d_first=at, d_token=at, d_request=at)
    f.update(kw)
    return avsg.avsg_prefixes(**f)


def aligned(at):
    return (at + 255) // 256 * 256


@pytest.mark.parametrize("kw,code", BAD_PAGES)
def test_bad_pages(lib, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages(**kw)
    n, work = ctypes.c_size_t(), aligned(at)
    assert lib.avsg_page_fork_workspace(p, ctypes.byref(n)) == code
    assert lib.avsg_page_fork(p, at, at, work, 1 << 40, None) == code
    assert lib.avsg_page_compact_workspace(p, ctypes.byref(n)) == code
    assert lib.avsg_page_compact(p, at, at, at, at, at, work, 1 << 40, None) == code
    assert lib.avsg_prefix_find_workspace(p, ctypes.byref(n)) == code
    assert lib.avsg_prefix_find(p, at, 1, prefixes(at), work, 1 << 40, None) == code
    assert lib.avsg_tree_keep_shared(p, at, at, at, 4, at, at, at, None) == code
    assert lib.avsg_rotary_write_axes(p, avsg.avsg_rotary(), 1, at, None) == code
    t = avsg.avsg_tree(q_per_kv=1, max_new=1)
    assert lib.avsg_prefix_attention(p, t, prefixes(at), None) == code
    assert lib.avsg_prefix_attention_workspace(p, 1, 1, 1, ctypes.byref(n)) == code


def test_null_and_misaligned_arguments(lib):
    p, at = pages()
    work = aligned(at)
    for i, bad in ((0, None), (1, None), (2, None), (2, work + 128)):
        args = [at, at, work]
        args[i] = bad
        assert lib.avsg_page_fork(p, *args, 1 << 40, None) == -1
    for i, bad in ((0, None), (1, None), (2, None), (3, None), (4, None), (5, None), (5, work + 16)):
        args = [at, at, at, at, at, work]
        args[i] = bad
        assert lib.avsg_page_compact(p, *args, 1 << 40, None) == -1
    for kw in (dict(num_tokens=-1), dict(reserved0=1), dict(d_leader=None), dict(d_shared=None), dict(d_first=None),
               dict(d_token=None), dict(d_request=None)):
        assert lib.avsg_prefix_find(p, at, 1, prefixes(at, **kw), work, 1 << 40, None) == -1
    assert lib.avsg_prefix_find(p, None, 1, prefixes(at), work, 1 << 40, None) == -1
    assert lib.avsg_prefix_find(p, at, -1, prefixes(at), work, 1 << 40, None) == -1
    assert lib.avsg_prefix_find(p, at, 1, None, work, 1 << 40, None) == -1
    assert lib.avsg_prefix_find(p, at, 1, prefixes(at), work + 1, 1 << 40, None) == -1
    for f in (lib.avsg_page_fork_workspace, lib.avsg_page_compact_workspace, lib.avsg_prefix_find_workspace):
        assert f(p, None) == -1
    assert lib.avsg_tree_keep_shared(p, None, at, at, 4, at, at, at, None) == -1
    for i in (0, 3, 4, 5):
        args = [at, at, 4, at, at, at]
        args[i] = None
        assert lib.avsg_tree_keep_shared(p, at, *args, None) == -1


def test_workspaces_that_are_too_small(lib):
    p, at = pages()
    work, n = aligned(at), ctypes.c_size_t()
    for size, call in ((lib.avsg_page_fork_workspace, lambda b: lib.avsg_page_fork(p, at, at, work, b, None)),
                       (lib.avsg_page_compact_workspace,
                        lambda b: lib.avsg_page_compact(p, at, at, at, at, at, work, b, None)),
                       (lib.avsg_prefix_find_workspace,
                        lambda b: lib.avsg_prefix_find(p, at, 1, prefixes(at), work, b, None))):
        assert size(p, ctypes.byref(n)) == 0 and n.value > 0
        assert call(n.value - 1) == -2


def test_wide_tables_are_refused(lib):
    p, at = pages(page_tokens=1, max_pages=(1 << 30) + 1)
    n, work = ctypes.c_size_t(), aligned(at)
    assert lib.avsg_page_fork_workspace(p, ctypes.byref(n)) == -2
    assert lib.avsg_page_fork(p, at, at, work, 1 << 60, None) == -2
    assert lib.avsg_page_compact(p, at, at, at, at, at, work, 1 << 60, None) == -2
    assert lib.avsg_prefix_find(p, at, 1, prefixes(at), work, 1 << 60, None) == -2


@pytest.mark.parametrize("axes,axis,kw,code", [
    (0, True, {}, -1), (-3, True, {}, -1), (2, False, {}, -1), (2, True, dict(rot_dim=3), -1),
    (2, True, dict(num_tokens=0), 0), (2, False, dict(num_tokens=0, rot_dim=0), 0), (2, True, dict(q_stride=255), -1),
])
def test_bad_axes(lib, axes, axis, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages()
    f = dict(num_tokens=4, num_q_heads=4, rot_dim=64, tokens_per_request=1, layer=1, q_stride=1 << 24, k_stride=128,
             v_stride=128, magnitude=1.0, d_q=at, d_k=at, d_v=at, d_freq=at, d_pos=at, d_slot=at, d_q_out=at)
    f.update(kw)
    assert lib.avsg_rotary_write_axes(p, avsg.avsg_rotary(**f), axes, at if axis else None, None) == code
    assert lib.avsg_rotary_write_axes(p, None, 1, at, None) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(num_tokens=-1), -1), (dict(q_per_kv=0), -1), (dict(q_per_kv=65), -7), (dict(max_new=0), -1),
    (dict(layer=2), -1), (dict(window=-1), -1), (dict(softcap=-1.0), -1), (dict(reserved0=1), -1),
    (dict(q_stride=257), -1), (dict(d_q=None), -1), (dict(d_first=None), -1), (dict(d_out=8), -1),
    (dict(d_work=128), -1),
])
def test_bad_attention(lib, kw, code):
    from decode_serving_gb300 import avsg
    p, at = pages()
    f = dict(num_tokens=4, q_per_kv=2, max_new=4, layer=1, q_stride=256, d_q=at, d_first=at, d_out=at,
             d_work=aligned(at), work_bytes=1 << 40)
    f.update(kw)
    assert lib.avsg_prefix_attention(p, avsg.avsg_tree(**f), prefixes(at), None) == code


def test_attention_wants_its_groups(lib):
    from decode_serving_gb300 import avsg
    p, at = pages()
    t = avsg.avsg_tree(num_tokens=0, q_per_kv=2, max_new=4, layer=1)
    assert lib.avsg_prefix_attention(p, t, prefixes(at), None) == 0
    assert lib.avsg_prefix_attention(p, t, None, None) == -1
    assert lib.avsg_prefix_attention(p, None, prefixes(at), None) == -1
    for kw in (dict(num_tokens=-1), dict(reserved0=1)):
        assert lib.avsg_prefix_attention(p, t, prefixes(at, **kw), None) == -1
    n = ctypes.c_size_t()
    assert lib.avsg_prefix_attention_workspace(pages(head_dim=96)[0], 4, 1, 1, ctypes.byref(n)) == -7
    assert lib.avsg_prefix_attention_workspace(p, 4, 1, -1, ctypes.byref(n)) == -1
    assert lib.avsg_prefix_attention_workspace(p, 4, 1, 1, None) == -1


def test_struct_layout(tmp_path):
    from decode_serving_gb300 import avsg
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "avsg.h"\nint main(void){'
                   'printf("%zu %zu %zu\\n", sizeof(avsg_prefixes), offsetof(avsg_prefixes, d_leader),'
                   ' offsetof(avsg_prefixes, d_request)); return 0;}\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    x = avsg.avsg_prefixes
    assert [int(v) for v in got] == [ctypes.sizeof(x), x.d_leader.offset, x.d_request.offset]


def test_rotary_axes():
    from decode_serving_gb300.paged import rotary_axes
    assert rotary_axes([2, 3]).tolist() == [0, 0, 1, 1, 1]
    assert rotary_axes([2, 3, 1], dealt=True).tolist() == [0, 1, 2, 0, 1, 1]
    assert rotary_axes([0, 2], dealt=True).tolist() == [1, 1]
    for bad in ([], [1, -1]):
        with pytest.raises(ValueError):
            rotary_axes(bad)


def test_the_fork_of_the_definition_keeps_count_of_pages():
    """A worked example, and the count of holders in a run of random forks."""
    lens, tables = np.array([5, 0, 7]), np.array([[3, 1], [9, 9], [0, 2]])
    k = np.arange(6 * 4.0).reshape(1, 6, 1, 4, 1)
    free, shares = np.array([5, 4, -1, -1, -1, -1]), np.zeros(6, int)
    # request 1 becomes a copy of 0 (its page 1, a row of it filled, is copied to page 4); 2 ends
    got = ref.fork(lens, [0, 0, -1], tables, free, 2, shares, 4, [k])
    assert got[0].tolist() == [5, 5, 0] and got[1].tolist() == [[3, 1], [3, 4], [0, 2]]
    assert got[3] == 3 and got[2][:3].tolist() == [5, 2, 0] and got[4].tolist() == [0, 0, 0, 1, 0, 0]
    assert k[0, 4, 0, :, 0].tolist() == [4, 17, 18, 19]
    r = np.random.default_rng(1)
    lens, tables = r.integers(0, 20, 9), np.full((9, 6), -1)
    free, shares, count = r.permutation(120), np.zeros(120, int), 120
    for i, n in enumerate(lens):
        for x in range(-(-int(n) // 4)):
            count -= 1
            tables[i, x] = free[count]
    for _ in range(20):
        parent = np.where(r.random(9) < 0.4, np.arange(9), r.integers(-1, 9, 9))
        lens, tables, free, count, shares = ref.fork(lens, parent, tables, free, count, shares, 4, [])
        holders = np.zeros(120, int)
        for i, n in enumerate(lens):
            np.add.at(holders, tables[i, :-(-int(n) // 4)], 1)
        assert (shares == np.maximum(holders - 1, 0)).all()
        assert sorted(free[:count].tolist()) == np.nonzero(holders == 0)[0].tolist()
