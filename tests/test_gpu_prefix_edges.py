"""avsg_prefix_attention where its groups do not fit the step: what is latched, what is written."""
import pytest
import torch

from test_gpu_paged import BF16, F16
from test_gpu_prefix_attention import Shared

pytestmark = pytest.mark.gpu


def two_groups(new, dim, dtype):
    """Four requests in two groups, a good call's output, and the second group taken off the list."""
    s = Shared([100, 90, 130, 70], new, 16, 2, 4, dim, dtype, False, [((0, 1), 5), ((2, 3), 4)])
    s.attend()
    s.check()
    want = s.out.clone(), s.lse.clone()
    s.x.first[3:] = s.x.first[2].clone()
    return s, want


# 8 heads: four warps join a row of up to 190 tokens, two of up to 380, one of more (152 SMs)
@pytest.mark.parametrize("new", [[4, 2, 3, 1], [90, 70, 60, 60], [150, 150, 150, 150]])
@pytest.mark.parametrize("dim,dtype", [(64, F16), (128, BF16), (256, BF16)])
def test_rows_that_fail_beside_rows_that_do_not(new, dim, dtype):
    """The join comes to its end whichever of its warps sees the error first, and writes a row whole or not at all."""
    s, want = two_groups(new, dim, dtype)
    work = s.cache.attend_prefixes_workspace(4, max(new), s.total)
    listed = (new[0] + new[1]) * 8
    rows = [(x[:s.total].reshape(s.total * 8, -1).float(), off) for x, off in
            # A row is cut elsewhere than in the good call.  out: either rounds its weights and its result to the type,
            # half a step each, of means of values within 6.  lse: the sums of up to 280 weights in another order (half
            # a step of fp32 each), exp2 (2^-20 in all), the logarithm, its product and sum (a step of 8 each).
            ((want[0], 2 * 6 * 2 * torch.finfo(dtype).eps / 2 * 1.01),
             (want[1], 2 * (280 * 2.0**-24 + 2.0**-20 + 3 * 8 * 2.0**-23)))]
    for _ in range(50):
        work.fill_(255)
        s.out.fill_(9.0), s.lse.fill_(99.0)                # (no value of either)
        s.attend(work=work)
        assert s.cache.error()[0] == -4                    # (waits for the device)
        for x, mark, (good, off) in zip((s.out, s.lse), (9.0, 99.0), rows):
            got = x[:s.total].reshape(s.total * 8, -1).float()
            left, right = (got == mark).all(1), ((got - good).abs() <= off).all(1)
            assert left[listed:].all() and (left | right).all()
        s.cache.clear_error()


@pytest.mark.parametrize("dim,dtype,page,new", [(64, F16, 16, [4, 2, 3, 1]), (128, BF16, 16, [90, 70, 60, 60]),
                                                (256, BF16, 16, [3, 3, 2, 64]), (128, F16, 4, [4, 2, 3, 1])])
@pytest.mark.parametrize("what", ["list", "token", "twice", "leader", "length", "member"])
@pytest.mark.parametrize("work", ["reused", "zeros", "ones"])
def test_a_token_that_no_group_of_its_prefix_lists(dim, dtype, page, new, what, work):
    """It is latched whatever the workspace holds: a good call's entries for the same tokens, above all."""
    s = Shared([100, 90, 130, 70], new, page, 2, 4, dim, dtype, False, [((0, 1), 80 // page), ((2, 3), 64 // page)])
    scratch = s.cache.attend_prefixes_workspace(4, max(new), s.total)
    s.attend(work=scratch)
    s.check()
    if work != "reused":
        scratch.fill_(0 if work == "zeros" else 255)
    x = s.x
    if what == "list":                                     # the second group has no list
        x.first[3:] = x.first[2].clone()
    elif what == "token":                                  # another's token in the place of one
        x.token[0] = x.token[1].clone()
    elif what == "twice":                                  # the first request's list, in both groups
        x.token[int(x.first[2]):int(x.first[2]) + new[0]] = x.token[:new[0]].clone()
    elif what == "leader":                                 # the leader has no prefix, its members have
        x.shared[2] = 0
    elif what == "length":                                 # nor one of their length
        x.shared[0] = 64
    elif what == "member":
        x.shared[1] = 64
    s.attend(work=scratch)
    assert s.cache.error()[0] == -4


def test_prefixes_that_are_switched_off():
    """Without tokens in their prefixes, groups are lists that nobody reads: every request is alone."""
    s = Shared([100, 90, 130, 70], [4, 2, 3, 1], 16, 2, 4, 128, BF16, True, [((0, 1), 5), ((2, 3), 4)])
    work = s.cache.attend_prefixes_workspace(4, 4, s.total)
    s.attend(work=work)
    s.x.shared.zero_()
    s.attend(work=work)
    s.check()
    s.find()
    s.x.shared[2:] = 0                                     # one group of two
    s.attend(work=work)
    s.check()


def test_groups_of_an_earlier_step_are_latched():
    """Arrays that were found before another request joined the step."""
    s = Shared([100, 90, 130, 70], [4, 2, 0, 1], 16, 2, 4, 128, BF16, True, [((0, 1, 2), 5)])
    work = s.cache.attend_prefixes_workspace(4, 8, 20)
    s.attend(work=work, most=8)
    s.check()
    x = s.cache.prefix_arrays(20)
    s.cache.find_prefixes(s.first, x, s.cache.prefix_workspace(), min_tokens=1)
    s.x, x = x, s.x
    s.attend(work=work, most=8)
    s.check()                                              # (a longer list gives the same)
    s.x.shared[2] = 80                                     # what a step in which request 2 has a token would find
    s.first[3:] += 1
    s.q = torch.cat([s.q, s.q[:1]])
    s.out, s.lse, s.dmask = (torch.cat([t, t[:1]]) for t in (s.out, s.lse, s.dmask))
    s.attend(work=work, most=8)
    assert s.cache.error()[0] == -4
