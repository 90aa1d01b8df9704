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
