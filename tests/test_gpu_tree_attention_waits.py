"""A wait inside the tcgen05 kernel that gives up: the call latches AVSG_ERR_TIMEOUT and ends, with every
copy and product that it had issued awaited, and the context serves the next calls.  In the bounds-checked
build (a child process: the library is chosen once), whose waits can be given no time at all."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

SCRIPT = r"""
import sys
sys.path.insert(0, {tests!r})
import torch
from decode_serving_gb300 import avsg
from test_gpu_paged import BF16, F16
from test_gpu_tree_attention import Step
assert avsg.load_library()._name.endswith("libavsg_debug.so")
gave_up = 0
for dim, dtype in ((64, F16), (128, BF16), (256, BF16)):
    for lens, new, groups in (([300], [12], 4), ([3000, 40, 0], [12, 5, 40], 4), ([700, 5000], [64, 9], 16),
                              ([i * 20 for i in range(200)], [9] * 200, 8)):
        s = Step(lens, new, 16, 2, groups, dim, dtype, True)
        for _ in range(3):
            s.attend()
            code = s.cache.error()[0]
            assert code in (0, -5), code
            if code == 0:                             # nothing had to wait
                s.check(only={{0}})
            gave_up += code != 0
            s.cache.clear_error()
        few = Step([63, 300], [1, 2], 4, 2, 4, dim, dtype, False)
        few.attend()                                  # mma.sync, which has no such waits
        few.check()
print("gave up", gave_up)
"""


@pytest.fixture(scope="module")
def debug_lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from decode_serving_gb300 import build
    return build.build(debug_bounds=True)


@pytest.mark.parametrize("clocks", ["0", "2000", ""])
def test_waits_that_give_up_end_the_call_with_an_error(debug_lib, clocks):
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, AVSG_LIBRARY=debug_lib, AVSG_TREE_WAIT_CLOCKS=clocks)
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(tests=here)], cwd=os.path.dirname(here), env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "gave up" in r.stdout, r.stdout[-2000:] + r.stderr[-3000:]
    gave_up = int(r.stdout.split()[-1])
    assert gave_up > 0 if clocks == "0" else gave_up == 0 if clocks == "" else gave_up >= 0
