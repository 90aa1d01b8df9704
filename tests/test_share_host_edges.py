"""What a user reads about the operators of shared pages, and their host-side arithmetic (no GPU)."""
import math
import os
import random
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "decode_serving_gb300", "csrc")
MOST = 2**31 - 1


def test_the_documentation_says_when_to_compact():
    from decode_serving_gb300.paged import PagedCache
    for f in (PagedCache.fork, PagedCache.compact):
        assert "between steps, when every token is" in " ".join(f.__doc__.split()).lower()


@pytest.fixture(scope="module")
def split(tmp_path_factory):
    """Runs part_cost and first_sms on the host: lines of numbers in, a number each out."""
    from decode_serving_gb300 import build
    at = tmp_path_factory.mktemp("split")
    (at / "split.cu").write_text(r"""
#include <stdio.h>
#include "avsg_tree_attn.cuh"
int main() {
  char what;
  while (scanf(" %c", &what) == 1) {
    avsg::TreeArgs a{};
    if (what == 'c') {
      int part, len, shared, first[2], group[2];
      avsg::TreeArgs::Cost c{};
      if (scanf("%d %d %d %d %d %d %d %d %d %d %d %d %d", &part, &len, &shared, &first[0], &first[1], &group[0],
                &group[1], &a.window, &c.keys, &c.tpm, &c.begin, &c.tile, &c.small) != 13) return 1;
      a.len = &len, a.shared = &shared, a.first = first, a.group_first = group;
      a.cost[part] = c;
      printf("%.9g\n", avsg::tree::part_cost(a, part, 0));
    } else {
      float c0, c1;
      if (scanf("%d %d %f %f", &a.sms, &a.lead, &c0, &c1) != 4) return 1;
      printf("%d\n", avsg::tree::first_sms(a, c0, c1));
    }
  }
  return 0;
}
""")
    subprocess.run([build._nvcc()] + build.NVCC_FLAGS + ["-o", str(at / "split"), str(at / "split.cu")], check=True)

    def run(lines):
        text = "\n".join(" ".join(str(x) for x in line) for line in lines)
        out = subprocess.run([str(at / "split")], input=text, capture_output=True, text=True, check=True).stdout
        return [float(x) for x in out.split()]
    return run


def cost(part, length, shared, first, group, window, keys, tpm, begin, tile, small):
    """The same in whole numbers."""
    if part == 0:
        n, k = (group[1] - group[0] if shared else 0), min(shared, window or shared)
    else:
        n = first[1] - first[0]
        k = min(length - shared, window or length) + min(n, 64)
    tiles, full, rest = -(-k // keys), n // tpm, n % tpm
    return begin * (full + (rest > 0)) + tiles * (full * tile + (0 if rest == 0 else tile if 2 * rest > tpm else small))


def test_the_parts_costs_hold_up_to_the_longest_requests(split):
    r = random.Random(4)
    cases = []
    for length in (1, 63, 1000, 2**20 + 1, MOST - 1025, MOST - 1024, MOST - 255, MOST - 1, MOST):
        for shared in {0, min(length, 16), length // 2, length - length % 256, length}:
            for n in (1, 3, 64, 65, 4096, 1 << 22):
                for window in (0, 1, 300, MOST):
                    for part in (0, 1):
                        keys, tpm = r.choice((64, 128)), r.choice((1, 4, 64, 256))
                        cases.append((part, length, shared, (7, 7 + n), (5, 5 + 3 * n), window, keys, tpm, 950, 158, 105))
    got = split(["c", c[0], c[1], c[2], *c[3], *c[4], *c[5:]] for c in cases)
    assert len(got) == len(cases)
    for c, g in zip(cases, got):
        want = cost(*c)
        # Keys are counted up to 2^31 - 1025: at most 1024 + 64 fewer of over 2^31, 16 of 2^25 tiles (2^-20).  Five
        # conversions, two products and two sums of positive numbers in fp32, at most half a step (2^-24) each, and the
        # print's nine digits (2^-24 too).
        assert math.isfinite(g) and abs(g - want) <= (2.0**-20 + 10 * 2.0**-24) * want, (c, g, want)


def test_the_split_of_the_sms(split):
    r = random.Random(5)
    cases = [(152, lead, c0, c1) for lead in (0, 550, 2000) for c0 in (0, 1, 600, 1e5, 1e9, 1e13, 1e17) for c1 in (0, 1, 600, 1e5, 1e9, 1e13, 1e17)]
    cases += [(r.choice((1, 2, 148, 152)), r.randrange(1000), 10 ** r.uniform(2, 12), 10 ** r.uniform(2, 12)) for _ in range(500)]
    for (sms, lead, c0, c1), k in zip(cases, split(["s", *c] for c in cases)):
        k = int(k)
        if c0 == 0 or c1 == 0:
            assert k == (0 if c0 == 0 else sms)
            continue
        if sms == 1:                                       # (no room for two: the first part's one CTA has it)
            assert k in (0, 1)
            continue
        assert 1 <= k <= sms - 1
        # The fewest with which part 0 ends no later than part 1; a dozen roundings of 2^-24 and a root that loses
        # half of them: 2^-10 of an SM's share is far more.
        lead = min(lead, 0.5 * (c0 + c1) / sms)
        late = lambda k: c0 / k + lead - c1 / (sms - k)  # noqa: E731
        slack = 2.0**-10 * (c0 / k + c1 / (sms - k))
        assert k == sms - 1 or late(k) <= slack, (sms, lead, c0, c1, k)
        assert k == 1 or late(k - 1) >= -slack, (sms, lead, c0, c1, k)
