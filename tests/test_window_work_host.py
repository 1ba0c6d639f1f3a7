"""How a tile's key blocks under a window are counted and laid out (csrc/paged_work.cuh), on the CPU against the keys that
its tokens see, one by one."""
import random
import subprocess

import pytest

from exact_io_aware_32_gb300 import build

DRIVER = r"""
#include <cstdio>
#include "paged_work.cuh"
using namespace fa::paged;
int main() {
  fa::PagedArgs a{};
  Request q{};
  int tile;
  a.causal = 1;
  while (scanf("%d %d %d %d %d %d %d", &a.window, &a.sinks, &a.tpt, &q.n, &q.len, &tile, &a.page_shift) == 7) {
    const int nt = (q.n + a.tpt - 1) / a.tpt;
    const Band b = band_of(a, q, tile * a.tpt);
    int keys = keys_seen(a, q, (tile + 1) * a.tpt);
    if (keys) keys -= b.gap;
    printf("%d %d %d %d %d %d %d\n", b.sunk, b.skip, b.gap, b.low, keys, tiles_len<true>(a, q, tile, nt), tiles_len<true>(a, q, tile + 1, nt));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def bands(tmp_path_factory):
    d = tmp_path_factory.mktemp("band")
    (d / "driver.cu").write_text(DRIVER)
    exe = str(d / "driver")
    subprocess.check_call([build.nvcc()] + build.ARCH + build.FLAGS + ["-I", build.CSRC, str(d / "driver.cu"), "-o", exe])

    def run(cases):
        out = subprocess.run([exe], input="\n".join(" ".join(map(str, c)) for c in cases), capture_output=True, text=True, check=True)
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    return run


def test_bands_hold_what_the_tokens_see(bands):
    rng = random.Random(1)
    cases = []
    for _ in range(3000):
        tpt, n = rng.choice([1, 2, 4, 8, 25, 32, 64, 128, 256]), rng.choice([1, 2, 31, 33, 127, rng.randint(1, 600)])
        length = rng.choice([0, 1, n - 1, n, n + 1, n + rng.randint(0, 3000), rng.randint(0, n)])
        window, sinks = rng.choice([1, 2, 127, 128, 129, rng.randint(1, 2000), 10 ** 9]), rng.choice([0, 1, 4, 127, 128, 129, 400])
        cases.append((window, sinks, tpt, n, length, rng.randrange(-(-n // tpt)), rng.choice([4, 5, 6, 7, 8])))
    for c, (sunk, skip, gap, low, keys, before, after) in zip(cases, bands(cases)):
        window, sinks, tpt, n, length, tile, shift = c
        ps = 1 << shift
        assert gap == skip * ps
        at = [x if x < sunk * ps else x + gap for x in range(keys)]  # the request's key that stands in each place
        seen = set()
        for i in range(tile * tpt, min(n, (tile + 1) * tpt)):
            p = length - n + i
            mine = {j for j in range(p + 1) if p - j < window or j < sinks}
            seen |= mine
            if i in (tile * tpt, min(n, (tile + 1) * tpt) - 1):  # the kernels' rule, in places
                assert {x for x in range(keys) if x <= p - gap and not (x <= p - gap - min(window, length) and x >= sinks)} == \
                    {x for x, j in enumerate(at) if j in mine}, c
        assert seen <= set(at), c
        if length - n + tile * tpt >= 0:  # (else the first token sees no key)
            first = max(0, length - n + tile * tpt - window + 1)
            assert low == first - gap and {j // ps for j in at} == {j // ps for j in seen}, c
        # the bound by which calls without any cut are chosen
        assert keys <= -(-sinks // ps) * ps + window + tpt + ps - 2, c
        assert 2 <= after - before <= -(-keys // 128) + 5, c


def test_widths_near_32_bits(bands):
    """Windows and sinks as wide as they come, tokens that see no key."""
    big = 2 ** 31 - 512
    for n, length in ((1, big), (4000, big), (1 << 20, 0), (1 << 20, 5), (1, 1)):
        for window in (1, 1000, big):
            (sunk, skip, gap, low, keys, before, after), = bands([(window, big, 32, n, length, 0, 7)])
            first = max(length - n - min(window, length) + 1, 0)
            assert low == first and skip == gap == 0 and sunk == first // 128, (n, length, window)
            assert after - before >= 2
