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
  while (scanf("%d %d %d %d %d %d", &a.window, &a.sinks, &a.tpt, &q.n, &q.len, &tile) == 6) {
    const int nt = (q.n + a.tpt - 1) / a.tpt;
    const Band b = band_of(a, q, tile * a.tpt);
    int nb = (keys_seen(a, q, (tile + 1) * a.tpt) + 127) >> 7;
    if (nb) nb -= b.skip;
    printf("%d %d %d %d %d %d\n", b.sunk, b.skip, b.low, nb, tiles_len<true>(a, q, tile, nt), tiles_len<true>(a, q, tile + 1, nt));
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
        cases.append((window, sinks, tpt, n, length, rng.randrange(-(-n // tpt))))
    for c, (sunk, skip, low, nb, before, after) in zip(cases, bands(cases)):
        window, sinks, tpt, n, length, tile = c
        at = [j if j < sunk else j + skip for j in range(nb)]
        assert at == sorted(set(at)), c
        seen, lowest = set(), None
        for i in range(tile * tpt, min(n, (tile + 1) * tpt)):
            p = length - n + i
            if p >= 0:
                seen |= {j // 128 for j in range(max(0, p - window + 1), p + 1)} | {j // 128 for j in range(min(sinks, p + 1))}
                lowest = max(0, p - window + 1) if lowest is None else min(lowest, max(0, p - window + 1))
        assert seen <= set(at), c
        if lowest is not None and length - n + tile * tpt >= 0:  # (else the first token sees no key)
            assert low == lowest and (set(at) <= seen), c
        if at:  # the bound by which calls without any cut are chosen
            assert nb <= -(-sinks // 128) + (window + tpt + 126) // 128 + 1, c
        assert 2 <= after - before <= nb + 5, c


def test_widths_near_32_bits(bands):
    """Windows and sinks as wide as they come, tokens that see no key."""
    big = 2 ** 31 - 512
    for n, length in ((1, big), (4000, big), (1 << 20, 0), (1 << 20, 5), (1, 1)):
        for window in (1, 1000, big):
            (sunk, skip, low, nb, before, after), = bands([(window, big, 32, n, length, 0)])
            p = length - n
            w = min(window, length)
            assert low == max(p - w + 1, 0) and skip == 0 and sunk == low // 128, (n, length, window)
            assert after - before >= 2
