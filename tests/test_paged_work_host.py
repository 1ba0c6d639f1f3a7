"""The lengths by which the paged attention cuts its work (csrc/paged_work.cuh), run on the CPU against sums over the
tokens."""
import os
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
  int i, R;
  if (scanf("%d", &R) == 1 && R > 0) {  // a batch: its length as the kernels add it up, and the host's bound
    scanf("%d %d %d %d %d", &a.causal, &a.tpt, &a.T, &a.Hkv, &a.max_keys);
    int sum = 0;
    for (int r = 0; r < R; ++r) {
      scanf("%d %d", &q.n, &q.len);
      const int nt = tiles_of(a, q);
      if (nt) sum = add_len(sum, a.Hkv * tiles_len(a, q, nt, nt));
    }
    printf("%d %.1f\n", sum, fa::most_blocks(a.T, R, a.Hkv, a.tpt, a.max_keys));
    return 0;
  }
  while (scanf("%d %d %d %d %d", &a.causal, &a.tpt, &q.n, &q.len, &i) == 5) {
    const int nt = (q.n + a.tpt - 1) / a.tpt;
    printf("%d %d\n", tiles_len(a, q, i, nt), keys_seen(a, q, i * a.tpt));
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def lengths(tmp_path_factory):
    d = tmp_path_factory.mktemp("work")
    (d / "driver.cu").write_text(DRIVER)
    exe = str(d / "driver")
    subprocess.check_call([build.nvcc()] + build.ARCH + build.FLAGS + ["-I", build.CSRC, str(d / "driver.cu"), "-o", exe])

    def run(cases, batch=0):
        out = subprocess.run([exe], input=f"{batch}\n" + "\n".join(" ".join(map(str, c)) for c in cases),
                             capture_output=True, text=True, check=True).stdout.split()
        return [(int(a), float(b)) for a, b in zip(out[::2], out[1::2])]
    return run


def keys_of(causal, tpt, n, length, k):
    """Keys that the last token of tile k sees."""
    return max(0, length - n + min((k + 1) * tpt, n)) if causal else length


def test_lengths_are_sums_over_the_tiles(lengths):
    """Each tile counts for at least the keys it streams, all up to it for at most their number times the request's keys;
    exactly for the former where every token sees a key."""
    rng = random.Random(5)
    cases = []
    for _ in range(3000):
        tpt, n = rng.choice([1, 2, 3, 4, 8, 25, 32, 64, 128, 256]), rng.choice([1, 2, 31, 32, 33, 127, 700, rng.randint(1, 3000)])
        length = rng.choice([0, 1, n - 1, n, n + 1, n + rng.randint(0, 9000), rng.randint(0, n)])
        i = rng.randrange(-(-n // tpt))
        cases += [(rng.randint(0, 1), tpt, n, length, i)] * 2
        cases[-1] = cases[-1][:4] + (i + 1,)
    got = lengths(cases)
    for c, (a, _), (b, seen) in zip(cases[::2], got[::2], got[1::2]):
        causal, tpt, n, length, i = c
        keys = [keys_of(*c[:4], k) for k in range(i + 1)]
        assert seen == keys[-1], c
        assert b - a - 2 >= keys[-1] // 128 and b <= length * (i + 1) // 128 + 2 * (i + 1), c
        if not causal or length >= n:
            assert (a, b) == (sum(keys[:-1]) // 128 + 2 * i, sum(keys) // 128 + 2 * (i + 1)), c


def test_tokens_without_keys_count_few_blocks(lengths):
    """2^21 new tokens of which only the last 128 see a key: their tiles count for no more than the keys there are, not
    for what a text of 2^21 tokens would make them (8 heads of which were more blocks than 32 bits hold)."""
    n, tpt = 1 << 21, 32
    (got, _), = lengths([(1, tpt, n, 128, n // tpt)])
    assert 2 * (n // tpt) <= got <= 3 * (n // tpt)


def test_batches_stay_within_the_hosts_count(lengths):
    """Requests that share no rows never come to more blocks than the host admits a call by; requests that do are added
    up without an overflow."""
    rng = random.Random(6)
    for _ in range(60):
        R, tpt, keys = rng.choice([1, 2, 7, 200]), rng.choice([1, 4, 32, 256]), rng.choice([16, 1000, 70000])
        n = [rng.choice([0, 1, rng.randint(0, 600)]) for _ in range(R)]
        lens = [rng.choice([0, keys, rng.randint(0, keys)]) for _ in range(R)]
        T, Hkv = max(1, sum(n) + rng.randint(0, 3)), rng.choice([1, 8])
        (got, most), = lengths([(rng.randint(0, 1), tpt, T, Hkv, keys)] + list(zip(n, lens)), batch=R)
        assert got <= int(most), (R, tpt, keys)
    # every other request has all T rows
    T, R, keys = 1 << 16, 512, 131072
    (got, most), = lengths([(0, 32, T, 8, keys)] + [(T, keys), (0, keys)] * (R // 2), batch=R)
    assert got == 2 ** 31 - 1 > most
