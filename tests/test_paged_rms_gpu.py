"""Relative RMS errors of the paged attention by request and query head (paged_ref.rms_bound), where the bound of a single
element sees little: long texts, cut over the GPU and joined."""
import math

import pytest

import paged_ref
import parity
from test_paged_gpu import attend, check, on_gpu

pytestmark = pytest.mark.gpu

BATCHES = {
    "one long": ([(70000, 1)], 4, 2, 16, 1),
    "one long, five tokens": ([(30011, 5), (20, 1)], 8, 2, 128, 5),
    "decoding": ([(8000, 1), (4097, 1), (1000, 1), (129, 1), (2500, 1), (700, 1), (6000, 1)], 8, 2, 32, 1),
    "chunk on a long text": ([(20000, 90)], 4, 1, 64, 90),
    "prompt": ([(0, 1500)], 4, 2, 32, 1500),
    "mixed": ([(9000, 1), (1500, 700), (31, 1), (0, 520)], 4, 2, 256, 700),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("name", list(BATCHES))
def test_rms_error_by_request_and_head(name, d, fp8):
    lens, Hq, Hkv, ps, most = BATCHES[name]
    c = paged_ref.case(lens, Hq, Hkv, d, ps, fp8=fp8, seed=80 + d)
    o, lse = attend(c, on_gpu(c), max_new=most)
    parity.check_status()
    check(c, o, lse)
    ro, _, _ = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], 1 / math.sqrt(d), True,
                                   c["fk"], c["fv"])
    errors = paged_ref.rms_errors(o.cpu(), ro, c["start"])
    assert len(errors) == len(lens) * Hq
    worst = max(errors, key=lambda e: e[2])
    assert worst[2] <= paged_ref.rms_bound(fp8), worst
    print(name, d, fp8, worst)
