"""Windowed attention with many more items of one or a few key blocks than CTAs run at once, on the GPU: every element of every
head against the plain 64-bit form, and repeated calls.

The shorter the items, the nearer a CTA's next output follows the store of the one before; heads are random and independent,
so rows stored for another head, or written over before they were stored, are off by their whole size. Tolerances as in
test_window_gpu.py.
"""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import window_ref
from test_window_gpu import check, inputs, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,Hq,Hkv,N,window,sinks,lens", [
    (4, 400, 200, 128, 128, 0, None),                   # two heads of one block: both tiles in every item
    (3, 501, 167, 128, 50, 4, None),                    # three heads: items of two tiles and of one in turn
    (2, 800, 400, 1, 1, 0, None),
    (2, 700, 700, 200, 60, 0, None),                    # no groups: a tile of one block and one of two
    (5, 240, 80, 97, 97, 0, [97, 1, 50, 96, 2]),
    (6, 130, 130, 256, 300, 2, [256, 128, 1, 129, 200, 30]),  # no rows in the second tile of the short ones
    (4, 420, 60, 30, 10, 1, [1, 30, 17, 2]),            # seven heads
])
def test_many_short_items(B, Hq, Hkv, N, window, sinks, lens, d):
    q, k, v, _ = inputs(B, Hq, Hkv, N, N, d, N + Hq)
    ls = ints(lens)
    runs = [fa.forward_window(q, k, v, window, sinks, seqlens_q=ls, seqlens_k=ls) for _ in range(10)]
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_OK
    ref = window_ref.batch(q, k, v, window, sinks, 1.0 / math.sqrt(d), lens, lens)
    check("o", runs[0][0], ref)
    check("lse", runs[0][1], ref)
    for o, lse in runs[1:]:
        assert torch.equal(o, runs[0][0]) and torch.equal(lse, runs[0][1])


@pytest.mark.parametrize("d", [64, 128])
def test_short_items_beside_copies(d):
    """The same with the memory kept busy by copies on another stream, which delay the stores of the outputs."""
    q, k, v, _ = inputs(4, 402, 134, 128, 128, d, 5)
    alone = fa.forward_window(q, k, v, 70, 2)
    a, b = (torch.empty(1 << 28, dtype=torch.uint8, device="cuda") for _ in range(2))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    runs = []
    with torch.cuda.stream(other):
        for _ in range(40):
            b.copy_(a)
    for _ in range(20):
        runs.append(fa.forward_window(q, k, v, 70, 2))
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_OK
    for o, lse in runs:
        assert torch.equal(o, alone[0]) and torch.equal(lse, alone[1])
