"""Calls of the paged cache's operators that their documentation allows and that are easy to get wrong: stream handles,
steps back to back, lengths and tables at the limits of what is counted."""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import parity
from test_paged_gpu import attend, check, ints, on_gpu

pytestmark = pytest.mark.gpu


def test_stream_handles():
    """A raw handle names that very stream, 0 the default one: the work of a call stands behind what that stream holds."""
    c = paged_ref.case([(300, 1), (20, 3)], 4, 2, 64, 16, seed=40)
    g = on_gpu(c)
    want = attend(c, g, max_new=3)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for current, handle in ((side, 0), (side, torch.cuda.default_stream().cuda_stream),
                            (torch.cuda.default_stream(), side.cuda_stream)):
        with torch.cuda.stream(current), fa._on(handle, g["q"]):
            assert torch.cuda.current_stream().cuda_stream == handle
        # the queries arrive late on the handle's stream, which need not be the current one
        late = dict(g, q=torch.zeros_like(g["q"]))
        o, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        torch.cuda.synchronize()
        with torch.cuda.stream(torch.cuda.default_stream() if handle == 0 else side):
            torch.cuda._sleep(20000000)
            late["q"].copy_(g["q"])
        with torch.cuda.stream(current):
            attend(c, late, max_new=3, out=o, lse=lse, stream=handle)
        parity.check_status()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
