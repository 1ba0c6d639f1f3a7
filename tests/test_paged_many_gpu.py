"""Decoding batches of many short requests: many tiles a CTA, whose last blocks end the run in every place of the rings."""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import window_ref

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("window", [None, 90])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("R,most", [(256, 100), (200, 600), (97, 1000)])
def test_many_short_requests(R, most, d, fp8, window):
    """The kernels' waits are bounded by a second: one for a copy that is long there would show in the time of a call."""
    g = torch.Generator().manual_seed(R + d)
    c = paged_ref.case([(int(x), 1) for x in torch.randint(0, most, (R,), generator=g)], 8, 4, d, 16, fp8, seed=R)
    args = [c["q"].cuda(), c["k_cache"].cuda(), c["v_cache"].cuda(), ints(c["table"]), ints(c["start"]), ints(c["lens"])]
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for _ in range(3):
        begin.record()
        o, lse = fa.forward_paged(*args, max_new=1, descale_k=c["fk"], descale_v=c["fv"], window=window)
        end.record()
        end.synchronize()
        assert begin.elapsed_time(end) < 500
        assert fa.fa_device_status(True) == fa.FA_OK
    some = torch.arange(0, R, 7)  # every seventh request against the plain form
    w = window or 10 ** 9
    ro, rl, _ = window_ref.paged(c["q"][some], c["k_cache"], c["v_cache"], [c["table"][i] for i in some], list(range(len(some) + 1)),
                                 [c["lens"][i] for i in some], 1 / math.sqrt(d), w, 0, c["fk"], c["fv"])
    assert window_ref.rms(o.cpu()[some], ro) <= paged_ref.rms_bound(fp8)
    assert float((lse.cpu()[some].double() - rl).abs().max()) <= 2.0 ** -12 + 2.0 ** -22 * float(rl.abs().max())
