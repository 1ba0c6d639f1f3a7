"""Calls from threads that have used the GPU for nothing yet."""
import threading

import pytest
import torch

from exact_io_aware_32_gb300 import fa

pytestmark = pytest.mark.gpu


def in_a_thread(call):
    got = []
    t = threading.Thread(target=lambda: got.append(call()))
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("d", [64, 128])
def test_first_call_of_a_thread(d):
    """Every buffer is there already, so the library's call is the thread's first of all."""
    q, k, v = (torch.randn((1, 2, 211, d), device="cuda").to(torch.bfloat16) for _ in range(3))
    stream = int(torch.cuda.current_stream().cuda_stream)
    results = []
    for call in (lambda o, lse: fa.fa_fwd(q, k, v, o, lse, 1, 2, 211, d, 0.1, True, stream),
                 lambda o, lse: fa.fa_fwd_window(q, k, v, o, lse, 1, 2, 2, 211, 211, d, 0.1, 300, 0, None, None, stream)):
        o, lse = torch.zeros_like(q), torch.zeros((1, 2, 211), device="cuda")  # (new addresses: no tensor map is known yet)
        torch.cuda.synchronize()
        assert in_a_thread(lambda: call(o, lse)) == fa.FA_OK
        torch.cuda.synchronize()
        results.append((o, lse))
    assert fa.fa_device_status(True) == fa.FA_OK
    ro, rl = fa.forward(q, k, v, causal=True, scale=0.1)
    for o, lse in results:
        assert float((o.float() - ro.float()).abs().max()) <= 2.0 ** -6 * float(ro.abs().max()) and float((lse - rl).abs().max()) <= 1e-3
