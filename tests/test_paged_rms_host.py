"""The relative RMS error by request and head sees what the bound of a single element cannot: on a long text o averages down
to the size of that bound."""
import math

import pytest
import torch

import paged_ref


@pytest.mark.parametrize("fp8", [False, True])
def test_rms_sees_one_lost_block_of_values(fp8):
    """One block of 128 keys without its values, of a request of 70001 keys: within the bound of every element, far
    outside the RMS bound; the same with four blocks (a part of such a tile, cut for every SM) joined with 0.8 of their
    weight. Roundings alone stay inside."""
    c = paged_ref.case([(70000, 1)], 2, 1, 128, 16, fp8=fp8, seed=3)
    args = (c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], 1 / math.sqrt(128), True, c["fk"], c["fv"])
    ro, _, spread = paged_ref.attention(*args)
    bound = paged_ref.rms_bound(fp8)
    assert max(e for _, _, e in paged_ref.rms_errors(ro.to(torch.bfloat16), ro, c["start"])) <= bound

    def error_with(block, blocks, keep):
        v = c["v_cache"].float()
        for p in c["table"][0][block * 8:(block + blocks) * 8]:
            v[p] *= keep
        o = paged_ref.attention(c["q"], c["k_cache"], v, *args[3:])[0].to(torch.bfloat16)
        element = ((o.double() - ro).abs() / (2.0 ** -8 * ro.abs() + (2.0 ** -8 + 2.0 ** -12) * spread)).max()
        return float(element), min(e for _, _, e in paged_ref.rms_errors(o, ro, c["start"]))

    for what in ((300, 1, 0.0), (301, 4, 0.8)):
        element, rms = error_with(*what)
        assert element < 1.0 and rms > 2 * bound, (what, element, rms, bound)
