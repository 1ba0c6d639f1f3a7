"""A seeded sweep of random serving steps through plan, store and attention against the plain 64-bit forms: heads, types,
page sizes, lengths from none to thousands of tokens, lengths shorter than the new tokens, hints, padding, wide tables."""
import math
import random

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import parity
from test_paged_gpu import attend, check, f32, ints, on_gpu

pytestmark = pytest.mark.gpu


def draw(seed):
    rng = random.Random(seed)
    Hkv, G = rng.choice([1, 2, 3, 8]), rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 33])
    R = rng.choice([1, 1, 2, 5, 17, 90])
    most = rng.choice([1, 1, 2, 6, 40, 300])
    ctx = rng.choice([0, 20, 300, 3000 if R < 20 else 500])
    lens = [(rng.randint(0, ctx), rng.choice([1, 1, most, rng.randint(0, most)])) for _ in range(R)]
    return dict(lens=lens, Hq=Hkv * G, Hkv=Hkv, d=rng.choice([64, 128]), ps=rng.choice([16, 32, 64, 128, 256]), fp8=rng.random() < 0.5,
                pad=rng.choice([0, 0, 1, 50]), seed=seed, fused=rng.random() < 0.5,
                width=rng.choice([0, 0, 9, 4096 if R < 20 else 300])), rng


@pytest.mark.parametrize("seed", range(40))
def test_random_step(seed):
    kw, rng = draw(seed)
    c = paged_ref.case(**kw)
    g = on_gpu(c)
    n, ps = c["start"][-1], c["ps"]
    # plan: the tables as they were before the step, the free pages those that the case's tables go on with
    held = [[p if i < -(-a // ps) else -1 for i, p in enumerate(row)] for row, a in zip(c["table"], c["ctx"])]
    fresh = [p for row, a, b in zip(c["table"], c["ctx"], c["lens"]) for p in row[-(-a // ps):-(-b // ps)]]
    tab = ints(held)
    start, lens, slots, taken = fa.paged_plan(ints(c["ctx"]), ints(c["new"]), tab, ints(fresh + [0]), ps, c["T"])
    parity.check_status()
    want = paged_ref.plan(c["ctx"], c["new"], held, fresh, 0, ps, c["T"])
    assert (start.tolist(), lens.tolist(), slots.tolist(), int(taken), tab.tolist()) == want
    # store: the new rows over what the cache holds there
    fa.paged_store(g["k"], g["v"], slots, g["k_cache"], g["v_cache"], c["fk"], c["fv"])
    parity.check_status()
    at = torch.tensor(want[2][:n], dtype=torch.long)
    for name, x, f in (("k_cache", c["k"], c["fk"]), ("v_cache", c["v"], c["fv"])):
        rows = x[:n]
        if c["fp8"]:
            rows = paged_ref.e4m3(rows.double() / f32(f)).float().to(torch.float8_e4m3fn)
            c[name].view(torch.uint8)[at // ps, :, at % ps] = rows.view(torch.uint8)
        else:
            c[name][at // ps, :, at % ps] = rows
        assert torch.equal(g[name].cpu().view(torch.uint8), c[name].view(torch.uint8))
    # attention, also with lengths cut short
    cut = [max(0, a - rng.choice([0, 0, 0, 1, 30, b + 5])) for a, b in zip(c["lens"], c["new"])]
    for keys in (c["lens"], cut):
        g["lens"] = ints(keys)
        hint = rng.choice([1, max(c["new"] + [1]), 77, None])
        causal = rng.random() < 0.7
        o, lse = attend(c, g, causal=causal, max_new=hint)
        parity.check_status()
        check(c, o, lse, causal=causal, lens=keys)
        ro, rl, _ = paged_ref.attention(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], keys, 1 / math.sqrt(c["d"]),
                                        causal, c["fk"], c["fv"])
        # the bound is for many independent roundings: all requests' rows of a head together
        seen = torch.isfinite(rl[:n]).any(-1)
        if int(seen.sum()) * c["d"] >= 1024:
            for _, h, e in paged_ref.rms_errors(o[:n].cpu()[seen], ro[:n][seen], [0, int(seen.sum())]):
                assert e <= paged_ref.rms_bound(c["fp8"]), (h, e)
