"""Attention in a sliding window over the paged cache, and the rotation on the way into it, on the GPU against the plain
64-bit forms. Tolerances of the attention as in test_paged_gpu.py; of the rotation as in test_rope_gpu.py, and for E4M3 keys
half a step of the code (2^-4 of the value, 2^-10 below the normal codes) for the fp32 value within 2^-17 of the pair's size.
"""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import window_ref

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def hide(c, window, sinks):
    """Pages that no token of their request sees are given away: their entries name no page of the cache, or one full of NaN."""
    nan_page = c["free"][0]
    for cache in (c["k_cache"], c["v_cache"]):
        x = cache.view(torch.uint8) if c["fp8"] else cache
        x[nan_page] = 0x7F if c["fp8"] else math.nan
    for r, (ctx, n) in enumerate(zip(c["ctx"], c["new"])):
        for i in range(len(c["table"][r])):
            first, last = i * c["ps"], (i + 1) * c["ps"] - 1
            if n and first >= sinks and last <= ctx - window and last < ctx + n:
                c["table"][r][i] = (-3, 1 << 30, nan_page)[i % 3]


def attend(c, window, sinks, scale=None, **kw):
    return fa.forward_paged(c["q"].cuda(), c["k_cache"].cuda(), c["v_cache"].cuda(), ints(c["table"]), ints(c["start"]), ints(c["lens"]),
                            scale=scale, descale_k=c["fk"], descale_v=c["fv"], window=window, sinks=sinks, **kw)


def check(c, o, lse, window, sinks, scale=None):
    scale = 1.0 / math.sqrt(c["d"]) if scale is None else scale
    ro, rl, spread = window_ref.paged(c["q"], c["k_cache"], c["v_cache"], c["table"], c["start"], c["lens"], scale, window, sinks,
                                      c["fk"], c["fv"])
    n = c["start"][-1]
    o, lse, ro, rl, spread = o[:n].double().cpu(), lse[:n].double().cpu(), ro[:n], rl[:n], spread[:n]
    fin = torch.isfinite(rl)
    assert torch.equal(fin, torch.isfinite(lse)) and not torch.isnan(lse).any()
    score = 2.0 ** -12
    err = (o - ro).abs() / (2.0 ** -8 * ro.abs() + (2.0 ** -8 + score) * spread + 1e-30)
    assert float(err.max()) <= 1.0, float(err.max())
    assert float(o[~fin].abs().sum()) == 0.0
    el = (lse[fin] - rl[fin]).abs()
    assert not el.numel() or float(el.max()) <= score + 2.0 ** -22 * float(rl[fin].abs().max()), float(el.max())
    assert window_ref.rms(o, ro) <= paged_ref.rms_bound(c["fp8"])


EDGE = [(0, 1), (1, 1), (14, 1), (15, 1), (16, 1), (30, 1), (126, 1), (127, 1), (128, 1), (300, 1), (1999, 1)]
CHUNKS = [(0, 129), (5, 127), (900, 200), (0, 3), (130, 2), (127, 1), (250, 33)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks,ps", [(1, 0, 16), (1, 1, 32), (20, 4, 16), (128, 0, 64), (129, 130, 16), (300, 4, 128),
                                             (1000, 16, 256), (5000, 0, 16), (10 ** 9, 10 ** 9, 32)])
def test_single_tokens(window, sinks, ps, d, fp8):
    c = paged_ref.case(EDGE, 8, 2, d, ps, fp8, seed=window % 97)
    hide(c, window, sinks)
    o, lse = attend(c, window, sinks, max_new=1)
    assert fa.fa_device_status(True) == fa.FA_OK
    check(c, o, lse, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks,ps,Hq,Hkv", [(1, 0, 16, 4, 2), (64, 4, 16, 6, 2), (129, 130, 32, 4, 1), (400, 1, 64, 8, 1),
                                                    (100, 300, 16, 3, 3), (3000, 0, 128, 2, 2)])
def test_chunks(window, sinks, ps, Hq, Hkv, d, fp8):
    c = paged_ref.case(CHUNKS, Hq, Hkv, d, ps, fp8, pad=3, seed=window, fused=True)
    hide(c, window, sinks)
    o, lse = attend(c, window, sinks)
    assert fa.fa_device_status(True) == fa.FA_OK
    check(c, o, lse, window, sinks)
    assert not o[c["start"][-1]:].any()


@pytest.mark.parametrize("fp8", [False, True])
def test_two_kernels(fp8):
    """Single tokens beside a chunk in a table wide enough that each kernel takes its own, cut tiles among both."""
    c = paged_ref.case([(700, 150)] + [(2500 + 13 * i, 1) for i in range(30)], 16, 8, 128, 32, fp8, seed=5, width=4000)
    hide(c, 2200, 140)
    o, lse = attend(c, 2200, 140, max_new=150)
    assert fa.fa_device_status(True) == fa.FA_OK
    check(c, o, lse, 2200, 140)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 1), (7, 7), (32, 1)])
def test_long_text_of_one(Hq, Hkv):
    c = paged_ref.case([(20000, 1)], Hq, Hkv, 128, 64, seed=Hq)
    for window, sinks in ((9000, 4), (1500, 260)):
        k = dict(c, table=[list(r) for r in c["table"]])
        hide(k, window, sinks)
        check(k, *attend(k, window, sinks, max_new=1), window, sinks)


def test_tokens_without_keys():
    c = paged_ref.case([(0, 5), (40, 3)], 4, 2, 64, 16, seed=2)
    c["lens"] = [2, 43]  # the first three tokens of the first request see no key
    check(c, *attend(c, 10, 1), 10, 1)
    c["lens"] = [0, 43]
    check(c, *attend(c, 10, 1), 10, 1)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_wide_window_is_the_causal_attention_and_repeats_are_identical():
    c = paged_ref.case(CHUNKS, 8, 2, 128, 16, seed=9)
    o, lse = attend(c, 2000, 0)
    ro, rl = fa.forward_paged(c["q"].cuda(), c["k_cache"].cuda(), c["v_cache"].cuda(), ints(c["table"]), ints(c["start"]), ints(c["lens"]))
    assert window_ref.rms(o, ro) <= paged_ref.rms_bound(False) and float((lse - rl)[lse.isfinite()].abs().max()) <= 2.0 ** -11
    again = attend(c, 2000, 0)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


def test_out_of_range_pages_in_the_window_are_reported():
    c = paged_ref.case([(300, 1)], 4, 2, 64, 16, seed=3)
    c["table"][0][17] = -1  # tokens 272 .. 287
    attend(c, 50, 0, max_new=1)
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    attend(c, 10, 0, max_new=1)
    assert fa.fa_device_status(True) == fa.FA_OK


# ---------------------------------------------------------------- rotation and store
def positions_of(c):
    return [p for a, n in zip(c["ctx"], c["new"]) for p in range(a, a + n)]


@pytest.mark.parametrize("R", [1, 3, 5000])
def test_positions(R):
    lens = [(i % 37, (0, 1, 3, 2, 0)[i % 5]) for i in range(R)]
    if R == 1:
        lens = [(7, 300)]
    start, seq = [0], []
    for a, n in lens:
        start.append(start[-1] + n)
        seq.append(a + n)
    T = start[-1] + 9
    out = fa.paged_positions(ints(start), ints(seq), T)
    assert out.tolist() == [p for a, n in lens for p in range(a, a + n)] + [-1] * 9
    held = torch.full((T,), 5, dtype=torch.int32, device="cuda")
    assert fa.paged_positions(ints(start), ints(seq), T, out=held) is held and torch.equal(held, out)


def test_positions_of_tokens_without_keys_and_odd_tables():
    assert fa.paged_positions(ints([0, 4]), ints([2]), 4).tolist() == [-1, -1, 0, 1]
    got = fa.paged_positions(ints([-5, 2, 1, 100]), ints([2, 3, 40]), 6).tolist()  # starts out of range and out of order
    assert len(got) == 6 and all(-1 <= x < 40 for x in got)


def store_case(fp8, norm, inter, d, rotary, Hq, Hkv, ps, lens, seed, w_type=torch.bfloat16):
    c = paged_ref.case(lens, Hq, Hkv, d, ps, fp8, pad=3, seed=seed, fused=True)
    g = torch.Generator().manual_seed(seed + 1)
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(w_type) if norm else None for _ in range(2)]
    freqs = fa.rope_frequencies(rotary, device="cpu") if rotary else torch.empty(0, dtype=torch.float64)
    pos = positions_of(c) + [0] * 3
    slots = [c["table"][r][p // ps] * ps + p % ps for r, (a, n) in enumerate(zip(c["ctx"], c["new"])) for p in range(a, a + n)] + [-1] * 3
    return c, w, freqs, pos, slots


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm,inter,d,rotary,Hq,Hkv,ps,lens", [
    (True, False, 128, 128, 32, 8, 16, [(5, 1), (300, 1), (15, 1)]), (False, True, 64, 16, 4, 4, 32, [(0, 130), (31, 2)]),
    (True, True, 64, 48, 5, 1, 128, [(100, 40)]), (False, False, 128, 64, 7, 7, 256, [(0, 1)]), (True, False, 64, 0, 6, 2, 64, [(9, 70), (1, 1)]),
    (False, False, 128, 128, 8, 2, 16, [(0, 700), (44, 300)])])
def test_rope_store(norm, inter, d, rotary, Hq, Hkv, ps, lens, fp8):
    c, w, freqs, pos, slots = store_case(fp8, norm, inter, d, rotary, Hq, Hkv, ps, lens, Hq + rotary, torch.float32 if inter else torch.bfloat16)
    base = torch.cat((c["q"], c["k"], c["v"]), 1).cuda()  # slices of one projection's output
    q, k, v = base.split([Hq, Hkv, Hkv], 1)
    kc, vc = c["k_cache"].cuda(), c["v_cache"].cuda()
    out = torch.full((c["T"], Hq, d), 3.0, dtype=torch.bfloat16, device="cuda")
    wq, wk = (None if x is None else x.cuda() for x in w)
    got = fa.paged_rope_store(q, k, v, ints(slots), ints(pos), freqs.cuda(), kc, vc, interleaved=inter, factor=0.9, q_weight=wq, k_weight=wk,
                              eps=1e-5, descale_k=c["fk"], descale_v=c["fv"], out=out)
    assert got is out and fa.fa_device_status(True) == fa.FA_OK
    n = c["start"][-1]
    assert (out[n:] == 3.0).all()
    p = torch.tensor(pos[:n])
    ref, size = (x.transpose(0, 1) for x in window_ref.rope(c["q"][:n].transpose(0, 1), w[0], p, freqs, inter, 0.9, 1e-5))
    assert float(((out[:n].double().cpu() - ref).abs() / (2.0 ** -8 * ref.abs() + 2.0 ** -17 * size + 1e-30)).max()) <= 1.0
    at = torch.tensor(slots[:n])
    ref, size = (x.transpose(0, 1) / c["fk"] for x in window_ref.rope(c["k"][:n].transpose(0, 1), w[1], p, freqs, inter, 0.9, 1e-5))
    have = kc.double().cpu()[at // ps, :, at % ps]
    half = 2.0 ** -4 if fp8 else 2.0 ** -8
    inside = ref.abs() < 448 if fp8 else torch.ones_like(ref, dtype=torch.bool)
    err = (have - ref).abs() / (half * ref.abs() + 2.0 ** -17 * size + (2.0 ** -10 if fp8 else 1e-30))
    assert float(err[inside].max()) <= 1.0 and (have[~inside].abs() >= 416).all()
    # values, and every other slot of both caches, as the store alone leaves them
    kc2, vc2 = c["k_cache"].cuda(), c["v_cache"].cuda()
    fa.paged_store(k, v, ints(slots), kc2, vc2, descale_k=c["fk"], descale_v=c["fv"])
    assert torch.equal(vc.view(torch.uint8), vc2.view(torch.uint8))
    rest = torch.ones((kc.shape[0], ps), dtype=torch.bool)
    rest[at // ps, at % ps] = False
    for a, b in ((kc, c["k_cache"]), (vc, c["v_cache"])):
        a, b = (x.view(torch.uint8).transpose(1, 2)[rest] for x in (a.cpu(), b))  # as bytes: NaN among them
        assert torch.equal(a, b)


def test_rope_store_in_place_and_left_out_rows():
    c, w, freqs, pos, slots = store_case(False, True, False, 64, 64, 4, 2, 16, [(3, 20)], 4)
    wq, wk = (x.cuda() for x in w)
    slots[5] = -1
    slots[7] = c["k_cache"].shape[0] * 16  # past the cache
    kc, vc = c["k_cache"].cuda(), c["v_cache"].cuda()
    args = (ints(slots), ints(pos), freqs.cuda())
    first = fa.paged_rope_store(c["q"].cuda(), c["k"].cuda(), c["v"].cuda(), *args, kc, vc, q_weight=wq, k_weight=wk)
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    assert not first[5].any() and first[7].any()
    base = torch.cat((c["q"], c["k"], c["v"]), 1).cuda()
    q, k, v = base.split([4, 2, 2], 1)
    before = base.clone()
    again = fa.paged_rope_store(q, k, v, *args, kc, vc, q_weight=wq, k_weight=wk, out=q)
    assert again is q and torch.equal(q[5], before[5, :4]) and torch.equal(base[:, 4:], before[:, 4:])
    keep = torch.arange(20, device="cuda") != 5
    assert torch.equal(q[:20][keep], first[:20][keep])
    fa.fa_device_status(True)


def test_layers_of_a_step_together_captured():
    """Plan, positions, rotation with store and attention in a window of two layers, captured in a graph and replayed with
    other lengths: what the calls one by one and the plain forms give."""
    torch.manual_seed(0)
    Hq, Hkv, d, ps, R, T, W, S = 8, 2, 128, 16, 3, 80, 40, 4
    freqs = fa.rope_frequencies(d)
    w = [(1 + 0.2 * torch.randn(d, device="cuda")).to(torch.bfloat16) for _ in range(2)]
    caches = [[torch.randn((40, Hkv, ps, d), device="cuda").to(torch.bfloat16) for _ in range(2)] for _ in range(2)]
    table = torch.full((R, 12), -1, dtype=torch.int32, device="cuda")
    free, head = torch.randperm(40, device="cuda").to(torch.int32), ints([0])
    ctx, new = ints([0, 0, 0]), ints([37, 5, 1])
    qkv = [torch.randn((T, Hq + 2 * Hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2)]

    def step():
        start, lens, slots, taken = fa.paged_plan(ctx, new, table, free, ps, T, free_head=head)
        pos = fa.paged_positions(start, lens, T)
        outs = []
        for x, (kc, vc) in zip(qkv, caches):
            q, k, v = x.split([Hq, Hkv, Hkv], 1)
            q = fa.paged_rope_store(q, k, v, slots, pos, freqs, kc, vc, q_weight=w[0], k_weight=w[1])
            outs += fa.forward_paged(q, kc, vc, table, start, lens, max_new=40, window=W, sinks=S)
        return start, lens, pos, taken, outs

    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        captured = step()
    history = [[[], [], []] for _ in range(2)]  # by layer and request: the rows of q, k, v so far
    for lens_c, lens_n in (([0, 0, 0], [37, 5, 1]), ([37, 5, 1], [1, 40, 1]), ([38, 45, 2], [1, 1, 33])):
        ctx.copy_(ints(lens_c))
        new.copy_(ints(lens_n))
        for x in qkv:
            x.copy_(torch.randn(x.shape, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_device_status(True) == fa.FA_OK
        start, lens, pos, taken, outs = captured
        at = start.tolist()
        assert pos.tolist()[:at[-1]] == [p for c, n in zip(lens_c, lens_n) for p in range(c, c + n)]
        for layer in range(2):
            o, lse = outs[2 * layer], outs[2 * layer + 1]
            for r in range(R):
                rows = qkv[layer][at[r]:at[r + 1]]
                history[layer][r].append(rows.clone())
                x = torch.cat(history[layer][r])
                p = torch.arange(x.shape[0], device="cuda")
                q, k = (window_ref.rope(y.transpose(0, 1), wy, p, freqs, False, 1.0, 1e-6)[0].to(torch.bfloat16)
                        for y, wy in ((x[:, :Hq], w[0]), (x[:, Hq:Hq + Hkv], w[1])))
                v = x[:, Hq + Hkv:].transpose(0, 1)
                ref = window_ref.batch(q[None, :, lens_c[r]:], k[None], v[None], W, S, 1 / math.sqrt(d))
                got = o[at[r]:at[r + 1]].transpose(0, 1)[None]
                # q and k once more rounded than the plain form's: half a step each moves a score by 2^-8 sum |q k| scale
                assert window_ref.rms(got, ref["o"]) <= 1e-2
        head += taken
