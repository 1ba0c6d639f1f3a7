"""Rotation, norms and attention in a window as they are used together, at drawn sizes, and what their helpers refuse.

Tolerance of a layer's results, relative RMS: the path from the projection to a gradient of it passes at most eight roundings
to bf16 (rotated q and k, P, o, dS, dq or dk, the rotated-back gradient, and the key or query in the last product), each spread
over half a step, 2^-8 / sqrt(3) = 0.00226; independent ones add up to 0.0064, here 0.01. A row turned by one position too many
or a window one key too wide is above 0.05.
"""
import math
import random

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import paged_ref
import test_window_gpu
import test_window_paged_gpu
import window_ref

pytestmark = pytest.mark.gpu


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(12))
def test_windows_drawn(seed, d):
    r = random.Random(100 * d + seed)
    Hkv = r.choice([1, 1, 2, 3])
    Nk = r.choice([r.randint(1, 130), r.randint(100, 700), r.randint(500, 1300)])
    Nq = Nk if r.random() < 0.5 else r.randint(1, Nk)
    B = r.randint(1, 3)
    lens_q = lens_k = None
    if r.random() < 0.5:
        lens_k = [r.randint(1, Nk) for _ in range(B)]
        lens_q = [r.randint(1, min(Nq, n)) for n in lens_k]
    window, sinks = r.randint(1, Nk + 50), r.choice([0, 0, r.randint(1, 40), r.randint(1, Nk)])
    test_window_gpu.run(B, Hkv * r.choice([1, 2, 3, 4, 7]), Hkv, Nq, Nk, d, window, sinks, lens_q, lens_k, seed=seed)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("seed", range(8))
def test_paged_windows_drawn(seed, d, fp8):
    r = random.Random(1000 * d + 10 * seed + fp8)
    Hkv = r.choice([1, 2, 3])
    single = r.random() < 0.4
    reqs = [(r.choice([0, r.randint(0, 200), r.randint(0, 1500)]), 1 if single or r.random() < 0.4 else r.randint(0, 150))
            for _ in range(r.randint(1, 9))]
    if not any(n for _, n in reqs):
        reqs.append((9, 1))
    c = paged_ref.case(reqs, Hkv * r.choice([1, 2, 4, 5]), Hkv, d, r.choice([16, 32, 64, 128, 256]), fp8, seed=seed)
    window, sinks = r.choice([1, r.randint(1, 64), r.randint(1, 900)]), r.choice([0, r.randint(1, 20), r.randint(1, 300)])
    test_window_paged_gpu.hide(c, window, sinks)
    o, lse = test_window_paged_gpu.attend(c, window, sinks, max_new=max(n for _, n in reqs))
    assert fa.fa_device_status(True) == fa.FA_OK
    test_window_paged_gpu.check(c, o, lse, window, sinks)


def layer(qkv, Hq, Hk, freqs, pos, wq, wk, window, sinks):
    """A fused projection's [B, N, Hq + 2 Hk, d] to the attention's result, by the library."""
    q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hk, Hk], 2))
    q, k = fa.rope(q, k, freqs, pos, q_weight=wq, k_weight=wk)
    return fa.attention_window(q, k, v.contiguous(), window, sinks)


def plain_layer(qkv, Hq, Hk, freqs, pos, wq, wk, window, sinks):
    q, k, v = (x.transpose(1, 2) for x in qkv.split([Hq, Hk, Hk], 2))
    q, k = (window_ref.rope(x, w, pos[:, None], freqs, False, 1.0, 1e-6)[0] for x, w in ((q, wq), (k, wk)))
    k, v = (x.repeat_interleave(Hq // Hk, 1) for x in (k, v))
    N, i = q.shape[2], torch.arange(q.shape[2], device="cuda")
    s = (q @ k.mT / math.sqrt(q.shape[-1])).masked_fill(~window_ref.sees(i[:, None], i[None], window, sinks), -math.inf)
    return torch.softmax(s, -1) @ v


@pytest.mark.parametrize("d,Hq,Hk,N,rotary,window,sinks", [(64, 4, 2, 333, 64, 100, 3), (128, 6, 2, 260, 32, 129, 0), (128, 2, 2, 1, 128, 1, 0)])
def test_a_layer_and_its_gradients(d, Hq, Hk, N, rotary, window, sinks):
    B = 2
    qkv, dO = randn((B, N, Hq + 2 * Hk, d), 1), randn((B, Hq, N, d), 2)
    wq, wk = (1 + 0.2 * torch.randn(d, generator=torch.Generator().manual_seed(s)).cuda() for s in (3, 4))
    freqs = fa.rope_frequencies(rotary)
    pos = torch.stack((torch.arange(N), 70000 + torch.arange(N))).int().cuda()
    results = []
    for f, kind in ((layer, lambda x: x), (plain_layer, lambda x: x.double())):
        leaves = [kind(x).detach().clone().requires_grad_() for x in (qkv, wq, wk)]
        o = f(leaves[0], Hq, Hk, freqs, pos, leaves[1], leaves[2], window, sinks)
        results.append((o.detach(), *torch.autograd.grad(o, leaves, dO.to(o.dtype))))
    assert fa.fa_device_status(True) == fa.FA_OK
    for x, ref in zip(*results):
        assert x.shape == ref.shape and window_ref.rms(x, ref) <= 1e-2


def test_a_layer_captured_with_its_backward():
    """Replays with new inputs give what the eager calls give."""
    d, Hq, Hk, N = 64, 4, 2, 200
    freqs, pos = fa.rope_frequencies(d), torch.arange(N, dtype=torch.int32, device="cuda").repeat(2, 1)
    leaves = [x.requires_grad_() for x in (randn((2, N, Hq + 2 * Hk, d), 1), 1 + 0.1 * randn((d,), 2), 1 + 0.1 * randn((d,), 3))]
    dO = randn((2, Hq, N, d), 4)

    def step():
        o = layer(leaves[0], Hq, Hk, freqs, pos, leaves[1], leaves[2], 60, 2)
        return o, torch.autograd.grad(o, leaves, dO)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o, grads = step()
    with torch.no_grad():
        leaves[0].copy_(randn(tuple(leaves[0].shape), 5))
        leaves[2].mul_(1.5)
        dO.copy_(randn(tuple(dO.shape), 6))
    graph.replay()
    torch.cuda.synchronize()
    ro, rg = step()
    assert torch.equal(o, ro) and all(torch.equal(a, b) for a, b in zip(grads, rg))
    assert fa.fa_device_status(True) == fa.FA_OK


@pytest.mark.parametrize("norm", [False, True])
def test_broadcast_inputs(norm):
    """One key row for all heads and one query row for all tokens, by strides of 0: the results of the copies, and gradients
    that are sums over them."""
    B, Hq, Hk, N, d = 2, 3, 4, 50, 64
    freqs = fa.rope_frequencies(d)
    w = 1 + 0.2 * randn((d,), 7) if norm else None
    q0, k0 = randn((B, Hq, 1, d), 1).requires_grad_(), randn((B, 1, N, d), 2).requires_grad_()
    q, k = q0.expand(B, Hq, N, d), k0.expand(B, Hk, N, d)
    y = fa.rope(q, k, freqs, q_weight=w, k_weight=w)
    c = fa.forward_rope(q.detach().contiguous(), k.detach().contiguous(), freqs, q_weight=w, k_weight=w)
    assert all(torch.equal(a, b) for a, b in zip(y, c))
    g = randn((B, Hq, N, d), 3), randn((B, Hk, N, d), 4)
    got = torch.autograd.grad(y, (q0, k0), g)
    full = fa.backward_rope(*g, freqs, q=q.detach().contiguous(), k=k.detach().contiguous(), q_weight=w, k_weight=w)
    assert torch.equal(got[0], full[0].sum(2, keepdim=True)) and torch.equal(got[1], full[1].sum(1, keepdim=True))


def test_only_some_gradients_and_unused_results():
    q, k = randn((1, 2, 9, 64), 1), randn((1, 1, 9, 64), 2)
    freqs, w = fa.rope_frequencies(32), (1 + 0.2 * randn((64,), 3)).requires_grad_()
    y, _ = fa.rope(q, k, freqs, q_weight=w, k_weight=w.detach())  # the weight alone, of one result
    g = randn((1, 2, 9, 64), 4)
    dw, = torch.autograd.grad(y, w, g)
    ref = fa.backward_rope(g, torch.zeros_like(k), freqs, q=q, k=k, q_weight=w.detach(), k_weight=w.detach())[2]
    assert torch.equal(dw, ref.to(torch.bfloat16))
    alone, none = fa.rope(q.requires_grad_(), None, freqs)
    assert none is None
    alone.sum().backward()
    assert torch.equal(q.grad, fa.backward_rope(torch.ones_like(q), None, freqs)[0])


def test_rows_far_apart():
    """A row past 2^32 bytes from its neighbour."""
    big = torch.empty((2, (1 << 31) + 64), dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((2, 2, 5, 64), (big.stride(0), 64 * 5, 64, 1))
    src = randn((2, 2, 5, 64), 1)
    x.copy_(src)
    freqs = fa.rope_frequencies(64)
    ref, _ = fa.forward_rope(src, None, freqs)
    assert torch.equal(fa.forward_rope(x, None, freqs)[0], ref)
    fa.forward_rope(x, None, freqs, out=(x,))
    assert torch.equal(x, ref)


def test_helpers_refuse():
    q, k = randn((2, 4, 10, 64), 1), randn((2, 2, 10, 64), 2)
    freqs, w = fa.rope_frequencies(64), randn((64,), 3)
    o, lse = fa.forward_window(q, k, k, 4)
    cache, packed, three = randn((4, 2, 16, 64), 4), randn((3, 4, 64), 5), ints([0, 1, 2])
    table, start, lens = ints([[0, 1]]), ints([0, 3]), ints([20])
    paged = (packed, cache, cache, table, start, lens)
    kv = packed[:, :2]
    for call in (
            lambda: fa.forward_rope(q.half(), k, freqs), lambda: fa.forward_rope(q, k[:, :, :9], freqs), lambda: fa.forward_rope(q[0], k, freqs),
            lambda: fa.forward_rope(q, k, freqs.float()), lambda: fa.forward_rope(q, k, freqs.cpu()), lambda: fa.forward_rope(q, k, freqs[None]),
            lambda: fa.forward_rope(q, k.cpu(), freqs), lambda: fa.forward_rope(q.transpose(2, 3), k.transpose(2, 3), freqs),
            lambda: fa.forward_rope(q, k, freqs, ints([0] * 9)), lambda: fa.forward_rope(q, k, freqs, torch.arange(10, device="cuda")),
            lambda: fa.forward_rope(q, k, freqs, ints([[0] * 10] * 3)), lambda: fa.forward_rope(q, k, freqs, k_weight=w),
            lambda: fa.forward_rope(q, k, freqs, q_weight=w[:32], k_weight=w), lambda: fa.forward_rope(q, k, freqs, q_weight=w, k_weight=w.float()),
            lambda: fa.forward_rope(q, k, freqs, out=(q,)), lambda: fa.forward_rope(q, k, freqs, out=(k, q)),
            lambda: fa.backward_rope(q, k, freqs, q_weight=w, k_weight=w), lambda: fa.backward_rope(q, k, freqs, q=k, k=k, q_weight=w, k_weight=w),
            lambda: fa.forward_window(q.half(), k, k, 4), lambda: fa.forward_window(q, k, k[:, :1], 4), lambda: fa.forward_window(q, k[:1], k[:1], 4),
            lambda: fa.forward_window(q.transpose(1, 2), k, k, 4), lambda: fa.forward_window(q, k.cpu(), k, 4),
            lambda: fa.forward_window(q, k, k, 1 << 31), lambda: fa.forward_window(q, k, k, 4, seqlens_k=ints([3])),
            lambda: fa.backward_window(q, k, k, o, lse[:1], q, 4), lambda: fa.backward_window(q, k, k, o, lse, q.float(), 4),
            lambda: fa.backward_window(q, k, k, o, lse, q, 4, workspace=torch.empty(1 << 20, dtype=torch.uint8)),
            lambda: fa.forward_paged(*paged, causal=False, window=4), lambda: fa.forward_paged(*paged, sinks=4),
            lambda: fa.paged_positions(start.cpu(), lens, 3), lambda: fa.paged_positions(start, lens, -1),
            lambda: fa.paged_positions(start, lens, 3, out=ints([0, 0])),
            lambda: fa.paged_rope_store(packed, kv, kv, three, three[:2], freqs, cache, cache),
            lambda: fa.paged_rope_store(packed, packed, packed, three, three, freqs, cache, cache),
            lambda: fa.paged_rope_store(packed, kv, kv, three, three, freqs, cache, cache, out=kv)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: fa.forward_window(q, k, k, 0), lambda: fa.forward_window(q, k, k, 4, -1), lambda: fa.forward_window(k, q, q, 4),
                 lambda: fa.forward_window(q, k[:, :, :9].contiguous(), k[:, :, :9].contiguous(), 4), lambda: fa.forward_paged(*paged, window=0),
                 lambda: fa.backward_window(q, k, k, o, lse, q, 4, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
                 lambda: fa.forward_rope(q, k, freqs[:20]), lambda: fa.forward_rope(q, k, freqs, q_weight=w),
                 lambda: fa.forward_rope(q, k, freqs, factor=math.nan), lambda: fa.forward_rope(q[:, :, :0], k[:, :, :0], freqs),
                 lambda: fa.forward_rope(q, k, freqs, out=(q, k[:, :1].expand(2, 2, 10, 64)))):
        with pytest.raises(fa.FAError):
            call()
    assert fa.fa_device_status(True) == fa.FA_OK
