"""Attention in a sliding window on the GPU, forward and backward, every element against the plain 64-bit form.

Tolerances: the bounds that window_ref.attention derives from the roundings; over whole tensors the relative RMS errors of
independent roundings spread over half a step (2^-8 / sqrt(3) = 0.00226 each): o has two of them (0.0032), dv two, dq and dk
two and those of o in D: below 0.005 with room for few rows; one key too many or too few of a window of 200
is 0.07.
"""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import window_ref

pytestmark = pytest.mark.gpu


def inputs(B, Hq, Hkv, Nq, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    shapes = ((B, Hq, Nq, d), (B, Hkv, Nk, d), (B, Hkv, Nk, d), (B, Hq, Nq, d))
    return [torch.randn(s, generator=g).to(torch.bfloat16).cuda() for s in shapes]


def ints(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def check(name, x, ref):
    r, b = ref[name], ref["bound_" + name]
    x = x.double()
    fin = r.isfinite()
    assert torch.equal(fin, x.isfinite()) and torch.equal(x[~fin], r[~fin]), name
    over = ((x - r)[fin].abs() / b[fin]).max() if fin.any() else 0.0
    assert float(over) <= 1.0, (name, float(over))
    if name != "lse":
        assert window_ref.rms(x, r) <= 5e-3, (name, window_ref.rms(x, r))


def run(B, Hq, Hkv, Nq, Nk, d, window, sinks, lens_q=None, lens_k=None, seed=0, scale=None, backward=True):
    q, k, v, dO = inputs(B, Hq, Hkv, Nq, Nk, d, seed)
    lq, lk = ints(lens_q), ints(lens_k)
    o, lse = fa.forward_window(q, k, v, window, sinks, scale, lq, lk)
    grads = fa.backward_window(q, k, v, o, lse, dO, window, sinks, scale, lq, lk) if backward else ()
    torch.cuda.synchronize()
    assert fa.fa_device_status(True) == fa.FA_OK
    ref = window_ref.batch(q, k, v, window, sinks, scale or 1.0 / math.sqrt(d), lens_q, lens_k, dO if backward else None)
    check("o", o, ref)
    check("lse", lse, ref)
    for name, x in zip(("dq", "dk", "dv"), grads):
        check(name, x, ref)
    return o, lse, grads


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,window,sinks", [
    (1, 1, 0), (1, 5, 3), (5, 1, 0), (5, 2, 1), (127, 64, 0), (128, 128, 4), (129, 128, 4), (129, 1, 0), (300, 1, 1), (300, 2, 0),
    (300, 127, 0), (300, 128, 0), (300, 129, 0), (300, 128, 130), (513, 256, 4), (513, 257, 128), (513, 100, 129), (513, 300, 513),
    (513, 513, 0), (513, 100000, 0), (513, 512, 1000000), (700, 130, 300), (900, 250, 1)])
def test_sizes(N, window, sinks, d):
    run(1, 2, 2, N, N, d, window, sinks, seed=N + window)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (2, 1), (3, 1), (6, 2), (8, 2), (5, 1)])
def test_grouped_heads(Hq, Hkv, d):
    run(2, Hq, Hkv, 300, 300, d, 140, 3, seed=Hq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,Nk,window,sinks", [
    (1, 1, 1, 0), (1, 700, 200, 4), (1, 700, 1, 0), (1, 700, 1000, 0), (2, 130, 2, 1), (100, 228, 129, 0), (128, 777, 200, 4),
    (130, 700, 64, 0), (300, 1000, 300, 150), (129, 513, 385, 0), (33, 1000, 20, 0)])
def test_last_rows_of_longer_keys(Nq, Nk, window, sinks, d):
    """Keys that no row sees (before every window) get zero gradients."""
    run(1, 4, 2, Nq, Nk, d, window, sinks, seed=Nk)


@pytest.mark.parametrize("d", [64, 128])
def test_padding(d):
    for lens_q, lens_k in (([300, 1, 128, 129], [400, 101, 400, 129]), ([2, 299, 300, 257], None), (None, [300, 399, 400, 301])):
        N, Nk = 300, 400
        ok_q = lens_q or [N] * 4
        lens_k2 = lens_k or [Nk] * 4
        o, lse, (dq, dk, dv) = run(4, 2, 1, N, Nk, d, 130, 5, lens_q, lens_k, seed=11)
        for b in range(4):
            assert not o[b, :, ok_q[b]:].any() and not dq[b, :, ok_q[b]:].any()
            assert (lse[b, :, ok_q[b]:] == -math.inf).all()
            assert not dk[b, :, lens_k2[b]:].any() and not dv[b, :, lens_k2[b]:].any()


@pytest.mark.parametrize("d", [64, 128])
def test_many_tiles(d):
    """More tiles than the persistent CTAs take in one round, the last round not full."""
    run(2, 10, 5, 2500, 2500, d, 300, 4, seed=3)
    run(1, 26, 26, 1900, 2000, d, 700, 0, seed=4)


@pytest.mark.parametrize("d", [64, 128])
def test_wide_window_is_the_causal_attention(d):
    q, k, v, dO = inputs(2, 3, 3, 500, 500, d, 5)
    o, lse = fa.forward_window(q, k, v, 500)
    ro, rl = fa.forward(q, k, v, causal=True)
    assert window_ref.rms(o, ro) <= 5e-3 and float((lse - rl).abs().max()) <= 2.0 ** -10
    for x, r in zip(fa.backward_window(q, k, v, o, lse, dO, 500), fa.backward(q, k, v, ro, rl, dO, causal=True)):
        assert window_ref.rms(x, r) <= 5e-3


def test_repeats_are_identical():
    q, k, v, dO = inputs(2, 12, 3, 1000, 1000, 128, 6)
    runs = []
    for _ in range(3):
        o, lse = fa.forward_window(q, k, v, 300, 200)
        runs.append((o, lse, *fa.backward_window(q, k, v, o, lse, dO, 300, 200)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.parametrize("d", [64, 128])
def test_hidden_keys_do_not_count(d):
    """Large scores and values where a window hides them change nothing, a sharp softmax included."""
    q, k, v, dO = inputs(1, 2, 1, 600, 600, d, 7)
    k[:, :, :100] *= 30  # seen by the first rows only
    v[:, :, :100] *= 1000
    o, lse = fa.forward_window(q, k, v, 128, 0)
    late = slice(300, 600)
    ref = window_ref.batch(q[:, :, late], k, v, 128, 0, 1 / math.sqrt(d))
    check("o", o[:, :, late], ref)
    check("lse", lse[:, :, late], ref)


def test_differences():
    """Gradients against central differences of the 64-bit form, through autograd."""
    q, k, v, dO = inputs(1, 2, 1, 150, 150, 64, 8)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o = fa.attention_window(*leaves, 40, 2)
    grads = torch.autograd.grad(o, leaves, dO)

    def loss(*x):
        return float((window_ref.batch(*x, 40, 2, 0.125)["o"] * dO.double()).sum())

    g = torch.Generator().manual_seed(1)
    for n, (x, gx) in enumerate(zip((q, k, v), grads)):
        u = torch.randn(x.shape, generator=g, dtype=torch.float64).cuda()
        h = 1e-5
        args = [[y.double() for y in (q, k, v)] for _ in range(2)]
        args[0][n], args[1][n] = args[0][n] + h * u, args[1][n] - h * u
        slope = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        ref = window_ref.batch(q, k, v, 40, 2, 0.125, dO=dO)
        bound = float((ref[("bound_dq", "bound_dk", "bound_dv")[n]] * u.abs()).sum())  # of the gradient's own roundings
        assert abs(float((gx.double() * u).sum()) - slope) <= bound + 1e-6 * abs(slope)


def test_autograd_of_expanded_and_strided_gradients():
    q, k, v, _ = inputs(2, 4, 2, 200, 200, 64, 9)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    fa.attention_window(*leaves, 50, 1).sum().backward()  # the gradient of o is one expanded number
    o, lse = fa.forward_window(q, k, v, 50, 1)
    ones = torch.ones_like(o)
    for x, r in zip(leaves, fa.backward_window(q, k, v, o, lse, ones, 50, 1)):
        assert torch.equal(x.grad, r)
    t = [x.clone().requires_grad_() for x in (q, k, v)]
    w = torch.randn((200, 2, 4, 64), device="cuda").to(torch.bfloat16)
    (fa.attention_window(*t, 50, 1).permute(2, 0, 1, 3) * w).sum().backward()  # a transposed one
    for x, r in zip(t, fa.backward_window(q, k, v, o, lse, w.permute(1, 2, 0, 3).contiguous(), 50, 1)):
        assert torch.equal(x.grad, r)


def test_captured_and_replayed():
    q, k, v, dO = inputs(2, 4, 2, 400, 400, 128, 10)
    other = inputs(2, 4, 2, 400, 400, 128, 11)
    lens = ints([400, 250])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        o, lse = fa.forward_window(q, k, v, 100, 4, seqlens_q=lens, seqlens_k=lens)  # (warm-up)
        fa.backward_window(q, k, v, o, lse, dO, 100, 4, seqlens_q=lens, seqlens_k=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        o, lse = fa.forward_window(q, k, v, 100, 4, seqlens_q=lens, seqlens_k=lens)
        grads = fa.backward_window(q, k, v, o, lse, dO, 100, 4, seqlens_q=lens, seqlens_k=lens)
    for x, y in zip((q, k, v, dO), other):
        x.copy_(y)
    lens.copy_(ints([33, 400]))
    graph.replay()
    torch.cuda.synchronize()
    ro, rl = fa.forward_window(q, k, v, 100, 4, seqlens_q=lens, seqlens_k=lens)
    assert torch.equal(o, ro) and torch.equal(lse, rl)
    for x, r in zip(grads, fa.backward_window(q, k, v, ro, rl, dO, 100, 4, seqlens_q=lens, seqlens_k=lens)):
        assert torch.equal(x, r)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_other_streams():
    """Two calls at once on streams of their own, a handle among them, with the current stream busy elsewhere."""
    a, b = inputs(1, 4, 2, 700, 700, 128, 12), inputs(1, 4, 2, 700, 700, 128, 13)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, l1 = fa.forward_window(*a[:3], 200, 4, stream=s1)
    o2, l2 = fa.forward_window(*b[:3], 200, 4, stream=int(s2.cuda_stream))
    g1 = fa.backward_window(*a[:3], o1, l1, a[3], 200, 4, stream=s1)
    g2 = fa.backward_window(*b[:3], o2, l2, b[3], 200, 4, stream=int(s2.cuda_stream))
    torch.cuda.synchronize()
    for x, o, l, g in ((a, o1, l1, g1), (b, o2, l2, g2)):
        ro, rl = fa.forward_window(*x[:3], 200, 4)
        assert torch.equal(o, ro) and torch.equal(l, rl)
        assert all(torch.equal(p, r) for p, r in zip(g, fa.backward_window(*x[:3], ro, rl, x[3], 200, 4)))


def test_lengths_out_of_range_are_clamped_and_reported():
    q, k, v, _ = inputs(3, 2, 1, 200, 300, 64, 14)
    lens_q, lens_k = ints([500, 0, 150]), ints([300, 20, 100])
    o, lse = fa.forward_window(q, k, v, 64, 2, seqlens_q=lens_q, seqlens_k=lens_k)
    assert fa.fa_device_status(True) == fa.FA_ERR_INVALID_ARG
    ref = window_ref.batch(q, k, v, 64, 2, 0.125, [200, 1, 100], [300, 20, 100])
    check("o", o, ref)
    check("lse", lse, ref)


def test_a_wait_that_runs_out_is_reported():
    q, k, v, _ = inputs(1, 2, 1, 200, 200, 128, 15)
    assert fa.fa_test_arm_fault(1) == fa.FA_OK
    fa.forward_window(q, k, v, 64)
    assert fa.fa_device_status(True) == fa.FA_ERR_TIMEOUT
    run(1, 2, 1, 200, 200, 128, 64, 0)
