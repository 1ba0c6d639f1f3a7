"""Rotation by position and the norms of heads on the GPU against the plain 64-bit forms.

Tolerances, element by element. Forward: one rounding to bf16 (2^-8 of the value) after fp32 work: an angle to 2^-24 of a
turn (2 pi 2^-24 < 2^-21) and cosine and sine to a few last places, so a pair's elements are off by less than 2^-19 of the
pair's size; the norm's sum of d squares, square root and products by less than 2^-18 relatively (d + 8 roundings of 2^-24).
Backward without norms the same. With norms dx = r (u - xh mean(u xh)): the fp32 work is off by less than 2^-16 of r (|u| + |xh|
mean |u xh|). dw is an fp32 sum over all rows: off by less than (rows added in sequence) 2^-24 of the sum of magnitudes,
below 2^-14 of it here, and far less in relative RMS (2^-18 with errors in no order).
"""
import math

import pytest
import torch

from exact_io_aware_32_gb300 import fa
import window_ref

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


def randn(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16).cuda()


def make(B, Hq, Hk, N, d, seed, fused=True):
    if fused:  # slices of one projection's output
        x = randn((B, N, Hq + 2 * Hk, d), seed)
        return x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hk].transpose(1, 2)
    return randn((B, Hq, N, d), seed), randn((B, Hk, N, d), seed + 1)


def weights(d, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype).cuda() for _ in range(2)]


def check(y, ref, size):
    assert y.isfinite().all()
    over = ((y.double() - ref).abs() / (HALF * ref.abs() + 2.0 ** -17 * size + 1e-30)).max()
    assert float(over) <= 1.0, float(over)


def check_dx(dx, dy, x, w, pos, freqs, inter, factor, eps):
    ref, dw = window_ref.rope_backward(dy, x, w, pos, freqs, inter, factor, eps)
    if w is None:
        size = window_ref.rope(dy, None, pos, freqs, inter, factor, eps)[1]
    else:
        x = x.double()
        r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
        u = window_ref.rope(dy, None, pos, freqs, inter, factor, eps)[1] * w.double().abs()
        xh = (x * r).abs()
        size = 2 * r * (u + xh * (u * xh).mean(-1, keepdim=True))
    over = ((dx.double() - ref).abs() / (HALF * ref.abs() + 2.0 ** -17 * size + 1e-30)).max()
    assert float(over) <= 1.0, float(over)
    return dw


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("d,rotary,Hq,Hk,N,fused", [
    (64, 64, 12, 12, 1, True), (64, 16, 1, 1, 7, False), (64, 48, 5, 1, 33, True), (128, 128, 32, 8, 1, True),
    (128, 128, 8, 2, 130, True), (128, 64, 7, 7, 19, False), (128, 112, 3, 1, 65, True), (128, 16, 40, 4, 5, False),
    (64, 0, 6, 2, 9, True), (128, 0, 4, 4, 3, False)])
def test_forward_and_backward(d, rotary, Hq, Hk, N, fused, norm, inter):
    B, eps, factor = 2, 1e-5, 1.25
    q, k = make(B, Hq, Hk, N, d, N + Hq, fused)
    freqs = fa.rope_frequencies(rotary) if rotary else torch.empty(0, dtype=torch.float64, device="cuda")
    pos = (torch.arange(N, dtype=torch.int32) * 3 + torch.tensor([[5], [70000]], dtype=torch.int32)).cuda()
    wq, wk = weights(d, 3) if norm else (None, None)
    kw = dict(interleaved=inter, factor=factor, q_weight=wq, k_weight=wk, eps=eps)
    yq, yk = fa.forward_rope(q, k, freqs, pos, **kw)
    assert yq.is_contiguous() and yk.is_contiguous()
    gq, gk = randn((B, Hq, N, d), 8), randn((B, Hk, N, d), 9)
    dq, dk, dwq, dwk = fa.backward_rope(gq, gk, freqs, pos, q=q, k=k, **kw)
    p = pos[:, None]
    for x, w, y, g, dx, dw in ((q, wq, yq, gq, dq, dwq), (k, wk, yk, gk, dk, dwk)):
        check(y, *window_ref.rope(x, w, p, freqs, inter, factor, eps))
        ref = check_dx(dx, g, x, w, p, freqs, inter, factor, eps)
        assert (dw is None) == (ref is None)
        if dw is not None:
            assert dw.dtype == torch.float32 and window_ref.rms(dw, ref) <= 2.0 ** -18


@pytest.mark.parametrize("norm", [False, True])
def test_many_tokens(norm):
    """More tokens than warps that run at once; the sums over all rows."""
    q, k = make(3, 8, 2, 3001, 128, 1)
    freqs = fa.rope_frequencies(128, linear=4.0)
    wq, wk = weights(128, 2, torch.float32) if norm else (None, None)
    kw = dict(q_weight=wq, k_weight=wk)
    y = fa.forward_rope(q, k, freqs, **kw)
    g = randn((3, 8, 3001, 128), 4), randn((3, 2, 3001, 128), 5)
    dq, dk, dwq, dwk = fa.backward_rope(*g, freqs, q=q, k=k, **kw)
    pos = torch.arange(3001, device="cuda")
    for x, w, yx, gx, dx, dw in ((q, wq, y[0], g[0], dq, dwq), (k, wk, y[1], g[1], dk, dwk)):
        check(yx, *window_ref.rope(x, w, pos, freqs, False, 1.0, 1e-6))
        ref = check_dx(dx, gx, x, w, pos, freqs, False, 1.0, 1e-6)
        if norm:
            assert window_ref.rms(dw, ref) <= 2.0 ** -18
    again = fa.backward_rope(*g, freqs, q=q, k=k, **kw)
    assert all(a is b or torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))


@pytest.mark.parametrize("start", [0, 1 << 20, (1 << 31) - 9, -5])
def test_far_positions(start):
    """Angles keep 2^-24 of a turn wherever a text stands. (The 64-bit form itself loses 2^-53 of an angle of 2^31: 2^-22.)"""
    q, k = make(1, 2, 1, 8, 64, 6)
    freqs = fa.rope_frequencies(64)
    pos = torch.arange(start, start + 8, dtype=torch.int64).to(torch.int32).cuda()
    y, _ = fa.forward_rope(q, k, freqs, pos)
    check(y, *window_ref.rope(q, None, pos, freqs, False, 1.0, 1e-6))


def test_rotation_keeps_products_of_pairs():
    """q.k after the rotation depends on the distance alone, and positions 0 change nothing."""
    q, k = make(1, 1, 1, 1, 128, 7, fused=False)
    freqs = fa.rope_frequencies(128)
    zero = fa.forward_rope(q, k, freqs, torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(zero[0], q) and torch.equal(zero[1], k)


def test_in_place_and_given_outputs():
    q, k = make(2, 4, 2, 50, 64, 8)
    freqs = fa.rope_frequencies(32)
    yq, yk = fa.forward_rope(q, k, freqs)
    outs = torch.full((2, 4, 50, 64), 7.0, device="cuda", dtype=torch.bfloat16), torch.empty((2, 2, 50, 64), device="cuda", dtype=torch.bfloat16)
    a, b = fa.forward_rope(q, k, freqs, out=outs)
    assert a.data_ptr() == outs[0].data_ptr() and torch.equal(outs[0], yq) and torch.equal(outs[1], yk)
    base = q._base.clone()
    v_before = base[:, :, 6:].clone()
    sq, sk = base[:, :, :4].transpose(1, 2), base[:, :, 4:6].transpose(1, 2)
    fa.forward_rope(sq, sk, freqs, out=(sq, sk))
    assert torch.equal(sq, yq) and torch.equal(sk, yk) and torch.equal(base[:, :, 6:], v_before)


def test_queries_alone():
    q, _ = make(2, 3, 1, 20, 64, 9)
    freqs = fa.rope_frequencies(64)
    (w, _) = weights(64, 4)
    y, none = fa.forward_rope(q, None, freqs, q_weight=w)
    assert none is None
    check(y, *window_ref.rope(q, w, torch.arange(20, device="cuda"), freqs, False, 1.0, 1e-6))
    g = randn((2, 3, 20, 64), 3)
    dq, dk, dwq, dwk = fa.backward_rope(g, None, freqs, q=q, q_weight=w)
    assert dk is None and dwk is None
    ref = check_dx(dq, g, q, w, torch.arange(20, device="cuda"), freqs, False, 1.0, 1e-6)
    assert window_ref.rms(dwq, ref) <= 2.0 ** -18


def test_differences():
    """Gradients against central differences of the 64-bit form, through autograd, of inputs and weights."""
    q, k = make(1, 2, 1, 9, 64, 10)
    freqs = fa.rope_frequencies(32)
    wq, wk = weights(64, 5)
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, wq, wk)]
    y = fa.rope(leaves[0], leaves[1], freqs, q_weight=leaves[2], k_weight=leaves[3], factor=1.1)
    g = [randn(tuple(x.shape), 20 + i) for i, x in enumerate(y)]
    grads = torch.autograd.grad(y, leaves, g)
    pos = torch.arange(9, device="cuda")

    def loss(q, k, wq, wk):
        return sum(float((window_ref.rope(x, w, pos, freqs, False, 1.1, 1e-6)[0] * gx.double()).sum()) for x, w, gx in ((q, wq, g[0]), (k, wk, g[1])))

    base = [x.detach().double() for x in leaves]
    gen = torch.Generator().manual_seed(2)
    for n, gx in enumerate(grads):
        assert gx.dtype == torch.bfloat16 and gx.shape == leaves[n].shape
        u = torch.randn(base[n].shape, generator=gen, dtype=torch.float64).cuda()
        h = 1e-5
        up, down = list(base), list(base)
        up[n], down[n] = base[n] + h * u, base[n] - h * u
        slope = (loss(*up) - loss(*down)) / (2 * h)
        assert abs(float((gx.double() * u).sum()) - slope) <= float((HALF * 1.01 * gx.double().abs() * u.abs()).sum()) + 1e-5


def test_autograd_of_expanded_gradients():
    q, k = make(1, 2, 2, 30, 64, 11)
    q, k = q.detach().requires_grad_(), k.detach().requires_grad_()
    freqs = fa.rope_frequencies(64)
    yq, yk = fa.rope(q, k, freqs)
    (yq.sum() + yk.sum()).backward()
    ones = torch.ones_like(yq)
    dq, dk, _, _ = fa.backward_rope(ones, ones, freqs)
    assert torch.equal(q.grad, dq) and torch.equal(k.grad, dk)


def test_captured_and_on_streams():
    q, k = make(2, 4, 2, 100, 128, 12)
    freqs = fa.rope_frequencies(128)
    wq, wk = weights(128, 6)
    pos = torch.arange(100, dtype=torch.int32, device="cuda")
    g = randn((2, 4, 100, 128), 1), randn((2, 2, 100, 128), 2)
    kw = dict(q_weight=wq, k_weight=wk)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    fa.forward_rope(q, k, freqs, pos, stream=s, **kw)
    fa.backward_rope(*g, freqs, pos, q=q, k=k, stream=int(s.cuda_stream), **kw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y = fa.forward_rope(q, k, freqs, pos, **kw)
        grads = fa.backward_rope(*g, freqs, pos, q=q, k=k, **kw)
    pos += 1000
    q._base.copy_(randn(tuple(q._base.shape), 30))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((*y, *grads), (*fa.forward_rope(q, k, freqs, pos, **kw), *fa.backward_rope(*g, freqs, pos, q=q, k=k, **kw))):
        assert torch.equal(a, b)
    assert fa.fa_device_status(True) == fa.FA_OK


def test_frequencies():
    f = fa.rope_frequencies(128, 10000.0).cpu()
    i = torch.arange(64, dtype=torch.float64)
    assert torch.allclose(f, 10000.0 ** (-i / 64), rtol=1e-14, atol=0)
    assert torch.allclose(fa.rope_frequencies(128, linear=8.0).cpu(), f / 8, rtol=1e-14, atol=0)
    b = fa.rope_frequencies(128, base_stretch=8.0).cpu()
    assert b[0] == f[0] and math.isclose(float(b[-1]), float(f[-1]) / 8, rel_tol=1e-12)
    r = fa.rope_frequencies(128, ramp=(8.0, 4096, 1.0, 32.0)).cpu()
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(r[turns >= 32], f[turns >= 32]) and torch.allclose(r[turns <= 1], f[turns <= 1] / 8, rtol=1e-14, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert ((r < f) & (r > f / 8))[mid].all()
