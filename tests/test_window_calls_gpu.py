"""Calls of the windowed attention and the rotation that their documentation allows, on the GPU."""
import pytest
import torch

from exact_io_aware_32_gb300 import fa
from test_window_gpu import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
def test_workspace_anywhere_on_16_bytes(d):
    """The same bits whatever 16-byte boundary the workspace begins at, and nothing behind its end is touched."""
    q, k, v, dO = inputs(2, 4, 2, 333, 400, d, 1)
    o, lse = fa.forward_window(q, k, v, 100, 3)
    ref = fa.backward_window(q, k, v, o, lse, dO, 100, 3)
    need = fa.fa_bwd_window_workspace_bytes(2, 4, 2, 333, 400, d, 100, 3)
    arena = torch.empty(need + 512, dtype=torch.uint8, device="cuda")
    for at in (16, 48, 240, 256):
        arena.fill_(0xA5)
        got = fa.backward_window(q, k, v, o, lse, dO, 100, 3, workspace=arena[at:at + need])
        assert all(torch.equal(x, r) for x, r in zip(got, ref)), at
        assert (arena[:at] == 0xA5).all() and (arena[at + need:] == 0xA5).all()
    assert fa.fa_device_status(True) == fa.FA_OK


def off_by(x, n):
    """x as a contiguous view that begins n elements into its storage."""
    y = torch.empty(x.numel() + n, dtype=x.dtype, device=x.device)[n:].view(x.shape)
    y.copy_(x)
    assert y.is_contiguous() and y.data_ptr() % 16
    return y


@pytest.mark.parametrize("n", [1, 4])
def test_gradients_that_begin_anywhere(n):
    """Contiguous gradients off 16 bytes, as a slice of a larger buffer is, give what aligned ones give."""
    q, k, v, dO = inputs(1, 4, 2, 130, 130, 64, 2)
    freqs = fa.rope_frequencies(64)
    dk = dO[:, :2].contiguous()
    x = [y.requires_grad_() for y in (q, k, v)]
    for out, leaves, g in ((fa.attention_window(*x, 50, 1), x, (dO,)), (fa.rope(q, k, freqs), x[:2], (dO, dk)),
                           (fa.attention(q, q, q, causal=True), x[:1], (dO,)),
                           (fa.attention(q, q, q, dropout_p256=25, seed=3), x[:1], (dO,))):
        ref = torch.autograd.grad(out, leaves, g, retain_graph=True)
        got = torch.autograd.grad(out, leaves, [off_by(y, n) for y in g])
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("linear", [False, True])
@pytest.mark.parametrize("kind", ["attention", "dropout", "attention_window", "rope", "norm rope"])
def test_second_derivatives_are_refused(kind, linear):
    """A gradient made with create_graph is right, and the gradient of it an error, not one that leaves terms out, also where the
    loss is linear in the outputs. (Of a rotation without norms it is then zero, which is right.)"""
    q, k, v, _ = (x.requires_grad_() for x in inputs(1, 2, 2, 40, 40, 64, 3))
    w = torch.ones(64, device="cuda", requires_grad=True)
    freqs = fa.rope_frequencies(64)
    out = {"attention": lambda: fa.attention(q, k, v), "dropout": lambda: fa.attention(q, k, v, dropout_p256=20, seed=1),
           "attention_window": lambda: fa.attention_window(q, k, v, 9), "rope": lambda: fa.rope(q, k, freqs)[0],
           "norm rope": lambda: fa.rope(q, k, freqs, q_weight=w, k_weight=w)[0]}[kind]

    def gradients(**kw):
        y = out().float()
        return torch.autograd.grad((y if linear else y.square()).sum(), q, **kw)[0]
    first, plain = gradients(create_graph=True), gradients()
    assert torch.equal(first, plain)
    loss = q.float().square().sum() + first.float().square().sum()  # a penalty on the gradient beside another term
    if kind == "rope" and linear:
        assert torch.equal(torch.autograd.grad(loss, q)[0], 2 * q)
        return
    with pytest.raises(RuntimeError, match="second derivatives"):
        loss.backward()


def test_gradients_with_create_graph_accumulate():
    """backward(create_graph=True) fills the leaves' gradients as without it, unused ones left out."""
    for kw in (dict(), dict(create_graph=True)):
        q, k, v, dO = inputs(1, 4, 2, 60, 60, 128, 4)
        q.requires_grad_()
        w = torch.ones(128, device="cuda", requires_grad=True)
        freqs = fa.rope_frequencies(128)
        x, y = fa.rope(q, k, freqs, q_weight=w, k_weight=w)
        fa.attention_window(x, y, v, 20, 1).backward(dO, **kw)
        if not kw:
            ref = q.grad, w.grad
    assert torch.equal(q.grad, ref[0]) and torch.equal(w.grad, ref[1])
    q.grad = w.grad = None  # (a gradient with a graph refers to its leaf)
