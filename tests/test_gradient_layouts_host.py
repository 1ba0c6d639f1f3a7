"""Gradients as autograd hands them over, brought into the form that the kernels read (on the CPU)."""
import pytest
import torch

from exact_io_aware_32_gb300 import fa


def view(off, shape, dtype=torch.bfloat16):
    """A contiguous tensor that begins 'off' elements into its storage."""
    n = 1
    for s in shape:
        n *= s
    return torch.randn(n + off, generator=torch.Generator().manual_seed(off)).to(dtype)[off:].view(shape)


@pytest.mark.parametrize("call", [fa._gradient, fa._rows_contiguous])
@pytest.mark.parametrize("off", [0, 1, 2, 4, 7, 8, 12])
def test_contiguous_gradients_begin_on_16_bytes(off, call):
    x = view(off, (2, 3, 5, 64))
    y = call(x)
    assert y.dtype == torch.bfloat16 and y.is_contiguous() and y.data_ptr() % 16 == 0 and torch.equal(x, y)
    assert (y.data_ptr() == x.data_ptr()) == (x.data_ptr() % 16 == 0)  # copied only where it has to be


@pytest.mark.parametrize("call", [fa._gradient, fa._rows_contiguous])
def test_other_layouts_and_types(call):
    for x in (view(3, (2, 5, 3, 64)).transpose(1, 2), view(1, (2, 3, 64, 5)).transpose(2, 3), torch.ones(()).to(torch.bfloat16).expand(2, 3, 5, 64),
              view(1, (2, 3, 5, 64), torch.float32), view(1, (2, 3, 5, 66))[..., :64], view(0, (2, 3, 5, 72))[..., 8:]):
        y = call(x)
        assert y.dtype == torch.bfloat16 and y.stride(3) == 1 and y.data_ptr() % 16 == 0 and torch.equal(x.to(torch.bfloat16), y)
        assert all(s % 8 == 0 for s in y.stride()[:3])
