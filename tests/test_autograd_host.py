"""What the attention's backward pass hands to the library, on the CPU: the
library's forward and backward are replaced by a record of their arguments."""
import pytest
import torch

from exact_attention_67_gb300 import autograd


def offset(x):
    """The same values, contiguous, one element into a buffer of their own."""
    flat = torch.empty(x.numel() + 1, dtype=x.dtype)
    return flat[1:].view(x.shape).copy_(x)


def odd_stride(x):
    """The same values with a stride of 5 along the axis of one head."""
    return x.as_strided(x.shape, (x.stride(0), 5, x.stride(2), x.stride(3)))


@pytest.mark.parametrize("fp32_o", [False, True])
@pytest.mark.parametrize("spoil", [offset, odd_stride, lambda x: x.transpose(2, 3).contiguous().transpose(2, 3),
                                   lambda x: x[..., :1, :].expand_as(x)])
def test_gradients_that_cannot_be_read_in_place(monkeypatch, spoil, fp32_o):
    given = []

    def forward(q, k, v, causal, scale, window, fp32_o=False):
        o = torch.zeros_like(q)
        return (o, q.new_zeros(q.shape[:3]), o.float()) if fp32_o else (o, q.new_zeros(q.shape[:3]))

    def backward(q, k, v, o, lse, do, causal, scale, window, o32=None):
        given.append(do)
        return do, do, do

    monkeypatch.setattr(autograd, "_forward", forward)
    monkeypatch.setattr(autograd, "_backward", backward)
    q, k, v, g = (torch.randn(2, 1, 5, 64, generator=torch.Generator().manual_seed(s)).half() for s in range(4))
    q.requires_grad_()
    bad = spoil(g)
    autograd.attention(q, k, v, fp32_o=fp32_o).backward(bad)
    got, = given
    assert got.data_ptr() % 16 == 0 and got.stride(3) == 1 and all(s and s % 8 == 0 for s in got.stride()[:3])
    assert torch.equal(got, bad) and torch.equal(q.grad, bad)
