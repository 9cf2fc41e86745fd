"""rotary and rotary_backward under automatic differentiation, on the CPU: the
native call is replaced by the definition in 64 bits, so what is tested is which
calls are made with what."""
import pytest
import torch
from torch.autograd import forward_ad

import exact_attention_67_gb300 as ex
from exact_attention_67_gb300 import paged


class Definition:
    """The native module's rotary_new on host tensors; keeps what it was given."""

    def __init__(self):
        self.given = []

    def rotary_new(self, q, k, positions, inv_freq, interleaved, inverse, factor, stream):
        assert not interleaved
        n = inv_freq.numel()
        w = torch.polar(torch.full((positions.numel(), n), float(factor), dtype=torch.float64),
                        (-1 if inverse else 1) * positions.double()[:, None] * inv_freq)

        def turn(x):
            self.given.append(x)
            y = x.double().clone()
            z = torch.complex(y[..., :n].contiguous(), y[..., n: 2 * n].contiguous()) * w
            y[..., :n], y[..., n: 2 * n] = z.real, z.imag
            return y.to(x.dtype)

        return 0, turn(q.detach()), None if k is None else turn(k.detach())


@pytest.fixture
def native(monkeypatch):
    d = Definition()
    monkeypatch.setattr(paged, "_native", lambda: d)
    return d


FREQ, _ = ex.rotary_frequencies(32, device="cpu")
POS = torch.arange(5, dtype=torch.int32) + 3


def half(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).half()


def turn(x, inverse=False, factor=1.5):
    return Definition().rotary_new(x, None, POS, FREQ, False, inverse, factor, None)[1]


@pytest.mark.parametrize("call,inverse", [(ex.rotary, False), (ex.rotary_backward, True)])
def test_forward_mode(native, call, inverse):
    """The map is linear: the tangents are the same call on the inputs' tangents."""
    q, k, tq, tk = (half(1, h, 5, 64, seed=s) for s, h in enumerate((3, 2, 3, 2)))
    for with_k in (True, False):
        for no_grad in (False, True):
            with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
                out = call(forward_ad.make_dual(q, tq), forward_ad.make_dual(k, tk) if with_k else None, POS, FREQ, factor=1.5)
                for o, x, t in zip(out if with_k else [out], (q, k), (tq, tk)):
                    primal, tangent = forward_ad.unpack_dual(o)
                    assert torch.equal(primal, turn(x, inverse))
                    assert tangent is not None and torch.equal(tangent, turn(t, inverse))
    # A tangent of one input only: the other output moves by nothing.
    with forward_ad.dual_level():
        a, b = call(q, forward_ad.make_dual(k, tk), POS, FREQ, factor=1.5)
        ta, tb = forward_ad.unpack_dual(a).tangent, forward_ad.unpack_dual(b).tangent
        assert ta is None or not ta.any()
        assert torch.equal(tb, turn(tk, inverse))


@pytest.mark.parametrize("call,inverse", [(ex.rotary, False), (ex.rotary_backward, True)])
def test_reverse_mode(native, call, inverse):
    q, k, gq, gk = (half(1, h, 5, 64, seed=s) for s, h in enumerate((3, 2, 3, 2)))
    q.requires_grad_(), k.requires_grad_()
    out = call(q, k, POS, FREQ, factor=1.5)
    torch.autograd.backward(out, (gq, gk))
    assert torch.equal(q.grad, turn(gq, not inverse)) and torch.equal(k.grad, turn(gk, not inverse))
    with torch.no_grad():
        assert not call(q, None, POS, FREQ).requires_grad


@pytest.mark.parametrize("call,inverse", [(ex.rotary, False), (ex.rotary_backward, True)])
def test_second_order(native, call, inverse):
    """Of f = (sum of y^2 over a weight) / 2 the gradient is R^T (w R x) and its
    derivative along t is R^T (w R t): by reverse over reverse, forward over reverse
    and reverse over forward, to the roundings of the f16 values."""
    x, t, w = half(1, 2, 5, 64, seed=1), half(1, 2, 5, 64, seed=2), half(1, 2, 5, 64, seed=3)
    want = turn(w * turn(t, inverse), not inverse)

    def gradient(q):
        y = call(q, None, POS, FREQ, factor=1.5)
        return torch.autograd.grad(y, q, w * y, create_graph=True)[0]

    q = x.clone().requires_grad_()
    twice, = torch.autograd.grad(gradient(q), q, t)
    with forward_ad.dual_level():
        over = forward_ad.unpack_dual(gradient(forward_ad.make_dual(x.clone().requires_grad_(), t))).tangent
        q = x.clone().requires_grad_()
        v = t.clone().requires_grad_()
        y = call(forward_ad.make_dual(q, v), None, POS, FREQ, factor=1.5)
        ty = forward_ad.unpack_dual(y).tangent
        under, = torch.autograd.grad(ty, v, w * ty.detach())
    for got in (twice, over, under):
        assert got is not None and torch.allclose(got.double(), want.double(), rtol=2 ** -8, atol=2 ** -8)


def offset(x, by=1):
    """The same values, contiguous, in a buffer of their own from element `by` on."""
    flat = torch.empty(x.numel() + by, dtype=x.dtype)
    y = flat[by:].view(x.shape)
    assert y.is_contiguous() and y.data_ptr() % 16
    return y.copy_(x)


def odd_stride(x):
    """The same values with a stride of 5 along an axis of one."""
    y = x.as_strided(x.shape, (x.stride(0), 5, x.stride(2), x.stride(3)))
    assert x.shape[1] == 1 and y.is_contiguous()
    return y


@pytest.mark.parametrize("spoil", [offset, odd_stride, lambda x: x.transpose(2, 3).contiguous().transpose(2, 3),
                                   lambda x: x[..., :1, :].expand_as(x)])
def test_gradients_that_cannot_be_read_in_place(native, spoil):
    """The native call gets them aligned, d contiguous, with strides of its kind."""
    q, g = half(2, 1, 5, 64, seed=1).requires_grad_(), half(2, 1, 5, 64, seed=2)
    bad = spoil(g)
    y = ex.rotary(q, None, POS, FREQ, factor=1.5)
    native.given.clear()
    y.backward(bad)
    got, = native.given
    assert got.data_ptr() % 16 == 0 and got.stride(3) == 1 and all(s % 8 == 0 for s in got.stride()[:3])
    assert torch.equal(q.grad, turn(bad, True))
    with forward_ad.dual_level():
        native.given.clear()
        out = ex.rotary(forward_ad.make_dual(q.detach(), bad), None, POS, FREQ, factor=1.5)
        assert torch.equal(forward_ad.unpack_dual(out).tangent, turn(bad))
        assert native.given[-1].data_ptr() % 16 == 0 and all(s % 8 == 0 for s in native.given[-1].stride()[:3])
