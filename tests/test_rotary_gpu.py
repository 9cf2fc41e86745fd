"""Rotary positions against the definition in 64 bits, as complex products.

Bound on an element's error, fixed before the first run.  With x1, x2 its pair
and m the factor, the kernel's cos and sin are off by at most 2^-22 (a few
steps of 2^-24 from sincospi, the product with m, and the angle kept to 2^-33 of
a turn), and the two products and their sum round three times at 2^-24 of at
most m (|x1| + |x2|): in all below 2^-20 m (|x1| + |x2|).  The rounding to the
output's type adds half a step, 2^-8 (bf16) or 2^-11 (f16) of the value, or
2^-25 below f16's normal range."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_67_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def turned(x, pos, freq, factor, interleaved, sign=1):
    """x [..., N, d] turned at pos [N] or broadcastable to x's leading axes + [N]."""
    n = len(freq)
    w = factor * np.exp(1j * sign * np.asarray(pos, np.float64)[..., None] * freq)
    one, two = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = (x[..., one] + 1j * x[..., two]) * w
    y, size = x.copy(), np.zeros_like(x)
    y[..., one], y[..., two] = z.real, z.imag
    size[..., one] = size[..., two] = factor * (np.abs(x[..., one]) + np.abs(x[..., two]))
    return y, size


def check(got, want, size, dtype):
    err = np.abs(f64(got) - want)
    bound = HALF[dtype] * np.abs(want) + 2.0 ** -20 * size + 2.0 ** -25
    assert np.all(err <= bound), f"off by {np.max(err - bound):.3e} over the bound at {np.argmax(err - bound)}"


CASES = [
    # (B, N, Hq, Hk, d, rot, interleaved, dtype, layout, first position)
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, "bhnd", 0),
    (2, 37, 5, 1, 128, 128, False, torch.bfloat16, "bnhd", 12),
    (3, 130, 8, 2, 128, 64, True, torch.float16, "bhnd", 1 << 20),
    (2, 65, 3, 3, 64, 20, False, torch.float16, "bnhd", 99999),
    (1, 33, 4, 4, 64, 6, True, torch.bfloat16, "bhnd", -7),
    (1, 40, 2, 1, 64, 2, False, torch.bfloat16, "bhnd", 5),
    (1, 50, 2, 1, 128, 24, True, torch.bfloat16, "bhnd", 2 ** 31 - 64),
    (1, 50, 7, 1, 128, 72, False, torch.float16, "bnhd", 3),
    (1, 5000, 6, 2, 128, 128, True, torch.bfloat16, "bhnd", 0),
    # Eight tokens a block, blocks across batch entries and a part of one at the end.
    (3, 3333, 5, 1, 64, 64, False, torch.bfloat16, "bhnd", 11),
    (3, 3333, 2, 3, 64, 64, True, torch.float16, "bnhd", 11),
]


def inputs(B, N, H, d, dtype, layout, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, N, d, generator=g).to(dtype).to(DEV)
    return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "bnhd" else x


@pytest.mark.parametrize("B,N,Hq,Hk,d,rot,interleaved,dtype,layout,first", CASES, ids=lambda x: str(x))
def test_rotary_and_its_gradient(B, N, Hq, Hk, d, rot, interleaved, dtype, layout, first):
    import exact_attention_67_gb300 as ex
    q, k = inputs(B, N, Hq, d, dtype, layout, 1), inputs(B, N, Hk, d, dtype, layout, 2)
    freq, factor = ex.rotary_frequencies(rot, yarn=8.0)
    pos = (first + torch.arange(N) + 11 * torch.arange(B)[:, None]).clamp(max=2 ** 31 - 1).to(torch.int32).to(DEV)
    fr, p = freq.cpu().numpy(), pos.cpu().numpy()[:, None]
    for out, x in zip(ex.rotary(q, k, pos, freq, interleaved, factor), (q, k)):
        check(out, *turned(f64(x), p, fr, factor, interleaved), dtype)
        assert out.stride() == x.stride()
    for out, x in zip(ex.rotary_backward(q, k, pos, freq, interleaved, factor), (q, k)):
        check(out, *turned(f64(x), p, fr, factor, interleaved, -1), dtype)
    # Q alone, shared positions, in place, on another stream: the same bits.
    whole = ex.rotary(q, None, pos[0], freq, interleaved, factor)
    stream, same = torch.cuda.Stream(), q.clone()
    stream.wait_stream(torch.cuda.current_stream())
    ex.attn_rotary(same, same, None, None, pos[0], freq, interleaved, False, factor, stream)
    stream.synchronize()
    assert torch.equal(same, whole)


def test_packed_and_defaults():
    import exact_attention_67_gb300 as ex
    g = torch.Generator().manual_seed(3)
    q = torch.randn(70, 4, 64, generator=g).to(torch.bfloat16).to(DEV)
    k = torch.randn(70, 2, 64, generator=g).to(torch.bfloat16).to(DEV)
    freq, _ = ex.rotary_frequencies(64)
    for out, x in zip(ex.rotary(q, k), (q, k)):
        check(out.transpose(0, 1), *turned(f64(x).transpose(1, 0, 2), np.arange(70), freq.cpu().numpy(), 1.0, False),
              torch.bfloat16)
    empty = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    assert ex.rotary(empty).shape == empty.shape


def test_autograd_matches_formula_and_differences():
    """The map is linear: a loss sum(g * y) changes by exactly sum(dx * grad)
    when x moves by dx, up to the outputs' rounding (half a step of each y on
    either side) and the gradient's (half a step of each grad)."""
    import exact_attention_67_gb300 as ex
    B, N, H, d, rot = 2, 19, 3, 64, 32
    q, k = inputs(B, N, H, d, torch.float16, "bhnd", 5), inputs(B, N, 1, d, torch.float16, "bhnd", 6)
    freq, factor = ex.rotary_frequencies(rot, linear=4.0)
    pos = torch.arange(N, dtype=torch.int32, device=DEV) + 1000
    gq, gk = inputs(B, N, H, d, torch.float16, "bnhd", 7), inputs(B, N, 1, d, torch.float16, "bhnd", 8)
    q.requires_grad_(), k.requires_grad_()
    yq, yk = ex.rotary(q, k, pos, freq, True, factor)
    torch.autograd.backward((yq, yk), (gq, gk))
    fr, p = freq.cpu().numpy(), pos.cpu().numpy()
    for x, g in ((q, gq), (k, gk)):
        check(x.grad, *turned(f64(g), p, fr, factor, True, -1), torch.float16)
    with torch.no_grad():
        moved = (q + inputs(B, N, H, d, torch.float16, "bhnd", 9)).contiguous()
        y2 = ex.rotary(moved, None, pos, freq, True, factor)
        dx = f64(moved) - f64(q)
        change = np.sum(f64(gq) * (f64(y2) - f64(yq)))
        bound = np.sum(np.abs(f64(gq)) * (np.abs(f64(y2)) + np.abs(f64(yq)))) + np.sum(np.abs(dx * f64(q.grad)))
        assert abs(change - np.sum(dx * f64(q.grad))) <= 1.02 * 2.0 ** -11 * bound
    # An expanded gradient, as of a plain sum, is read through a copy.
    q.grad = None
    ex.rotary(q, None, pos, freq, True, factor).sum().backward()
    check(q.grad, *turned(np.ones(q.shape), p, fr, factor, True, -1), torch.float16)


def test_unusual_frequencies():
    """Zero, denormal, tiny, negative and large frequencies against rational
    arithmetic: an angle is off by 2^-53 of itself (the double 1 / 2 pi and its
    product) and 2^-33 turns, cos and sin of it by 2^-22 more in fp32."""
    from fractions import Fraction
    import exact_attention_67_gb300 as ex
    pi = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
    fs = [0.0, 5e-324, 1e-300, 1e-12, 1e-3, 0.5, -0.5, 1.0, 3.0, -7.5, 100.0, 2.0 ** 20 + 0.3]
    ps = [0, 1, -1, 2, 77, 999]
    freq = torch.tensor(fs, dtype=torch.float64, device=DEV)
    q = torch.zeros(1, 1, len(ps), 64, dtype=torch.float16, device=DEV)
    q[..., : len(fs)] = 1.0                                         # pairs (1, 0): the outputs are cos and sin
    y = ex.rotary(q, None, torch.tensor(ps, dtype=torch.int32, device=DEV), freq)[0, 0].double().cpu().numpy()
    for i, p in enumerate(ps):
        for j, f in enumerate(fs):
            turns = Fraction(f) * p / (2 * pi)
            angle = 2 * np.pi * float(turns - round(turns))
            off = 2 * np.pi * (abs(float(turns)) * 2.0 ** -53 + 2.0 ** -33) + 2.0 ** -22
            for got, want in ((y[i, j], np.cos(angle)), (y[i, j + len(fs)], np.sin(angle))):
                assert abs(got - want) <= 2.0 ** -11 * abs(want) + 2.0 ** -25 + off, (p, f, got, want)


def test_capture_and_replay():
    import exact_attention_67_gb300 as ex
    q, k = inputs(1, 300, 4, 128, torch.bfloat16, "bhnd", 11), inputs(1, 300, 2, 128, torch.bfloat16, "bhnd", 12)
    pos = torch.arange(300, dtype=torch.int32, device=DEV)
    freq, _ = ex.rotary_frequencies(128)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    ex.attn_rotary(q, qo, k, ko, pos, freq)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.attn_rotary(q, qo, k, ko, pos, freq)
    pos.add_(12345)
    graph.replay()
    torch.cuda.synchronize()
    check(qo, *turned(f64(q), 12345 + np.arange(300), freq.cpu().numpy(), 1.0, False), torch.bfloat16)
    check(ko, *turned(f64(k), 12345 + np.arange(300), freq.cpu().numpy(), 1.0, False), torch.bfloat16)


def test_forward_and_backward_captured():
    import exact_attention_67_gb300 as ex
    q = inputs(2, 40, 3, 64, torch.bfloat16, "bhnd", 13).requires_grad_()
    g = inputs(2, 40, 3, 64, torch.bfloat16, "bhnd", 14)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    freq, _ = ex.rotary_frequencies(64)

    def step():
        y = ex.rotary(q, None, pos, freq)
        return y, torch.autograd.grad(y, q, g)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, dq = step()
    pos.add_(777)
    graph.replay()
    torch.cuda.synchronize()
    p, fr = 777 + np.arange(40), freq.cpu().numpy()
    check(y, *turned(f64(q), p, fr, 1.0, False), torch.bfloat16)
    check(dq, *turned(f64(g), p, fr, 1.0, False, -1), torch.bfloat16)


def test_then_attention():
    """Rotary then the framework's causal attention, forward and backward, as a
    training step runs them, against both in 64 bits."""
    import exact_attention_67_gb300 as ex
    import oracle
    from tests.parity import check_fwd, check_grads
    B, H, N, d = 1, 2, 200, 64
    q, k, v, do = (inputs(B, N, H, d, torch.bfloat16, "bhnd", 20 + i) for i in range(4))
    freq, _ = ex.rotary_frequencies(d)
    pos = torch.arange(N, dtype=torch.int32, device=DEV) + 500
    q.requires_grad_(), k.requires_grad_(), v.requires_grad_()
    rq, rk = ex.rotary(q, k, pos, freq)
    o = ex.attention(rq, rk, v, causal=True)
    o.backward(do)
    fr, p, scale = freq.cpu().numpy(), pos.cpu().numpy(), float(torch.tensor(d ** -0.5, dtype=torch.float32))
    o_ref, lse_ref = oracle.attention_fwd(f64(rq), f64(rk), f64(v), True, scale)
    check_fwd(f64(o), lse_ref, o_ref, lse_ref, "rotary + attention")
    dq, dk, dv = oracle.attention_bwd(f64(rq), f64(rk), f64(v), f64(do), True, scale)
    check_grads([("dQ", f64(q.grad), turned(dq, p, fr, 1.0, False, -1)[0]),
                 ("dK", f64(k.grad), turned(dk, p, fr, 1.0, False, -1)[0]), ("dV", f64(v.grad), dv)], "rotary + attention")


def test_refusals():
    import exact_attention_67_gb300 as ex
    q = inputs(1, 8, 2, 64, torch.bfloat16, "bhnd", 1)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    freq, _ = ex.rotary_frequencies(64)
    with pytest.raises(TypeError):
        ex.rotary(q, None, pos.long(), freq)
    with pytest.raises(TypeError):
        ex.rotary(q.float(), None, pos, freq)
    with pytest.raises(ValueError):
        ex.rotary(q, None, pos[:7], freq)
    with pytest.raises(ValueError):
        ex.rotary(q, None, pos, freq.float())
    with pytest.raises(ValueError):
        ex.rotary(q, q[:, :, :4], pos, freq)
    with pytest.raises(ValueError):
        ex.rotary(q, None, pos.cpu(), freq)
    with pytest.raises(ex.ExattnError):
        ex.rotary(q[:, :0], q, pos, freq)      # no query head, but keys
    with pytest.raises(ex.ExattnError):
        ex.rotary(q, None, pos, freq, factor=0.0)
    with pytest.raises(ex.ExattnError):
        ex.rotary(q, None, pos, ex.rotary_frequencies(128)[0])  # more than a head


@pytest.mark.parametrize("name,sign", [("rotary", 1), ("rotary_backward", -1)])
def test_forward_mode_and_second_order(name, sign):
    """Tangents are turned like the values, with the same bound; rotary_backward is
    differentiable itself."""
    import exact_attention_67_gb300 as ex
    from torch.autograd import forward_ad
    call = getattr(ex, name)
    q, k, tq, tk = (inputs(2, 37, h, 64, torch.bfloat16, "bnhd", 30 + i) for i, h in enumerate((3, 1, 3, 1)))
    freq, factor = ex.rotary_frequencies(64, yarn=2.0)
    pos = torch.arange(37, dtype=torch.int32, device=DEV) + 9
    fr, p = freq.cpu().numpy(), pos.cpu().numpy()
    with forward_ad.dual_level():
        out = call(forward_ad.make_dual(q, tq), forward_ad.make_dual(k, tk), pos, freq, True, factor)
        for o, x, t in zip(out, (q, k), (tq, tk)):
            got = forward_ad.unpack_dual(o)
            check(got.primal, *turned(f64(x), p, fr, factor, True, sign), torch.bfloat16)
            check(got.tangent, *turned(f64(t), p, fr, factor, True, sign), torch.bfloat16)
    q.requires_grad_()
    g = tq.clone().requires_grad_()
    dq, = torch.autograd.grad(call(q, None, pos, freq, True, factor), q, g, create_graph=True)
    check(dq, *turned(f64(tq), p, fr, factor, True, -sign), torch.bfloat16)
    back, = torch.autograd.grad(dq, g, q.detach())
    check(back, *turned(f64(q), p, fr, factor, True, sign), torch.bfloat16)


@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_that_are_not_finite(interleaved):
    """Their pairs are NaN, as by the formula, position 0 among them; the others are
    what they are without them."""
    import exact_attention_67_gb300 as ex
    q = inputs(1, 40, 3, 64, torch.bfloat16, "bhnd", 41)
    freq, _ = ex.rotary_frequencies(64)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    want = ex.rotary(q, None, pos, freq, interleaved)
    for at, bad in ((0, float("nan")), (7, float("inf")), (31, -float("inf"))):
        f = freq.clone()
        f[at] = bad
        hit = torch.zeros(64, dtype=torch.bool, device=DEV)
        hit[[2 * at, 2 * at + 1] if interleaved else [at, at + 32]] = True
        for y in (ex.rotary(q, None, pos, f, interleaved), ex.rotary_backward(q, None, pos, f, interleaved)):
            assert bool(torch.isnan(y[..., hit]).all()) and not bool(torch.isnan(y[..., ~hit]).any())
        assert torch.equal(ex.rotary(q, None, pos, f, interleaved)[..., ~hit], want[..., ~hit])
        pages = torch.zeros(2, 40, 1, 8, 64, dtype=torch.bfloat16, device=DEV)
        table = torch.arange(5, dtype=torch.int32, device=DEV)[None]
        k = q[0, :1].transpose(0, 1).contiguous()
        ex.attn_cache_append(k, k, pages[0], pages[1], table, torch.tensor([40], dtype=torch.int32, device=DEV), inv_freq=f,
                             interleaved=interleaved)
        stored = pages[0, :5, 0].reshape(40, 64)
        assert bool(torch.isnan(stored[:, hit]).all()) and torch.equal(stored[:, ~hit], want[0, 0][:, ~hit])
