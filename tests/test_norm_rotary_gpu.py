"""Norms of the heads with the rotary turn, their gradient and the same into a paged
cache, against the definition in 64 bits.

Bounds on an element's error, fixed before the first run; u = 2^-24, the fp32 half step.
  Size of a row: its squares are all positive, each goes through at most 24 additions
    (16 in a thread, 5 exchanges) and 3 more roundings, rsqrt is good to 2 steps: r is
    off by less than 2^-19 of itself, and n = x r g, two products, by 2^-18.9.
  Turn: 2^-20 of size = m (|n1| + |n2|) (test_rotary_gpu), so the output by 2^-18 of it,
    and half a step of the output's type, 2^-8 (bf16) or 2^-11 (f16) of the value, or
    2^-25 below f16's normal range.
  Gradient, h = m R^T dy off by 2^-20 H, H = m (|dy1| + |dy2|): the sum of g h x by
    (2^-20 + 27 u + u) of sum H |g x|, so mean(g h e) by 2^-17 of M = mean(H |g e|), and
    dx = (g h - e mean) r by 2^-16 of r (H |g| + |e| M), and the rounding to its type.
  Gains' gradient: a term h e by 2^-18 of H |e|; the additions a term goes through: at
    most 600 in a thread, 64 in a block, 40 over the blocks, below 2^10 u in all, so
    2^-14 + 2^-18 of sum H |e|, and the rounding to the gain's type."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_67_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def eps32(eps):
    return float(np.float32(eps))


def pairs(freq, interleaved):
    n = len(freq)
    return (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))


def turned(x, pos, freq, factor, interleaved, sign=1):
    """x [..., N, d] turned at pos, and the size of each element's terms."""
    y, size = x.copy(), np.abs(x)
    if len(freq):
        w = factor * np.exp(1j * sign * np.asarray(pos, np.float64)[..., None] * freq)
        one, two = pairs(freq, interleaved)
        z = (x[..., one] + 1j * x[..., two]) * w
        y[..., one], y[..., two] = z.real, z.imag
        size[..., one] = size[..., two] = factor * (np.abs(x[..., one]) + np.abs(x[..., two]))
    return y, size


def normed(x, gain, pos, freq, factor, interleaved, eps=EPS):
    s = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps32(eps))
    return turned(x / s * gain, pos, freq, factor, interleaved)


def normed_grad(dy, x, gain, pos, freq, factor, interleaved, eps=EPS):
    """(dx, its bound's unit, dg, its bound's unit); sums over all axes but the last for dg."""
    s = np.sqrt(np.mean(x * x, -1, keepdims=True) + eps32(eps))
    h, H = turned(dy, pos, freq, factor, interleaved, -1)
    e = x / s
    u = gain * h
    dx = (u - e * np.mean(u * e, -1, keepdims=True)) / s
    M = np.mean(H * np.abs(gain * e), -1, keepdims=True)
    axes = tuple(range(x.ndim - 1))
    return dx, (H * np.abs(gain) + np.abs(e) * M) / s, (h * e).sum(axes), (H * np.abs(e)).sum(axes)


def check(got, want, size, dtype, unit=2.0 ** -18):
    err = np.abs(f64(got) - want)
    bound = HALF[dtype] * np.abs(want) + unit * size + 2.0 ** -25
    assert np.all(err <= bound), f"off by {np.max(err - bound):.3e} over the bound at {np.argmax(err - bound)}"


CASES = [
    # (B, N, Hq, Hk, d, rot, interleaved, dtype, gain type, layout, first position)
    (1, 1, 1, 1, 64, 64, False, torch.bfloat16, torch.bfloat16, "bhnd", 0),
    (2, 37, 5, 1, 128, 128, False, torch.bfloat16, torch.float32, "bnhd", 12),
    (3, 130, 8, 2, 128, 64, True, torch.float16, torch.float16, "bhnd", 1 << 20),
    (2, 65, 3, 3, 64, 20, False, torch.float16, torch.float32, "bnhd", 99999),
    (1, 33, 4, 4, 64, 6, True, torch.bfloat16, torch.bfloat16, "bhnd", -7),
    (2, 40, 3, 2, 128, 6, False, torch.bfloat16, torch.float32, "bnhd", 5),
    (1, 41, 2, 1, 128, 2, True, torch.float16, torch.float16, "bhnd", 5),
    (1, 50, 2, 1, 128, 24, True, torch.bfloat16, torch.bfloat16, "bhnd", 2 ** 31 - 64),
    (1, 50, 7, 1, 128, 72, False, torch.float16, torch.float32, "bnhd", 3),
    (1, 77, 7, 1, 128, 36, False, torch.bfloat16, torch.float32, "bnhd", 3),
    (1, 5000, 6, 2, 128, 128, True, torch.bfloat16, torch.bfloat16, "bhnd", 0),
    # Eight tokens a block, blocks across batch entries and a part of one at the end.
    (3, 3333, 5, 1, 64, 64, False, torch.bfloat16, torch.float32, "bhnd", 11),
    (3, 3333, 2, 3, 64, 64, True, torch.float16, torch.float32, "bnhd", 11),
    (1, 9999, 1, 1, 64, 6, False, torch.bfloat16, torch.float32, "bhnd", 11),
]


def rows(B, N, H, d, dtype, layout, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, N, d, generator=g) * torch.exp(spread * torch.randn(B, H, N, 1, generator=g))
    x = x.to(dtype).to(DEV)
    return x.transpose(1, 2).contiguous().transpose(1, 2) if layout == "bnhd" else x


def gain_of(d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (1 + 0.3 * torch.randn(d, generator=g)).to(dtype).to(DEV)


def case(B, N, Hq, Hk, d, rot, interleaved, dtype, gtype, layout, first):
    import exact_attention_67_gb300 as ex
    freq, factor = ex.rotary_frequencies(rot, yarn=8.0)
    pos = (first + torch.arange(N) + 11 * torch.arange(B)[:, None]).clamp(max=2 ** 31 - 1).to(torch.int32).to(DEV)
    return dict(x=(rows(B, N, Hq, d, dtype, layout, 1), rows(B, N, Hk, d, dtype, layout, 2)),
                dy=(rows(B, N, Hq, d, dtype, layout, 3, 0.5), rows(B, N, Hk, d, dtype, layout, 4, 0.5)),
                gain=(gain_of(d, gtype, 5), gain_of(d, gtype, 6)), pos=pos, freq=freq, factor=factor,
                args=(f64(freq), factor, interleaved), p=pos.cpu().numpy()[:, None])


@pytest.mark.parametrize("c", CASES, ids=lambda c: "-".join(str(x).replace("torch.", "") for x in c))
def test_norm_and_its_gradient(c):
    import exact_attention_67_gb300 as ex
    s, interleaved, dtype, gtype = case(*c), c[6], c[7], c[8]
    how = dict(positions=s["pos"], inv_freq=s["freq"], interleaved=interleaved, factor=s["factor"], eps=EPS)
    for out, x, g in zip(ex.norm_rotary(*s["x"], *s["gain"], **how), s["x"], s["gain"]):
        assert out.stride() == x.stride() and out.dtype == dtype
        check(out, *normed(f64(x), f64(g), s["p"], *s["args"]), dtype)
    grads = ex.norm_rotary_backward(*s["dy"], *s["x"], *s["gain"], **how)
    again = ex.norm_rotary_backward(*s["dy"], *s["x"], *s["gain"], **how)
    for i in range(2):
        dx, dx_size, dg, dg_size = normed_grad(f64(s["dy"][i]), f64(s["x"][i]), f64(s["gain"][i]), s["p"], *s["args"])
        check(grads[i], dx, dx_size, dtype, 2.0 ** -16)
        check(grads[2 + i], dg, dg_size, gtype, 2.0 ** -14 + 2.0 ** -18)
        assert grads[2 + i].dtype == gtype and tuple(grads[2 + i].shape) == (c[4],)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_without_k_or_gains_and_packed():
    import exact_attention_67_gb300 as ex
    s = case(1, 45, 3, 2, 128, 128, False, torch.bfloat16, torch.float32, "bnhd", 9)
    how = dict(positions=s["pos"], inv_freq=s["freq"], factor=s["factor"], eps=EPS)
    ones = np.ones(128)
    check(ex.norm_rotary(s["x"][0], **how), *normed(f64(s["x"][0]), ones, s["p"], *s["args"]), torch.bfloat16)
    dq, dk, dqg, dkg = ex.norm_rotary_backward(s["dy"][0], None, s["x"][0], None, None, None, **how)
    assert dk is None and dqg is None and dkg is None
    check(dq, *normed_grad(f64(s["dy"][0]), f64(s["x"][0]), ones, s["p"], *s["args"])[:2], torch.bfloat16, 2.0 ** -16)
    # A gain of Q only; packed tensors of one batch entry give the same bits.
    both = ex.norm_rotary(*s["x"], s["gain"][0], None, **how)
    packed = [x[0].transpose(0, 1) for x in s["x"]]  # [N, H, d]
    flat = dict(how, positions=s["pos"][0])
    got = ex.norm_rotary(*packed, s["gain"][0], None, **flat)
    assert all(torch.equal(a, b[0].transpose(0, 1)) for a, b in zip(got, both))
    g4 = ex.norm_rotary_backward(*s["dy"], *s["x"], s["gain"][0], None, **how)
    g3 = ex.norm_rotary_backward(*(x[0].transpose(0, 1) for x in s["dy"]), *packed, s["gain"][0], None, **flat)
    assert g4[3] is None and g3[3] is None and torch.equal(g3[2], g4[2])
    assert all(torch.equal(a, b[0].transpose(0, 1)) for a, b in zip(g3[:2], g4[:2]))


def test_defaults_and_empty():
    import exact_attention_67_gb300 as ex
    x = rows(2, 20, 2, 64, torch.float16, "bhnd", 1)
    freq, _ = ex.rotary_frequencies(64)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    assert torch.equal(ex.norm_rotary(x), ex.norm_rotary(x, None, None, None, pos, freq, False, 1.0, 1e-6))
    none, g = x[:, :, :0], gain_of(64, torch.float32, 1)
    assert ex.norm_rotary(none, none, g, g)[0].shape == none.shape
    got = ex.norm_rotary_backward(none, none, none, none, g, g)
    assert got[0].shape == none.shape and not got[2].any() and not got[3].any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_of_zeros_nan_and_far_values(dtype):
    import exact_attention_67_gb300 as ex
    x = rows(1, 8, 2, 128, dtype, "bhnd", 3)
    x[0, 0, 0] = 0
    x[0, 0, 1, 5] = float("nan")
    x[0, 0, 2, 7] = float("inf")
    x[0, 0, 3] = torch.finfo(dtype).tiny
    x[0, 0, 4] = 60000.0
    pos, (freq, _) = torch.arange(8, dtype=torch.int32, device=DEV), ex.rotary_frequencies(128)
    y = ex.norm_rotary(x, None, None, None, pos, freq, eps=EPS)
    good = [0, 3, 4, 5, 6, 7]
    want, size = normed(f64(x[0, 0, good]), np.ones(128), np.array(good), f64(freq), 1.0, False)
    check(y[0, 0, good], want, size, dtype)
    assert y[0, 0, 1].isnan().all() and not y[0, 0, good].isnan().any() and not y[0, 1].isnan().any()
    # NaN and infinities stay in their rows of dx too.
    dy = rows(1, 8, 2, 128, dtype, "bhnd", 4)
    dx = ex.norm_rotary_backward(dy, None, x, None, None, None, pos, freq, eps=EPS)[0]
    assert dx[0, 0, 1].isnan().all() and not dx[0, 0, good].isnan().any() and not dx[0, 1].isnan().any()
    # With eps = 0 a row of zeros is 0 / 0.
    assert ex.norm_rotary(x, None, None, None, pos, freq, eps=0.0)[0, 0, 0].isnan().all()


def test_outputs_in_place_and_strided():
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import attn_norm_rotary, attn_norm_rotary_backward, attn_norm_rotary_backward_workspace_size
    s = case(2, 300, 4, 2, 128, 64, False, torch.bfloat16, torch.float32, "bnhd", 9)
    how = dict(positions=s["pos"], inv_freq=s["freq"], factor=s["factor"], eps=EPS)
    want = ex.norm_rotary(*s["x"], *s["gain"], **how)
    want_grad = ex.norm_rotary_backward(*s["dy"], *s["x"], *s["gain"], **how)
    # Q and K as views of one projection [B, N, Hq + 2 Hk, d], in place.
    qkv = torch.zeros(2, 300, 8, 128, dtype=torch.bfloat16, device=DEV)
    q, k = qkv[:, :, :4].transpose(1, 2), qkv[:, :, 4:6].transpose(1, 2)
    q.copy_(s["x"][0])
    k.copy_(s["x"][1])
    attn_norm_rotary(q, q, k, k, s["pos"], s["freq"], *s["gain"], False, s["factor"], EPS)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and not qkv[:, :, 6:].any()
    ws = torch.empty(attn_norm_rotary_backward_workspace_size(2, 300, 128), dtype=torch.uint8, device=DEV)
    for over in ("dy", "x"):
        dy, x = [[t.clone(memory_format=torch.preserve_format) for t in s[n]] for n in ("dy", "x")]
        out = dy if over == "dy" else x
        dg = [torch.empty(128, device=DEV) for _ in range(2)]
        ws.fill_(255)  # NaN: nothing in it is read before it is written
        attn_norm_rotary_backward(dy[0], x[0], out[0], dy[1], x[1], out[1], s["pos"], s["freq"], *s["gain"], *dg, False, s["factor"],
                                  EPS, ws)
        assert all(torch.equal(a, b) for a, b in zip((*out, *dg), want_grad))
    # One gain's gradient only.
    dg = torch.empty(128, device=DEV)
    attn_norm_rotary_backward(s["dy"][0], s["x"][0], dy[0], s["dy"][1], s["x"][1], dy[1], s["pos"], s["freq"], *s["gain"], None, dg,
                              False, s["factor"], EPS, ws)
    assert torch.equal(dg, want_grad[3])


def test_autograd_is_the_gradient():
    import exact_attention_67_gb300 as ex
    s = case(2, 65, 4, 2, 64, 32, True, torch.bfloat16, torch.float32, "bnhd", 100)
    how = dict(positions=s["pos"], inv_freq=s["freq"], interleaved=True, factor=s["factor"], eps=EPS)
    leaves = [t.clone().requires_grad_() for t in (*s["x"], *s["gain"])]
    q, k = ex.norm_rotary(*leaves, **how)
    # An expanded gradient, and one at an odd stride.
    one = torch.tensor(0.5, dtype=torch.bfloat16, device=DEV).expand(q.shape)
    odd = torch.empty(2, 2, 65, 65, dtype=torch.bfloat16, device=DEV)[..., :64].copy_(s["dy"][1])
    got = torch.autograd.grad((q, k), leaves, (one, odd))
    want = ex.norm_rotary_backward(one.contiguous(), odd.contiguous(), *s["x"], *s["gain"], **how)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # Only what is wanted.
    leaf = s["gain"][0].clone().requires_grad_()
    y = ex.norm_rotary(s["x"][0], None, leaf, None, **how)
    assert torch.equal(torch.autograd.grad(y, leaf, s["dy"][0])[0],
                       ex.norm_rotary_backward(s["dy"][0], None, s["x"][0], None, leaf.detach(), None, **how)[2])
    with pytest.raises(RuntimeError):
        g, = torch.autograd.grad(ex.norm_rotary(s["x"][0], None, leaf, None, **how), leaf, s["dy"][0].clone().requires_grad_(), create_graph=True)
        g.sum().backward()


def test_gradient_against_differences():
    """<dx, v> against (L(x + t v) - L(x - t v)) / 2 t of the definition in 64 bits: the
    difference's own error is t^2 of third derivatives, 1e-8 here; dx's by its bound."""
    import exact_attention_67_gb300 as ex
    s = case(1, 9, 2, 1, 64, 64, False, torch.float16, torch.float32, "bhnd", 3)
    grads = ex.norm_rotary_backward(s["dy"][0], None, s["x"][0], None, s["gain"][0], None, s["pos"], s["freq"], factor=s["factor"], eps=EPS)
    x, dy, gain = f64(s["x"][0]), f64(s["dy"][0]), f64(s["gain"][0])
    want, unit, want_g, unit_g = normed_grad(dy, x, gain, s["p"], *s["args"])

    def loss(x, gain):
        return np.sum(dy * normed(x, gain, s["p"], *s["args"])[0])

    rng = np.random.default_rng(0)
    for _ in range(4):
        v, w = rng.standard_normal(x.shape) * np.std(x, -1, keepdims=True), rng.standard_normal(gain.shape)
        t = 1e-4
        slope = (loss(x + t * v, gain) - loss(x - t * v, gain)) / (2 * t)
        bound = np.sum((2.0 ** -11 * np.abs(want) + 2.0 ** -16 * unit + 2.0 ** -25) * np.abs(v))
        assert abs(np.sum(f64(grads[0]) * v) - slope) <= bound + 1e-6 * np.sum(np.abs(want * v))
        slope = (loss(x, gain + t * w) - loss(x, gain - t * w)) / (2 * t)
        assert abs(np.sum(f64(grads[2]) * w) - slope) <= np.sum((2.0 ** -13 * unit_g) * np.abs(w)) + 1e-6 * np.sum(np.abs(want_g * w))


def test_on_another_stream_and_captured():
    import exact_attention_67_gb300 as ex
    s = case(1, 300, 4, 2, 128, 128, False, torch.bfloat16, torch.bfloat16, "bhnd", 3)
    how = dict(positions=s["pos"], inv_freq=s["freq"], factor=s["factor"], eps=EPS)
    want, want_grad = ex.norm_rotary(*s["x"], *s["gain"], **how), ex.norm_rotary_backward(*s["dy"], *s["x"], *s["gain"], **how)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, grad = ex.norm_rotary(*s["x"], *s["gain"], stream=side, **how), ex.norm_rotary_backward(*s["dy"], *s["x"], *s["gain"], stream=side, **how)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*got, *grad), (*want, *want_grad)))
    # A whole step, forward and backward, captured, replayed on other inputs.
    x = [torch.zeros_like(t).requires_grad_() for t in s["x"]]
    gain = [torch.ones_like(t).requires_grad_() for t in s["gain"]]
    dy = [torch.zeros_like(t) for t in s["dy"]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ex.norm_rotary(*x, *gain, **how)
        grads = torch.autograd.grad(out, (*x, *gain), dy)
    with torch.no_grad():
        for a, b in zip((*x, *gain, *dy), (*s["x"], *s["gain"], *s["dy"])):
            a.copy_(b)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip((*out, *grads), (*want, *want_grad)))


# ---------------------------------------------------------------- into the cache
@pytest.mark.parametrize("d,rot,interleaved,page,dtype,even", [
    (128, 128, False, 16, torch.bfloat16, False), (64, 20, True, 8, torch.float16, False), (128, 6, False, 32, torch.bfloat16, True),
    (64, 0, False, 16, torch.float16, False), (128, 0, False, 1024, torch.bfloat16, True)])
def test_append_with_norms(d, rot, interleaved, page, dtype, even):
    import exact_attention_67_gb300 as ex
    Hq, Hk, B = 6, 2, 5
    new = [7] * B if even else [1, 0, 30, 4, 9]
    lens = [n + o for n, o in zip(new, (0, 3, 100, 21, 15))]
    width = max(-(-m // page) for m in lens)
    g = torch.Generator().manual_seed(3)
    table = torch.randperm(B * width, generator=g).view(B, width).to(torch.int32).to(DEV)
    total = sum(new) + (0 if even else 2)  # and two rows of no sequence
    q, k, v = (rows(1, total, H, d, dtype, "bnhd", i)[0].transpose(0, 1) for i, H in enumerate((Hq, Hk, Hk)))
    kc, vc = (torch.full((B * width, Hk, page, d), 7.0, dtype=dtype, device=DEV) for _ in range(2))
    qg, kg = gain_of(d, torch.float32, 1), gain_of(d, torch.float32, 2)
    freq, factor = ex.rotary_frequencies(rot, linear=2.0) if rot else (None, 1.0)
    cu = None if even else torch.tensor(np.cumsum([0] + new), dtype=torch.int32, device=DEV)
    q_out = torch.full_like(q, 3.0)
    ex.attn_cache_append(k, v, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device=DEV), cu, q=q, q_out=q_out, inv_freq=freq,
                         interleaved=interleaved, factor=factor, q_gain=qg, k_gain=kg, eps=EPS)
    at = np.concatenate([np.arange(m - n, m) for n, m in zip(new, lens)])
    seq = np.repeat(np.arange(B), new)
    fr = f64(freq) if rot else np.zeros(0)
    n = sum(new)
    check(q_out[:n], *normed(f64(q)[:n], f64(qg), at[:, None], fr, factor, interleaved), dtype)
    assert (q_out[n:] == 3.0).all()
    pages, off = table.cpu().numpy()[seq, at // page], at % page
    check(kc[pages, :, off], *normed(f64(k)[:n], f64(kg), at[:, None], fr, factor, interleaved), dtype)
    assert torch.equal(vc[pages, :, off], v[:n])
    untouched = torch.ones(B * width, page, dtype=torch.bool)
    untouched[pages, off] = False
    assert (kc.transpose(1, 2).cpu()[untouched] == 7.0).all() and (vc.transpose(1, 2).cpu()[untouched] == 7.0).all()


def test_append_in_place_and_without_q():
    import exact_attention_67_gb300 as ex
    cache = ex.PagedCache(16, 16, 2, 2, 64, dtype=torch.float16)
    seqs = [cache.add(), cache.add()]
    step = cache.extend(seqs, [20, 3])
    q, k, v = (rows(1, 23, H, 64, torch.float16, "bnhd", i)[0].transpose(0, 1) for i, H in enumerate((4, 2, 2)))
    g, freq = gain_of(64, torch.float16, 1), ex.rotary_frequencies(64)[0]
    out = torch.empty_like(q)
    cache.append(0, step, k, v, q, out, freq, q_gain=g, k_gain=g, eps=EPS)
    cache.append(1, step, k, v, inv_freq=freq, k_gain=g, eps=EPS)
    p = cache.pages(seqs[0])[0]  # full of the first sequence's rows
    assert torch.equal(cache.k_cache(0)[p], cache.k_cache(1)[p]) and torch.equal(cache.v_cache(0)[p], cache.v_cache(1)[p])
    cache.append(1, step, k, v, q, q, freq, q_gain=g, k_gain=g, eps=EPS)
    assert torch.equal(q, out)
    # The same numbers as the norm alone, at the positions of the step.
    pos = torch.tensor([*range(20), *range(3)], dtype=torch.int32, device=DEV)
    assert torch.equal(cache.k_cache(0)[p, :, :16].transpose(0, 1), ex.norm_rotary(k, None, g, None, pos, freq, eps=EPS)[:16])


def test_refusals():
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import ExattnError
    x, g = rows(1, 8, 2, 64, torch.bfloat16, "bhnd", 1), gain_of(64, torch.float32, 1)
    pos, freq = torch.arange(8, dtype=torch.int32, device=DEV), ex.rotary_frequencies(64)[0]
    for bad in (g[:32], g.view(1, 64), g.repeat(2)[::2], g.cpu()):
        with pytest.raises(ValueError):
            ex.norm_rotary(x, None, bad, None, pos, freq)
    with pytest.raises(TypeError):
        ex.norm_rotary(x, None, g.double(), None, pos, freq)
    with pytest.raises(ValueError, match="one type"):
        ex.norm_rotary(x, x, g, g.half(), pos, freq)
    with pytest.raises(ExattnError, match="VALUE"):
        ex.norm_rotary(x, None, g, None, pos, freq, eps=-1.0)
    with pytest.raises(ExattnError, match="ALIGN"):
        ex.norm_rotary(torch.empty(1032, dtype=torch.bfloat16, device=DEV)[4:1028].view(1, 2, 8, 64), None, g, None, pos, freq)
    with pytest.raises(ValueError):
        ex.norm_rotary_backward(x, None, x, x, g, g, pos, freq)
    with pytest.raises(ValueError):
        ex.norm_rotary_backward(x[:, :1], None, x, None, g, None, pos, freq)
    k = x[0].transpose(0, 1)
    kc = torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16, device=DEV)
    tables = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.full((1,), 8, dtype=torch.int32, device=DEV)
    for how in (dict(q_gain=g), dict(k_gain=g, q_gain=g), dict(q=k, q_out=k, k_gain=g), dict(q=k, q_out=k, q_gain=g), dict(q=k, q_out=k)):
        with pytest.raises(ValueError):
            ex.attn_cache_append(k, k, kc, kc.clone(), *tables, **how)


# ---------------------------------------------------------------- rows whose squares leave fp32
def far_rows(H, N, d, exponents, dtype, seed):
    """[1, H, N, d], row n of a size of 2^exponents[n % len]; the last row of every head has one large element."""
    g = torch.Generator().manual_seed(seed)
    at = torch.tensor([exponents[n % len(exponents)] for n in range(N)], dtype=torch.float64)
    x = torch.randn(1, H, N, d, generator=g, dtype=torch.float64).clamp(-3.5, 3.5) * torch.exp2(at)[:, None]
    x[:, :, -1, d // 3] = 2.0 ** max(exponents)
    return x.to(dtype).to(DEV)


def tight(got, want, size, dtype, unit):
    """As check, down to half of the type's smallest step: scaling by powers of two is exact, so the bounds are the same."""
    err, least = np.abs(f64(got) - want), 2.0 ** -134 if dtype == torch.bfloat16 else 2.0 ** -25
    bound = HALF[dtype] * np.abs(want) + unit * size + least * (1 + 2.0 ** -10)
    assert np.all(err <= bound), f"{np.argwhere(~(err <= bound))[:3]}: {f64(got)[~(err <= bound)][:3]} for {want[~(err <= bound)][:3]}"


@pytest.mark.parametrize("eps", [0.0, 1e-30, EPS, 1e30])
@pytest.mark.parametrize("d,rot,interleaved", [(128, 128, False), (64, 32, True), (64, 20, False), (128, 6, True)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_rows_whose_squares_leave_fp32(dtype, d, rot, interleaved, eps):
    """The definition holds for every finite row of the type, with a small or no eps too."""
    import exact_attention_67_gb300 as ex
    exponents = [-131, -120, -70, -63, -31, 0, 31, 33, 62, 70, 126] if dtype == torch.bfloat16 else [-24, -14, 0, 12]
    N, Hq, Hk = 3 * len(exponents) + 1, 3, 2
    x = [far_rows(H, N, d, exponents, dtype, i) for i, H in enumerate((Hq, Hk))]
    down = [-20 if e < -100 else -14 if dtype == torch.float16 else 0 for e in exponents]
    dy = [far_rows(H, N, d, down, dtype, 7 + i) for i, H in enumerate((Hq, Hk))]
    gain = [gain_of(d, torch.float32, 5 + i) for i in range(2)]
    pos, (freq, factor) = torch.arange(N, dtype=torch.int32, device=DEV), ex.rotary_frequencies(rot, yarn=8.0)
    args = (np.arange(N)[None, None], f64(freq), factor, interleaved, eps)
    how = dict(positions=pos, inv_freq=freq, interleaved=interleaved, factor=factor, eps=eps)
    for out, t, g in zip(ex.norm_rotary(*x, *gain, **how), x, gain):
        tight(out, *normed(f64(t), f64(g), *args), dtype, 2.0 ** -18)
    grads = ex.norm_rotary_backward(*dy, *x, *gain, **how)
    for i in range(2):
        dx, dx_size, dg, dg_size = normed_grad(f64(dy[i]), f64(x[i]), f64(gain[i]), *args)
        if dtype == torch.bfloat16 or eps > 0:
            tight(grads[i], dx, dx_size, dtype, 2.0 ** -16)
        check(grads[2 + i], dg, dg_size, torch.float32, 2.0 ** -14 + 2.0 ** -18)


def test_far_rows_into_the_cache():
    import exact_attention_67_gb300 as ex
    cache, exponents = ex.PagedCache(8, 16, 1, 2, 64), [-131, -70, 0, 70, 126]
    seq = cache.add()
    step = cache.extend([seq], 20)
    q, k, v = (far_rows(H, 20, 64, exponents, torch.bfloat16, i)[0].transpose(0, 1).contiguous() for i, H in enumerate((4, 2, 2)))
    g, freq = gain_of(64, torch.bfloat16, 1), ex.rotary_frequencies(64)[0]
    cache.append(0, step, k, v, q, q_out := torch.empty_like(q), freq, q_gain=g, k_gain=g, eps=0.0)
    args = (np.arange(20)[:, None], f64(freq), 1.0, False, 0.0)
    tight(q_out, *normed(f64(q), f64(g), *args), torch.bfloat16, 2.0 ** -18)
    stored = cache.k_cache(0)[list(cache.pages(seq))].transpose(1, 2).reshape(-1, 2, 64)[:20]
    tight(stored, *normed(f64(k), f64(g), *args), torch.bfloat16, 2.0 ** -18)
    assert torch.equal(cache.v_cache(0)[list(cache.pages(seq))].transpose(1, 2).reshape(-1, 2, 64)[:20], v)


def test_far_rows_of_zeros_nan_and_infinities():
    """Beside rows that need no scale: what is not finite stays in its row, and zeros are zeros with any eps above 0."""
    import exact_attention_67_gb300 as ex
    x = far_rows(1, 6, 128, [0], torch.bfloat16, 1)
    x[0, 0, 0] = 0
    x[0, 0, 1] *= 2.0 ** 70
    x[0, 0, 1, 5] = float("nan")
    x[0, 0, 2] *= 2.0 ** -70
    x[0, 0, 2, 7] = float("inf")
    for eps in (1e-40, 1e-30, 1e-6):
        y = ex.norm_rotary(x, eps=eps)
        assert not y[0, 0, 0].any() and y[0, 0, 1].isnan().all() and not y[0, 0, 3:].isnan().any()
        assert y[0, 0, 2].isnan().sum() == 2  # the infinity's pair
        dx = ex.norm_rotary_backward(x, None, x, None, None, None, eps=eps)[0]
        assert not dx[0, 0, 0].any() and dx[0, 0, 1].isnan().all() and not dx[0, 0, 3:].isnan().any()
