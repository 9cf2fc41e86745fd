"""Appending tokens to a paged cache and copying its pages: values against the
definition in 64 bits with the bound of test_rotary_gpu.py, and everything that
a call must not touch, bit for bit."""
import numpy as np
import pytest
import torch

from tests.test_rotary_gpu import check, f64, turned

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_67_gb300 import build
    build.build()


def randn(*shape, seed, dtype):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)


CASES = [
    # (new tokens, lengths, Hq, Hk, d, page size, rot (0: none), interleaved, dtype, token-major cache)
    ([1], [1], 1, 1, 64, 16, 64, False, torch.bfloat16, False),
    ([1] * 9, [1, 16, 17, 300, 5, 64, 128, 33, 2], 8, 2, 128, 16, 128, False, torch.bfloat16, False),
    ([7, 0, 130, 1, 64], [7, 40, 200, 9, 64], 3, 3, 64, 32, 32, True, torch.float16, True),
    ([5, 3], [2, 3], 2, 1, 128, 8, 6, False, torch.bfloat16, False),   # more new tokens than length: positions below 0
    ([600, 500], [70000, 500], 4, 4, 128, 128, 20, True, torch.bfloat16, False),
    ([40, 40], [41, 99], 0, 2, 64, 64, 0, False, torch.float16, True),
    ([4001, 3000, 1, 3002], [4001, 5000, 9, 3100], 3, 1, 64, 64, 64, False, torch.bfloat16, False),  # eight tokens a block
]


@pytest.mark.parametrize("new,lens,Hq,Hk,d,ps,rot,interleaved,dtype,token_major", CASES, ids=lambda x: str(x)[:40])
def test_append(new, lens, Hq, Hk, d, ps, rot, interleaved, dtype, token_major):
    import exact_attention_67_gb300 as ex
    B, pad = len(new), 3
    total = sum(new) + pad  # rows behind the last sequence stay as they are
    need = [-(-n // ps) for n in lens]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(4)).tolist()
    table = torch.full((B, max(need) + 1), -1, dtype=torch.int32)
    for b in range(B):
        for i in range(need[b]):
            table[b, i] = order.pop()
    if token_major:
        kc, vc = (randn(pages, ps, Hk, d, seed=s, dtype=dtype).transpose(1, 2) for s in (1, 2))
    else:
        kc, vc = (randn(pages, Hk, ps, d, seed=s, dtype=dtype) for s in (1, 2))
    kc0, vc0 = f64(kc), f64(vc)
    k, v = randn(total, Hk, d, seed=5, dtype=dtype), randn(total, Hk, d, seed=6, dtype=dtype)
    q = randn(total, Hq, d, seed=7, dtype=dtype) if Hq else None
    qo = torch.full_like(q, 7.0) if Hq else None
    freq, factor = ex.rotary_frequencies(rot, yarn=4.0) if rot else (None, 1.0)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    ex.attn_cache_append(k, v, kc, vc, table.to(DEV), seq, cu, q, qo, freq, interleaved, factor)
    torch.cuda.synchronize()
    pos = np.concatenate([lens[b] - new[b] + np.arange(new[b]) for b in range(B)])
    fr = freq.cpu().numpy() if rot else np.zeros(0)

    def turn(x):  # [tokens, H, d]
        y, s = turned(f64(x)[: total - pad].transpose(1, 0, 2), pos, fr, factor, interleaved)
        return y.transpose(1, 0, 2), s.transpose(1, 0, 2)

    if Hq:
        check(qo[: total - pad], *turn(q), dtype)
        assert torch.all(qo[total - pad:] == 7.0)
    ky, ks = turn(k)
    size = np.zeros_like(kc0)
    t = 0
    for b in range(B):
        for i in range(new[b]):
            p = pos[t]
            if p >= 0:
                page, row = int(table[b, p // ps]), p % ps
                kc0[page, :, row], size[page, :, row] = ky[t], ks[t]
                vc0[page, :, row] = f64(v[t])
            t += 1
    touched = size.sum((1, 3)) > 0
    check(kc, kc0, size, dtype)
    got = f64(kc)
    keep = ~np.broadcast_to(touched[:, None, :, None], got.shape)
    assert np.array_equal(got[keep], kc0[keep]) and np.array_equal(f64(vc), vc0)


def test_append_without_offsets_and_bad_tables():
    """The same tokens with and without cu_seqlens; page numbers outside the
    pool, positions past the table and offsets past the tensors store nothing."""
    import exact_attention_67_gb300 as ex
    B, ps, H, d, pages = 3, 16, 2, 64, 6
    k, v = randn(B * 2, H, d, seed=1, dtype=torch.bfloat16), randn(B * 2, H, d, seed=2, dtype=torch.bfloat16)
    table = torch.tensor([[0, 1], [2, 3], [4, 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([17, 2, 32], dtype=torch.int32, device=DEV)
    caches = [[torch.zeros(pages, H, ps, d, dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(3)]
    ex.attn_cache_append(k, v, *caches[0], table, lens)
    ex.attn_cache_append(k, v, *caches[1], table, lens, torch.tensor([0, 2, 4, 6], dtype=torch.int32, device=DEV))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    assert caches[0][0].any()
    bad = torch.tensor([[6, -1], [1 << 30, -(1 << 30)], [-5, 99]], dtype=torch.int32, device=DEV)
    ex.attn_cache_append(k, v, *caches[2], bad, lens)
    ex.attn_cache_append(k, v, *caches[2], table, lens + 40)       # past the table
    ex.attn_cache_append(k, v, *caches[2], table, lens - (1 << 30))
    ex.attn_cache_append(k, v, *caches[2], table, lens, torch.tensor([6, 9, 12, 90], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert not caches[2][0].any() and not caches[2][1].any()
    ex.attn_cache_append(k[:0], v[:0], *caches[2], table, lens)
    assert not caches[2][0].any()


@pytest.mark.parametrize("slabs,pages,block,n,dtype", [
    (1, 4, (1, 8, 64), 1, torch.bfloat16), (6, 70, (2, 16, 64), 33, torch.float16), (2, 5000, (1, 8, 64), 2300, torch.bfloat16),
    (3, 9, (5, 64, 128), 4, torch.bfloat16), (1, 3, (17, 256, 128), 1, torch.float16), (2, 6, (8,), 2, torch.float32),
])
def test_copy(slabs, pages, block, n, dtype):
    import exact_attention_67_gb300 as ex
    pool = randn(slabs, pages, *block, seed=n, dtype=dtype)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    src, dst = order[:n], order[n: 2 * n]
    want = pool.clone()
    want[:, dst.long().to(DEV)] = pool[:, src.long().to(DEV)]
    ex.attn_cache_copy(pool, src, dst.tolist())
    assert torch.equal(pool, want)


def test_copy_of_layouts_and_refusals():
    import exact_attention_67_gb300 as ex
    # Page-major storage: a page's slabs side by side; and a pool inside a wider tensor.
    store = randn(10, 3, 2, 16, 64, seed=1, dtype=torch.bfloat16)
    pool, want = store.transpose(0, 1), store.clone()
    ex.attn_cache_copy(pool, [1, 2, 9], [0, 5, 3])
    want[[0, 5, 3]] = want[[1, 2, 9]]
    assert torch.equal(store, want)
    wide = randn(2, 10, 4, 16, 64, seed=2, dtype=torch.bfloat16)
    want = wide.clone()
    ex.attn_cache_copy(wide[:, :, 1:3], [4], [7])
    want[:, 7, 1:3] = want[:, 4, 1:3]
    assert torch.equal(wide, want)
    for src, dst in (([0], [10]), ([-1], [2]), ([0, 1], [5, 5]), ([0, 1], [1, 2]), ([3], [3]),
                     (list(range(40)), list(range(40, 79)) + [40])):
        big = torch.zeros(1, 10 if len(src) < 5 else 200, 1, 8, 64, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(ex.ExattnError):
            ex.attn_cache_copy(big, src, dst)
    with pytest.raises(ValueError):
        ex.attn_cache_copy(pool, [1], [2, 3])
    with pytest.raises(ValueError):
        ex.attn_cache_copy(pool, torch.tensor([1], dtype=torch.int32, device=DEV), [2])
    with pytest.raises(ValueError):
        ex.attn_cache_copy(wide[:, :, :, ::2], [1], [2])  # a page with holes
    with pytest.raises(ex.ExattnError):
        ex.attn_cache_copy(wide[:1].expand(2, -1, -1, -1, -1), [1], [2])  # slabs on top of each other
    ex.attn_cache_copy(pool, [], [])


def test_a_captured_step():
    """Append and attention of one token a sequence, captured once and replayed as
    the sequences grow: the lengths and tables are read at the replay."""
    import exact_attention_67_gb300 as ex
    B, Hq, Hk, d, ps, width = 3, 8, 2, 64, 16, 12
    kc, vc = (torch.full((B * width, Hk, ps, d), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    table = torch.randperm(B * width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(B, width).to(DEV)
    lens = torch.tensor([0, 50, 14], dtype=torch.int32, device=DEV)
    first = lens.tolist()
    past = [randn(n, 2 * Hk, d, seed=30 + n, dtype=torch.bfloat16) for n in first]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(first)]), dtype=torch.int32, device=DEV)
    both = torch.cat(past)
    ex.attn_cache_append(both[:, :Hk], both[:, Hk:], kc, vc, table, lens, cu)
    q, k, v = (torch.zeros(B, h, d, dtype=torch.bfloat16, device=DEV) for h in (Hq, Hk, Hk))
    qo, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(Hq, B, device=DEV)
    freq, _ = ex.rotary_frequencies(d)
    ws = torch.empty(ex.attn_fwd_paged_workspace_size(B, Hq, Hk, B, 1, width * ps, d), dtype=torch.uint8, device=DEV)

    def step():
        lens.add_(1)
        ex.attn_cache_append(k, v, kc, vc, table, lens, None, q, qo, freq)
        ex.attn_fwd_paged(qo, kc, vc, o, lse, table, lens, None, 1, width * ps, True, d ** -0.5, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = [(p[:, :Hk].double(), p[:, Hk:].double()) for p in past]
    for i in range(40):
        for x, s in ((q, 100), (k, 200), (v, 300)):
            x.copy_(randn(*x.shape, seed=s + i, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        for b in range(B):
            p = first[b] + i
            mine = kc[table[b, p // ps], :, p % ps]
            want, size = turned(f64(k[b]), np.array([p]), freq.cpu().numpy(), 1.0, False)
            check(mine, want, size, torch.bfloat16)
            K, V = held[b]
            K, V = held[b] = torch.cat([K, mine[None].double()]), torch.cat([V, v[b][None].double()])
            x = torch.einsum("hgd,jhd->hgj", qo[b].double().view(Hk, Hq // Hk, d), K) * d ** -0.5
            w = torch.softmax(x, -1)
            out = torch.einsum("hgj,jhd->hgd", w, V).reshape(Hq, d)
            # The bound of test_paged_gpu.py.
            mass = torch.einsum("hgj,jhd->hgd", w, V.abs()).reshape(Hq, d)
            assert bool(((o[b].double() - out).abs() <= 2.0 ** -8 * out.abs() + (2.0 ** -10 + 2.0 ** -12) * mass + 2.0 ** -18).all())
    assert ex.device_error() == 0


def test_append_in_place_and_rows_before_the_first_sequence():
    """q_out may be q; rows before cu_seqlens[0] belong to no sequence, neither to the
    append nor to the attention after it."""
    import exact_attention_67_gb300 as ex
    new, lens, Hq, Hk, d, ps = [3, 1, 5], [40, 7, 5], 6, 2, 64, 16
    before, total = 4, 4 + 9
    q, k, v = (randn(total, h, d, seed=60 + i, dtype=torch.bfloat16) for i, h in enumerate((Hq, Hk, Hk)))
    pools = [randn(12, Hk, ps, d, seed=70 + i, dtype=torch.bfloat16) for i in range(2)]
    table = torch.arange(12, dtype=torch.int32, device=DEV).view(3, 4)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    freq, _ = ex.rotary_frequencies(d)
    offsets = np.concatenate([[0], np.cumsum(new)])
    kc, vc = (x.clone() for x in pools)
    qo = torch.empty_like(q[before:])
    cu = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    ex.attn_cache_append(k[before:], v[before:], kc, vc, table, seq, cu, q[before:], qo, freq)
    want = ex.forward_paged(qo, kc, vc, table, seq, cu, 5, 40)
    kc2, vc2 = (x.clone() for x in pools)
    q2, cu2 = q.clone(), cu + before
    ex.attn_cache_append(k, v, kc2, vc2, table, seq, cu2, q2, q2, freq)
    assert torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert torch.equal(q2[before:], qo) and torch.equal(q2[:before], q[:before])
    o, lse = torch.full_like(q2, 3.0), torch.full((Hq, total), 3.0, device=DEV)
    ws = torch.empty(ex.attn_fwd_paged_workspace_size(3, Hq, Hk, total, 5, 40, d), dtype=torch.uint8, device=DEV)
    ex.attn_fwd_paged(q2, kc2, vc2, o, lse, table, seq, cu2, 5, 40, True, d ** -0.5, ws)
    assert torch.equal(o[before:], want[0]) and torch.equal(lse[:, before:], want[1])
    assert torch.all(o[:before] == 3.0) and torch.all(lse[:, :before] == 3.0)
