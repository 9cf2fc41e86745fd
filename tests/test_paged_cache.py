"""The paged cache's host side (tables, reference counts, copy before write,
compaction) against a model that keeps every sequence's tokens, on the CPU: the
page copies are done by indexing.  And the refusals of the cache calls, which are
made before any launch."""
import ctypes
import random

import pytest
import torch

from exact_attention_67_gb300 import OutOfPages, PagedCache, rotary_frequencies


class HostCache(PagedCache):
    """A cache in host memory whose tokens are written and read by indexing."""

    def _copy(self, src, dst, stream):
        assert len(src) == len(set(dst)) == len(dst) and not set(src) & set(dst)
        self.pool[:, dst] = self.pool[:, src].clone()

    def write(self, step, values):
        t = 0
        for row, n, length in zip(step.page_table.tolist(), step.new, step.seqlens.tolist()):
            for p in range(length - n, length):
                self.pool[:, row[p // self.page_size], :, p % self.page_size] = float(values[t])
                t += 1

    def read(self, seq):
        rows = [self.pool[:, p] for p in self.pages(seq)]
        if not rows:
            return []
        got = torch.cat(rows, 2)[:, :, : self.length(seq)]
        assert bool((got == got[:1, :1, :, :1]).all())
        return got[0, 0, :, 0].tolist()


def consistent(cache):
    held = [0] * cache.num_pages
    for pages in cache._pages.values():
        assert len(set(pages)) == len(pages)
        for p in pages:
            held[p] += 1
    assert held == cache._refs
    assert sorted(cache._free) == [p for p in range(cache.num_pages) if held[p] == 0]
    for s, pages in cache._pages.items():
        assert len(pages) == -(-cache._length[s] // cache.page_size)


@pytest.mark.parametrize("seed", range(6))
def test_random_lives_of_sequences(seed):
    r = random.Random(seed)
    cache = HostCache(40, 8, 1, 1, 64, torch.float16, device="cpu")
    tokens = {}
    for _ in range(120):
        op = r.random()
        if op < 0.2 or not tokens:
            tokens[cache.add()] = []
        elif op < 0.35:
            s = r.choice(list(tokens))
            for f in cache.fork(s, r.randint(1, 3)):
                tokens[f] = list(tokens[s])
        elif op < 0.5:
            for s in r.sample(list(tokens), min(len(tokens), r.randint(1, 2))):
                cache.free(s)
                del tokens[s]
        elif op < 0.6:
            s = r.choice(list(tokens))
            n = r.randint(0, len(tokens[s]))
            cache.truncate(s, n)
            del tokens[s][n:]
        elif op < 0.7:
            used = cache.num_pages - cache.free_pages
            cache.compact()
            assert all(p < used for pages in cache._pages.values() for p in pages)
        else:
            seqs = r.sample(list(tokens), r.randint(1, min(len(tokens), 4)))
            new = [r.choice([0, 1, 1, 3, 8, 17]) for _ in seqs]
            before = {s: cache.pages(s) for s in tokens}
            try:
                step = cache.extend(seqs, new)
            except OutOfPages:
                assert before == {s: cache.pages(s) for s in tokens}
            else:
                values = [r.randrange(1000) for _ in range(sum(new))]
                cache.write(step, values)
                at = 0
                for s, n in zip(seqs, new):
                    tokens[s] += values[at: at + n]
                    at += n
                assert (step.cu_seqlens is None) == (len(set(new)) == 1 and new[0] > 0)
        consistent(cache)
        for s, want in tokens.items():
            assert cache.read(s) == want  # whole numbers below 2048 are exact in f16


def test_shared_last_page_is_copied_for_all_writers_but_one():
    cache = HostCache(16, 8, 2, 1, 64, device="cpu")
    s = cache.add()
    cache.extend([s], 12)
    a, b = cache.fork(s, 2)
    before = cache.free_pages
    cache.extend([s, a, b], 1)                    # three holders of the half-full page: two copies
    assert before - cache.free_pages == 2
    assert len({cache.pages(x)[1] for x in (s, a, b)}) == 3 and len({cache.pages(x)[0] for x in (s, a, b)}) == 1
    cache.free([a, b])
    assert cache.free_pages == before
    cache.extend([s], 0)
    assert cache.length(s) == 13
    with pytest.raises(OutOfPages):
        cache.extend([s], 16 * 8)
    assert cache.length(s) == 13 and cache.free_pages == before


def test_a_copy_that_fails_changes_nothing():
    class Failing(HostCache):
        def _copy(self, src, dst, stream):
            raise RuntimeError("no")

    cache = Failing(16, 8, 1, 1, 64, device="cpu")
    s = cache.add()
    cache.extend([s], 12)
    f, = cache.fork(s)
    state = (cache.pages(s), cache.pages(f), cache.length(f), cache.free_pages)
    with pytest.raises(RuntimeError):
        cache.extend([f], 20)
    assert state == (cache.pages(s), cache.pages(f), cache.length(f), cache.free_pages)
    consistent(cache)


def test_cache_refusals():
    for bad in (dict(page_size=12), dict(page_size=4), dict(num_pages=0), dict(head_dim=96), dict(dtype=torch.float32)):
        with pytest.raises(ValueError):
            PagedCache(**{**dict(num_pages=4, page_size=8, layers=1, kv_heads=1, head_dim=64, device="cpu"), **bad})
    cache = HostCache(4, 8, 1, 1, 64, device="cpu")
    s = cache.add()
    for call in (lambda: cache.extend([s, s], 1), lambda: cache.extend([7], 1), lambda: cache.free(9), lambda: cache.fork(3)):
        with pytest.raises(KeyError):
            call()
    for call in (lambda: cache.extend([], 1), lambda: cache.extend([s], [1, 2]), lambda: cache.extend([s], -1),
                 lambda: cache.truncate(s, 1)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(IndexError):
        cache.k_cache(1)


# ---------------------------------------------------------------- the C calls, before any launch
P = [0x100000 * (i + 1) for i in range(16)]  # fake addresses, never read


@pytest.fixture(scope="module")
def lib():
    from exact_attention_67_gb300 import _lib
    from exact_attention_67_gb300 import build as b
    b.build()
    return _lib.load()


def test_rotary_validation(lib):
    from exact_attention_67_gb300._lib import Strides
    s = Strides(2 * 8 * 64, 8 * 64, 64)

    def call(dt=0, q=P[0], qo=P[1], k=P[2], ko=P[3], pos=P[4], freq=P[5], rot=64, factor=1.0, Hq=2, Hk=2, N=8, d=64, sq=s,
             ps=0):
        return lib.attn_rotary(dt, q, sq, qo, s, Hq, k, s, ko, s, Hk, pos, ps, freq, rot, 0, 0, factor, 1, N, d, None)

    assert call(q=None) == call(qo=None) == call(pos=None) == call(freq=None) == call(k=None) == 1
    assert call(Hq=0) == call(N=0) == call(Hk=-1) == call(ps=-1) == 2
    assert call(q=P[0] + 8) == call(pos=P[4] + 2) == call(freq=P[5] + 4) == call(sq=Strides(0, 8 * 64, 60)) == 3
    assert call(dt=5) == call(d=80) == call(rot=0) == call(rot=66) == call(rot=7) == 4
    assert call(factor=0.0) == call(factor=float("nan")) == call(factor=float("inf")) == 9


def test_append_and_attention_validation(lib):
    from exact_attention_67_gb300._lib import Strides
    t, c = Strides(0, 64, 2 * 64), Strides(2 * 16 * 64, 16 * 64, 64)

    def append(q=P[0], k=P[2], kc=P[4], table=P[6], lens=P[7], freq=P[9], Hq=2, Hk=2, ps=16, pages=9, row=4, width=4, B=3,
               total=6, d=64, rot=64, cu=P[8], skc=c, factor=1.0):
        return lib.attn_cache_append(0, q, t, P[1], t, Hq, k, t, P[3], t, kc, skc, P[5], c, Hk, pages, ps, table, row, width,
                                     lens, cu, B, total, d, freq, rot, 0, factor, None)

    assert append(k=None) == append(kc=None) == append(table=None) == append(lens=None) == append(freq=None) == 1
    assert append(q=None) == 1
    assert append(Hk=0) == append(pages=0) == append(width=0) == append(row=3) == append(B=0) == append(total=0) == 2
    assert append(total=7, cu=None) == 2                       # 7 tokens over 3 sequences
    assert append(ps=12) == append(ps=4) == append(ps=2048) == append(d=32) == append(rot=3) == 4
    assert append(kc=P[4] + 8) == append(table=P[6] + 1) == append(skc=Strides(2048, 1024, 63)) == 3
    assert append(skc=Strides(0, 0, 63)) == 2                  # pages on top of one another
    assert append(factor=-1.0) == 9

    size = lib.attn_fwd_paged_workspace_size

    def attend(q=P[0], kc=P[2], o=P[4], lse=P[5], table=P[6], lens=P[7], cu=P[8], ps=16, pages=9, B=3, Hq=4, Hk=2, total=6,
               mq=4, mk=60, d=64, window=0, scale=0.1, ws=P[9], wsb=1 << 30, dt=0, so=Strides(0, 64, 256)):
        q4 = Strides(0, 64, 256)
        return lib.attn_fwd_paged(dt, q, q4, kc, c, P[3], c, o, so, lse, pages, ps, table, 4, 4, lens, cu, B, Hq, Hk, total, mq,
                                  mk, d, 1, window, scale, ws, wsb, None)

    assert attend(q=None) == attend(kc=None) == attend(o=None) == attend(lse=None) == attend(table=None) == 1
    assert attend(lens=None) == 1
    assert attend(Hq=5) == attend(Hq=1) == attend(total=0) == attend(mq=0) == attend(mk=0) == attend(mk=1 << 30) == 2
    assert attend(dt=3) == attend(d=96) == attend(ps=24) == attend(Hq=258, Hk=2) == 4
    assert attend(lse=P[5] + 2) == attend(o=P[4] + 8) == attend(so=Strides(0, 64, 100)) == attend(ws=P[9] + 8) == 3
    assert attend(window=-1) == attend(scale=0.0) == attend(scale=float("nan")) == 9
    need = size(3, 4, 2, 6, 4, 60, 64)
    assert need > 0 and attend(ws=None) == attend(wsb=need - 1) == 6
    assert size(3, 5, 2, 6, 4, 60, 64) == size(3, 4, 2, 6, 4, 60, 80) == size(0, 4, 2, 6, 4, 60, 64) == 0


def test_copy_validation(lib):
    def copy(src, dst, pool=P[0], slab=1 << 20, page=1 << 12, size=1 << 12, slabs=2, pages=256):
        n = len(src)
        a, b = (ctypes.c_int * max(n, 1))(*src), (ctypes.c_int * max(n, 1))(*dst)
        return lib.attn_cache_copy(pool, slab, page, size, slabs, pages, a, b, n, None)

    assert copy([], []) == 0
    assert copy([1], [2], pool=None) == 1
    assert copy([1], [256]) == copy([-1], [2]) == copy([1, 2], [3, 3]) == copy([1, 2], [2, 3]) == copy([5], [5]) == 9
    many = list(range(100))
    assert copy(many, [100 + i for i in many[:-1]] + [100]) == copy(many, [100 + i for i in many[:-1]] + [50]) == 9
    assert copy([1], [2], pool=P[0] + 8) == copy([1], [2], size=4090, page=4096) == copy([1], [2], page=(1 << 12) + 8) == 3
    assert copy([1], [2], slabs=0) == copy([1], [2], pages=0) == copy([1], [2], page=1 << 11) == 2
    assert copy([1], [2], slab=1 << 12) == 2     # slabs on top of one another


def test_frequencies():
    f, m = rotary_frequencies(8, base=100.0, device="cpu")
    assert m == 1.0 and torch.allclose(f, torch.tensor([1.0, 100 ** -0.25, 0.1, 100 ** -0.75], dtype=torch.float64))
    g, m = rotary_frequencies(8, base=100.0, linear=4.0, device="cpu")
    assert m == 1.0 and torch.equal(g, f / 4)
    g, m = rotary_frequencies(64, yarn=8.0, trained_length=4096, device="cpu")
    f, _ = rotary_frequencies(64, device="cpu")
    assert abs(m - (0.1 * 2.0794415416798357 + 1)) < 1e-15
    assert g[0] == f[0] and torch.isclose(g[-1], f[-1] / 8) and bool((g <= f).all()) and bool((g >= f / 8 * (1 - 1e-15)).all())
    for bad in (dict(rot_dim=7), dict(rot_dim=0), dict(base=0.0), dict(linear=2.0, yarn=2.0), dict(yarn=-1.0),
                dict(slow_turns=3.0, fast_turns=3.0)):
        with pytest.raises(ValueError):
            rotary_frequencies(**{**dict(rot_dim=8, device="cpu"), **bad})


def test_host_tensors_are_refused():
    import exact_attention_67_gb300 as ex
    q, kc = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.full((2,), 5, dtype=torch.int32)
    freq, _ = rotary_frequencies(64, device="cpu")
    for call in (lambda: ex.forward_paged(q, kc, kc, table, lens), lambda: ex.rotary(q, None, lens, freq),
                 lambda: ex.attn_cache_append(q[:, :2], q[:, :2], kc, kc, table, lens),
                 lambda: ex.attn_cache_copy(kc[None], [0], [1])):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("new", [1, [2, 3, 0]])
def test_other_counts_of_tokens_are_refused(monkeypatch, new):
    """append and attend take the rows that their step has made room for, and with
    offsets padding behind them."""
    from exact_attention_67_gb300 import cache as module
    made = []
    monkeypatch.setattr(module, "attn_cache_append", lambda k, *a: made.append(k.shape[0]))
    monkeypatch.setattr(module, "forward_paged", lambda q, *a: made.append(q.shape[0]))
    cache = HostCache(16, 8, 1, 2, 64, device="cpu")
    step = cache.extend([cache.add() for _ in range(3)], new)
    n = step.tokens
    assert n == (3 if new == 1 else 5)
    rows = lambda count, heads=2: torch.zeros(count, heads, 64, dtype=torch.bfloat16)  # noqa: E731
    for count in (n - 1, 0) + ((2 * n, n + 1) if new == 1 else ()):
        with pytest.raises(ValueError, match="new tokens"):
            cache.append(0, step, rows(count), rows(count))
        with pytest.raises(ValueError, match="new tokens"):
            cache.attend(0, step, rows(count, 4))
    with pytest.raises(ValueError, match="new tokens"):
        cache.attend(0, step, rows(n, 4)[None])
    assert made == []
    cache.append(0, step, rows(n), rows(n))
    cache.attend(0, step, rows(n, 4))
    assert made == [n, n]
    if new != 1:
        cache.append(0, step, rows(n + 3), rows(n + 3))
        cache.attend(0, step, rows(n + 3, 4))
        assert made[2:] == [n + 3, n + 3]


def test_pools_of_impossible_extent_are_refused(lib):
    """Page counts and strides whose product passes 64 bits."""
    one = (ctypes.c_int * 1)(1), (ctypes.c_int * 1)(2)
    for pages, stride in ((2 ** 31 - 1, 1 << 34), (2 ** 31 - 1, 1 << 39), (1 << 30, (1 << 34) + 16)):
        assert lib.attn_cache_copy(P[0], 1 << 43, stride, 4096, 4, pages, *one, 1, None) == 2
