"""Attention behind shared rows, without a GPU: what its C call refuses, its workspace,
and how PagedCache finds the groups."""
import pytest
import torch

P = [0x100000 + 0x100000 * i for i in range(16)]
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE, VALUE = 1, 2, 3, 4, 6, 9


@pytest.fixture(scope="module")
def lib():
    from exact_attention_67_gb300 import build as b
    b.build()
    from exact_attention_67_gb300 import _lib
    return _lib.load()


def call(lib, dtype=0, q=P[0], kc=P[1], vc=P[2], o=P[3], lse=P[4], table=P[5], lens=P[6], cu=None, groups_at=P[7], prefix=P[8], B=4, groups=2,
         Hq=8, Hk=2, total=4, mq=1, mk=1000, mg=2, d=64, scale=0.125, ws=P[9], ws_bytes=1 << 30, ps=16, sq=None):
    from exact_attention_67_gb300 import Strides
    s = Strides(0, 64, 512)
    c = Strides(2 * 16 * 64, 16 * 64, 64)
    return lib.attn_fwd_paged_shared(dtype, q, sq or s, kc, c, vc, c, o, s, lse, 100, ps, table, 64, 64, lens, cu, groups_at, prefix, B, groups,
                                     Hq, Hk, total, mq, mk, mg, d, 1, scale, ws, ws_bytes, None)


@pytest.mark.parametrize("how,status", [
    (dict(q=None), NULL), (dict(groups_at=None), NULL), (dict(prefix=None), NULL), (dict(table=None), NULL), (dict(lse=None), NULL),
    (dict(dtype=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(ps=24), UNSUPPORTED), (dict(Hq=9), SHAPE), (dict(groups=0), SHAPE),
    (dict(groups=-1), SHAPE), (dict(mg=0), SHAPE), (dict(mq=0), SHAPE), (dict(total=6), SHAPE), (dict(groups_at=P[7] + 2), ALIGN),
    (dict(prefix=P[8] + 1), ALIGN), (dict(q=P[0] + 8), ALIGN), (dict(scale=0.0), VALUE), (dict(scale=float("nan")), VALUE),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=1000), WORKSPACE), (dict(ws=P[9] + 8), ALIGN),
    (dict(mk=(1 << 30) - 1, Hk=8, B=1 << 20, total=1 << 20), SHAPE)])
def test_refusals(lib, how, status):
    assert call(lib, **how) == status


def test_workspace_size(lib):
    def size(B=4, groups=2, Hq=8, Hk=2, total=4, mq=1, mk=1000, mg=2, d=64):
        return lib.attn_fwd_paged_shared_workspace_size(B, groups, Hq, Hk, total, mq, mk, mg, d)
    n = size()
    assert n > 2 * 4 * 8 * (64 * 4 + 16) and call(lib, ws_bytes=n - 1) == WORKSPACE
    assert size(total=4000, B=4000) > n and size(mg=1 << 30) > 0
    for bad in (dict(groups=0), dict(mg=0), dict(B=0), dict(Hq=7), dict(d=32), dict(mk=0), dict(Hq=256, Hk=1)):
        assert size(**bad) == 0


def test_python_refusals():
    import exact_attention_67_gb300 as ex
    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ex.forward_paged_shared(q, c, c, torch.zeros(2, 2, dtype=torch.int32), i, i, i)


# ---------------------------------------------------------------- PagedCache
def cache_of(pages=200, ps=16, share_from=0):
    from exact_attention_67_gb300 import PagedCache
    return PagedCache(pages, ps, 1, 1, 64, device="cpu", share_from=share_from)


@pytest.fixture()
def no_copies(monkeypatch):
    from exact_attention_67_gb300 import cache
    monkeypatch.setattr(cache, "attn_cache_copy", lambda *a: None)


def groups(step):
    return None if step.cu_groups is None else (step.cu_groups.tolist(), step.prefix_lens.tolist(), step.max_group_q)


def test_groups_of_forks(no_copies):
    c = cache_of()
    a, b = c.add(), c.add()
    c.extend([a, b], [300, 200])
    fa, fb = c.fork(a, 3), c.fork(b, 2)
    # 300 rows: 18 whole pages (and a part that each copies before it writes), 256 in whole tiles.
    step = c.extend([*fa, b, *fb], 1, shared=True)
    assert groups(step) == ([0, 3, 6], [256] * 3 + [128] * 3, 3)
    assert c.extend([*fa, b, *fb], 0, shared=True).cu_groups.tolist() == [0, 3, 6]
    # Order matters: only neighbours are taken together.
    assert groups(c.extend([fa[0], fb[0], fa[1], fb[1]], 1, shared=True)) is None
    assert groups(c.extend([fa[0], fa[1]], [5, 2], shared=True)) == ([0, 2], [256, 256], 7)
    # Not asked for, and nothing shared.
    assert groups(c.extend([fa[0], fa[1]], 1)) is None
    d = c.add()
    c.extend([d], 256)
    assert groups(c.extend([a, d], 1, shared=True)) is None


def test_groups_take_in_what_saves_reads(no_copies):
    c = cache_of(2000)
    root = c.add()
    c.extend([root], 256)
    deep = c.fork(root, 1)[0]
    c.extend([deep], 1024 - 256)
    same = c.fork(deep, 3)
    # Four share 1024 rows; taking in the root's 256 would save 4 * 256 rows instead of 3 * 1024.
    assert groups(c.extend([deep, *same, root], 1, shared=True)) == ([0, 4, 5], [1024] * 4 + [0], 4)
    # One alone goes with whoever shares a tile.
    assert groups(c.extend([root, deep], 1, shared=True)) == ([0, 2], [256] * 2, 2)


def test_rows_that_new_tokens_stand_on_are_not_shared(no_copies):
    """A fork of an empty or short sequence, and new tokens that begin inside the common
    pages after a truncation: shared rows end before the first new token of each."""
    c = cache_of()
    a = c.add()
    c.extend([a], 400)
    f, g = c.fork(a, 2)
    c.truncate(f, 200)
    step = c.extend([f, g, a], 1, shared=True)
    n, p, m = groups(step)
    assert n == [0, 1, 3] and p == [0, 384, 384] or n == [0, 3] and p == [128] * 3
    for s, rows in zip(step.ids, p):
        assert rows <= c.length(s) - 1
    e = c.add()
    c.extend([e], 0)
    assert groups(c.extend([e, c.fork(e)[0]], 3, shared=True)) is None


def test_out_of_pages_leaves_the_cache(no_copies):
    from exact_attention_67_gb300 import OutOfPages
    c = cache_of(20)
    a = c.add()
    c.extend([a], 300)
    forks = c.fork(a, 2)
    with pytest.raises(OutOfPages):
        c.extend(forks, 16, shared=True)
    assert c.free_pages == 1 and [c.length(s) for s in forks] == [300, 300]


@pytest.mark.parametrize("new", [1, 5])
def test_groups_where_enough_reads_are_saved(no_copies, new):
    c = cache_of()
    a = c.add()
    c.extend([a], 300)
    forks = c.fork(a, 3)
    c.share_from = 2 * 256 * 64 * 4  # two of the three need not read 256 rows of K and V, one head of 64
    assert groups(c.extend(forks, new, shared=True)) == ([0, 3], [256] * 3, 3 * new)
    c.share_from += 1
    assert groups(c.extend(forks, new, shared=True)) is None


def test_sizes_that_cannot_pay_take_the_plain_workspace(lib):
    def sizes(B=16, groups=1, Hq=32, Hk=8, total=16, mq=1, mk=8192, mg=16, d=128):
        plain = lib.attn_fwd_paged_workspace_size(B, Hq, Hk, total, mq, mk, d)
        return lib.attn_fwd_paged_shared_workspace_size(B, groups, Hq, Hk, total, mq, mk, mg, d), plain

    shared, plain = sizes()
    assert shared > plain
    for how in (dict(mk=127), dict(groups=16), dict(mk=1024), dict(B=2, total=2), dict(Hk=1, mk=2048)):
        shared, plain = sizes(**how)
        assert shared == plain > 0
    # Chunks: of few tokens, of as many as fill their tiles alone.
    shared, plain = sizes(B=24, total=240, mq=10, mg=240, mk=4096)
    assert shared > plain
    shared, plain = sizes(B=24, total=24 * 64, mq=64, mg=24 * 64, mk=4096)
    assert shared == plain


# ---------------------------------------------------------------- which neighbours make a group
def family(rows, count, base=(), first=0):
    """Page lists of ``count`` sequences behind ``rows`` rows on common pages of 16, the first of them ``base``, and
    one page of their own."""
    common = list(base) + [first + i for i in range(rows // 16 - len(base))]
    return [common + [first + 10 ** 6 + i] for i in range(count)]


def saved_by(tables, before, ps=16):
    from exact_attention_67_gb300.cache import _groups
    offsets, shared = _groups(tables, before, ps)
    assert offsets[0] == 0 and offsets[-1] == len(tables) and sorted(set(offsets)) == offsets
    for i, j in zip(offsets, offsets[1:]):
        rows = shared[i]
        assert shared[i:j] == [rows] * (j - i) and rows % 128 == 0 and (j - i > 1 or rows == 0)
        assert all(t[: rows // ps] == tables[i][: rows // ps] and rows <= n for t, n in zip(tables[i:j], before[i:j]))
    return offsets, shared, sum(shared) - sum(shared[i] for i in offsets[:-1])


def lengths(tables, ps=16):
    return [len(t) * ps - 1 for t in tables]


def test_a_shallow_sequence_does_not_pull_a_deep_group_down():
    deep = family(16384, 31)
    x = deep[0][:8] + [7 * 10 ** 6]  # 128 rows in common with them
    for tables, at in (([x, *deep], [0, 1, 32]), ([*deep, x], [0, 31, 32]), ([*deep[:20], x, *deep[20:]], [0, 20, 21, 32])):
        offsets, shared, saved = saved_by(tables, lengths(tables))
        assert offsets == at and max(shared) == 16384
        assert saved == sum(j - i - 1 for i, j in zip(at, at[1:])) * 16384
    # Two deep groups behind one preamble, which the first sequence has alone.
    other = family(16384, 31, base=deep[0][:8], first=10 ** 5)
    tables = [x, *deep, *other]
    assert saved_by(tables, lengths(tables)) == ([0, 1, 32, 63], [0] + [16384] * 62, 60 * 16384)


def test_rows_under_a_truncation_end_the_group_there(no_copies):
    """As test_rows_that_new_tokens_stand_on_are_not_shared: the split that saves most is the only one."""
    c = cache_of()
    a = c.add()
    c.extend([a], 400)
    f, g = c.fork(a, 2)
    c.truncate(f, 200)
    assert groups(c.extend([f, g, a], 1, shared=True)) == ([0, 1, 3], [0, 384, 384], 2)


def test_groups_save_as_much_as_any_split():
    """Against every split of neighbours, on random prompts that branch (pages as the path in a tree)."""
    import random
    rng = random.Random(5)
    for _ in range(300):
        n, path, tables = rng.randint(1, 9), [], []
        for _ in range(n):
            path = path[: rng.randint(0, len(path))]
            path = path + [rng.randrange(10 ** 9) for _ in range(rng.choice((0, 1, 8, 16, 40)))]
            tables.append(list(path))
        before = [rng.randint(0, 16 * len(t)) if rng.random() < 0.3 else 16 * len(t) for t in tables]

        def rows(i, j):
            m = 0
            while all(len(t) > m and t[m] == tables[i][m] for t in tables[i:j]):
                m += 1
            return min(16 * m, *before[i:j], 1 << 30) // 128 * 128

        best = [0]
        for j in range(1, n + 1):
            best.append(max(best[i] + (j - i - 1) * rows(i, j) for i in range(j)))
        assert saved_by(tables, before)[2] == best[n]


def test_grouping_a_large_batch_is_quick():
    """Its time is on the host at every step: forks of one prompt, and prompts that all branch at other rows."""
    import time
    forks = family(4096, 2048)
    ladder = [list(range(8 * i)) + [10 ** 6 + i] for i in range(1, 300)]
    tables = ladder + ladder[::-1]
    for t in (forks, tables):
        begin = time.perf_counter()
        saved_by(t, lengths(t))
        assert time.perf_counter() - begin < 2.0


def test_several_tokens_have_to_save_more(no_copies):
    """What the reads saved have to make up for grows with the new tokens: at 126 MB one a sequence is even or gains
    (heads of 128 21.5 and 19.6 us, of 64 19.4 and 25.4), five lose (31.0 and 26.3, 38.2 and 34.9)."""
    from exact_attention_67_gb300 import PagedCache
    c = PagedCache(400, 16, 1, 8, 128, device="cpu")
    a = c.add()
    c.extend([a], 2048)
    forks = c.fork(a, 40)
    some = forks[:16]  # fifteen of them need not read 2,048 rows of K and V of 8 heads of 128: 126 MB
    assert groups(c.extend(some, 1, shared=True)) == ([0, 16], [2048] * 16, 16)
    assert groups(c.extend(some, [1] * 15 + [2], shared=True)) is None
    assert groups(c.extend(some, 5, shared=True)) is None
    assert groups(c.extend(forks, 5, shared=True)) == ([0, 40], [2048] * 40, 200)  # 327 MB
    assert groups(c.extend(some[:4], 1, shared=True)) is None
    c.share_from = 1 << 20  # as given, whatever the count
    assert groups(c.extend(some[:4], 5, shared=True)) == ([0, 4], [2048] * 4, 20)
