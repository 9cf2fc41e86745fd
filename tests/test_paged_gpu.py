"""Attention over a paged cache against the definition in 64 bits.

Everything in the cache that no query may see (rows behind a sequence's end,
pages of no sequence) holds NaN, and table entries past a sequence's pages hold
numbers outside the pool.

Bounds, fixed before the first run.  A weight relative to the others is off by
the f16 rounding, half a step: 2^-11 (its sum as much again where O is
normalised by the rounded ones), and by the errors of its fp32 score, below
2^-12 for these inputs; below f16's normal range by 2^-25 of the largest weight.
So with A = sum_j w_j |v_j|,
    |O - exact| <= h |O| + (2^-10 + 2^-12) A + 2^-24 sum_j |v_j|,
h the half step of the output's type (2^-8, 2^-11), and |lse - exact| <= 2^-12
(1 + |lse| 2^-10)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_67_gb300 import build
    build.build()


def randn(*shape, seed, dtype, scale=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).to(DEV)


class Problem:
    """A cache with sequences of the given lengths and their new tokens' queries."""

    def __init__(self, new, lens, Hq, Hk, d, ps, dtype, seed=0, token_major=False, pad=0, sigma=1.0):
        self.new, self.lens, self.Hq, self.Hk, self.d, self.ps, self.dtype, self.pad = new, lens, Hq, Hk, d, ps, dtype, pad
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((len(lens), max(max(need), 1) + 2), 1 << 30, dtype=torch.int32)
        shape = (pages, ps, Hk, d) if token_major else (pages, Hk, ps, d)
        self.kc, self.vc = (torch.full(shape, NAN, dtype=dtype, device=DEV) for _ in range(2))
        if token_major:
            self.kc, self.vc = self.kc.transpose(1, 2), self.vc.transpose(1, 2)
        self.k, self.v = [], []
        for b, n in enumerate(lens):
            k, v = randn(n, Hk, d, seed=seed + 10 * b + 1, dtype=dtype, scale=sigma), randn(n, Hk, d, seed=seed + 10 * b + 2, dtype=dtype)
            for i in range(need[b]):
                page = table[b, i] = order.pop()
                rows = slice(i * ps, min(n, (i + 1) * ps))
                self.kc[page, :, : rows.stop - rows.start] = k[rows].transpose(0, 1)
                self.vc[page, :, : rows.stop - rows.start] = v[rows].transpose(0, 1)
            self.k.append(k.double())
            self.v.append(v.double())
        self.table = table.to(DEV)
        self.q = randn(sum(new) + pad, Hq, d, seed=seed + 5, dtype=dtype, scale=sigma)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
        self.seq = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def run(self, causal=True, window=0, scale=None, cu=True, **kw):
        import exact_attention_67_gb300 as ex
        kw = {"max_seqlen_q": max(self.new), "max_seqlen_k": max(max(self.lens), 1)} | kw
        out = ex.forward_paged(self.q, self.kc, self.vc, self.table, self.seq, self.cu if cu else None, causal=causal,
                               window=window, scale=scale, **kw)
        torch.cuda.synchronize()
        assert ex.device_error() == 0
        return out

    def check(self, o, lse, causal=True, window=0, scale=None):
        scale = self.d ** -0.5 if scale is None else scale
        G, t = self.Hq // self.Hk, 0
        for b, (n, m) in enumerate(zip(self.new, self.lens)):
            if n == 0:
                continue
            q = self.q[t: t + n].double().view(n, self.Hk, G, self.d)
            pos = torch.arange(m - n, m, device=DEV)[:, None]
            j = torch.arange(m, device=DEV)[None]
            seen = torch.ones(n, m, dtype=torch.bool, device=DEV)
            if causal:
                seen &= j <= pos
            if window:
                seen &= (pos - j < window) & (j - pos < window)
            x = torch.einsum("ihgd,jhd->hgij", q, self.k[b]) * scale
            x = x.masked_fill(~seen, -torch.inf)
            L = torch.logsumexp(x, -1) if m else torch.full(x.shape[:-1], -torch.inf, dtype=torch.float64, device=DEV)
            w = torch.exp(x - L[..., None].clamp(min=-1e300))
            want = torch.einsum("hgij,jhd->ihgd", w, self.v[b]).reshape(n, self.Hq, self.d)
            size = torch.einsum("hgij,jhd->ihgd", w, self.v[b].abs()).reshape(n, self.Hq, self.d)
            tiny = 2.0 ** -24 * self.v[b].abs().sum(0).repeat_interleave(G, 0)
            err = (o[t: t + n].double() - want).abs()
            bound = HALF[self.dtype] * want.abs() + (2.0 ** -10 + 2.0 ** -12) * size + tiny
            assert bool((err <= bound).all()), f"sequence {b}: O off by {float((err - bound).max()):.3e} over the bound"
            L = L.permute(2, 0, 1).reshape(n, self.Hq).t()
            got = lse[:, t: t + n].double()
            none = torch.isinf(L)
            assert torch.equal(torch.isinf(got) & (got < 0), none), f"sequence {b}: rows without keys"
            el = (got - L)[~none].abs()
            assert not el.numel() or bool((el <= 2.0 ** -12 * (1 + L[~none].abs() * 2.0 ** -10)).all()), \
                f"sequence {b}: lse off by {float(el.max()):.3e}"
            t += n


CASES = [
    # (new, lens, Hq, Hk, d, page, dtype, causal, window)
    # Few rows a key head: the decode kernel.
    ([1], [1], 1, 1, 128, 16, torch.bfloat16, True, 0),
    ([1], [777], 32, 8, 128, 16, torch.bfloat16, True, 0),
    ([1] * 5, [0, 1, 127, 128, 129], 4, 4, 64, 64, torch.float16, True, 0),
    ([1] * 7, [3000, 5, 64, 999, 4096, 1, 250], 8, 1, 128, 128, torch.bfloat16, True, 0),
    ([1] * 40, [17 * i + 1 for i in range(40)], 12, 4, 64, 16, torch.bfloat16, True, 0),
    ([1] * 70, [100] * 70, 2, 2, 128, 8, torch.float16, True, 0),
    ([3, 1, 5, 0, 2], [700, 1, 5, 90, 1500], 9, 3, 128, 32, torch.bfloat16, True, 0),
    ([4, 4], [300, 2000], 4, 1, 64, 256, torch.float16, False, 0),
    ([2, 2, 1], [300, 2000, 40], 16, 2, 128, 16, torch.bfloat16, True, 100),
    ([5, 3], [2, 900], 3, 1, 64, 32, torch.float16, True, 0),     # positions below 0 see nothing
    ([3], [600], 5, 1, 128, 64, torch.bfloat16, False, 70),
    ([1], [70000], 2, 1, 128, 64, torch.bfloat16, True, 0),
    ([4, 1, 3], [900, 1, 4000], 16, 2, 128, 16, torch.bfloat16, True, 0),   # up to 32 rows
    ([1] * 6, [50, 1200, 128, 3, 900, 4000], 32, 1, 64, 32, torch.float16, True, 0),
    ([1, 1], [300, 5000], 20, 1, 128, 64, torch.float16, True, 0),
    ([2, 2, 0], [256, 1025, 7], 30, 2, 64, 128, torch.bfloat16, True, 200),
    ([7, 2], [5, 1500], 4, 1, 128, 8, torch.bfloat16, True, 0),
    # Units of few key tiles, that are not cut: more and fewer of them than SMs.
    ([1] * 300, [(37 * i) % 500 for i in range(300)], 4, 2, 128, 16, torch.bfloat16, True, 0),
    ([3] * 33, [1 + (91 * i) % 1020 for i in range(33)], 15, 5, 64, 32, torch.float16, True, 0),
    ([1] * 90, [9000 + i for i in range(90)], 8, 2, 64, 64, torch.bfloat16, True, 300),
    ([100, 1, 0, 333, 500], [100, 480, 12, 400, 500], 8, 2, 128, 64, torch.bfloat16, True, 0),
    ([700] * 3, [700, 900, 1024], 8, 8, 64, 16, torch.float16, True, 0),
    # More rows: the forward kernel.
    ([17], [17], 1, 1, 64, 16, torch.bfloat16, True, 0),
    ([130, 1, 40], [400, 33, 40], 4, 1, 128, 16, torch.bfloat16, True, 0),
    ([257, 64], [1000, 64], 2, 2, 64, 32, torch.float16, True, 0),
    ([100, 0, 300, 7], [4000, 50, 300, 2500], 10, 2, 128, 64, torch.float16, True, 0),
    ([90, 200], [700, 1200], 14, 2, 64, 128, torch.bfloat16, True, 150),
    ([60], [500], 6, 2, 128, 512, torch.bfloat16, False, 0),
    ([60, 33], [500, 2000], 6, 2, 64, 8, torch.float16, False, 130),
    ([40, 9], [30, 9], 20, 1, 128, 16, torch.bfloat16, True, 0),  # positions below 0
    ([3], [300], 128, 1, 128, 32, torch.bfloat16, True, 0),       # 128 query heads to a key head
    ([5, 5], [300, 31], 100, 2, 64, 32, torch.float16, True, 0),
    ([1500], [9000], 4, 1, 128, 64, torch.bfloat16, True, 0),
    ([1, 600, 1, 1, 31], [5000, 600, 3, 129, 2000], 8, 2, 128, 16, torch.bfloat16, True, 0),
]


@pytest.mark.parametrize("new,lens,Hq,Hk,d,ps,dtype,causal,window", CASES, ids=lambda x: str(x)[:30].replace(" ", ""))
def test_paged_attention(new, lens, Hq, Hk, d, ps, dtype, causal, window):
    p = Problem(new, lens, Hq, Hk, d, ps, dtype, seed=len(lens) + d, token_major=Hq % 2 == 1)
    p.check(*p.run(causal, window), causal, window)


def test_wide_scores_and_scale():
    """Scores spread over hundreds: the running maximum moves often."""
    for d, new, dtype in ((128, [1, 3], torch.bfloat16), (64, [200, 90], torch.float16)):
        p = Problem(new, [2000, 700], 4, 2, d, 32, dtype, seed=3, sigma=4.0)
        p.k = [k * 1.0 for k in p.k]
        p.check(*p.run(scale=0.05), scale=0.05)


def test_layouts_and_rows_left_alone():
    """Q a slice of a wider projection, O with strides of its own; rows behind the
    last sequence stay as they were; the same bits every time."""
    import exact_attention_67_gb300 as ex
    for new, Hq, Hk, d in (([1, 2, 0, 3], 6, 2, 128), ([70, 2, 0, 90], 6, 2, 64)):
        p = Problem(new, [400, 77, 5, 1000], Hq, Hk, d, 16, torch.bfloat16, seed=9, pad=5)
        total = sum(new) + 5
        wide = torch.zeros(total, Hq + 2 * Hk, d, dtype=torch.bfloat16, device=DEV)
        wide[:, :Hq] = p.q
        o = torch.full((Hq, total, d), 3.0, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
        lse = torch.full((Hq, total), 3.0, device=DEV)
        ws = torch.empty(ex.attn_fwd_paged_workspace_size(4, Hq, Hk, total, 90, 1000, d), dtype=torch.uint8, device=DEV)
        runs = []
        for _ in range(3):
            ex.attn_fwd_paged(wide[:, :Hq], p.kc, p.vc, o, lse, p.table, p.seq, p.cu, 90, 1000, True, d ** -0.5, ws)
            runs.append((o.clone(), lse.clone()))
        p.check(o, lse)
        assert torch.all(o[sum(new):] == 3.0) and torch.all(lse[:, sum(new):] == 3.0)
        assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_even_batches_need_no_offsets():
    for new in (1, 3, 40):
        p = Problem([new] * 4, [100, 900, new, 333], 8, 2, 64, 32, torch.float16, seed=new)
        a, b = p.run(), p.run(cu=False)
        assert all(torch.equal(x, y) for x, y in zip(a, b))
        p.check(*b)
        p.check(*p.run(cu=False, max_seqlen_q=None, max_seqlen_k=None))


def test_capture_and_replay_with_other_lengths():
    """A captured call reads the tables that are there at the replay."""
    import exact_attention_67_gb300 as ex
    for new, Hq in (([1, 1, 1], 8), ([40, 3, 60], 4)):
        p = Problem(new, [1500, 700, 90], Hq, 2, 128, 16, torch.bfloat16, seed=21)
        o, lse = torch.empty_like(p.q), torch.empty(Hq, p.q.shape[0], device=DEV)
        ws = torch.empty(ex.attn_fwd_paged_workspace_size(3, Hq, 2, sum(new), max(new), 1500, 128), dtype=torch.uint8,
                         device=DEV)
        seq = p.seq.clone()

        def call():
            ex.attn_fwd_paged(p.q, p.kc, p.vc, o, lse, p.table, seq, p.cu, max(new), 1500, True, 128 ** -0.5, ws)

        call()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
            call()
        for lens in ([1500, 700, 90], [1400, 64, 61], [1000, 3, 90]):
            seq.copy_(torch.tensor(lens, dtype=torch.int32))
            o.fill_(NAN)
            graph.replay()
            torch.cuda.synchronize()
            p.lens, full = lens, (p.k, p.v)
            p.k, p.v = [k[:n] for k, n in zip(p.k, lens)], [v[:n] for v, n in zip(p.v, lens)]
            p.check(o, lse)
            p.k, p.v = full


def test_two_calls_at_once():
    """Two streams, each with its own workspace and outputs, against the same calls
    one after the other."""
    import exact_attention_67_gb300 as ex
    problems = [Problem([1] * 6, [4000, 300, 2500, 17, 900, 3333], 8, 2, 128, 16, torch.bfloat16, seed=1),
                Problem([100, 7], [3000, 2000], 8, 2, 128, 32, torch.bfloat16, seed=2)]
    want = [p.run() for p in problems]
    streams = [torch.cuda.Stream() for _ in problems]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for p, s in zip(problems, streams):
            with torch.cuda.stream(s):
                got.append(ex.forward_paged(p.q, p.kc, p.vc, p.table, p.seq, p.cu, max(p.new), max(p.lens)))
    torch.cuda.synchronize()
    assert ex.device_error() == 0
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i % 2]))


def test_wrong_tables_and_bounds():
    """Page numbers outside the pool read as zeros, sequences beyond the given bounds
    are cut off, offsets past the tensors leave rows alone: wrong or short results,
    never an access out of bounds."""
    import exact_attention_67_gb300 as ex
    for new, Hq in (([2, 2], 4), ([50, 30], 4)):
        p = Problem(new, [200, 300], Hq, 2, 64, 16, torch.float16, seed=31)
        p.table[1, 3] = p.kc.shape[0] + 7       # keys 48..63 of sequence 1
        p.table[1, 4] = -3
        p.k[1][48:80] = 0.0
        p.v[1][48:80] = 0.0
        p.check(*p.run())
        o, lse = p.run(max_seqlen_k=128)        # only keys 0..127 are seen
        cut = Problem(new, [200, 300], Hq, 2, 64, 16, torch.float16, seed=31)
        cut.k, cut.v = [k[:128] for k in p.k], [v[:128] for v in p.v]
        cut.lens, cut.new = [128, 128], new
        cut.check(o, lse, causal=False)         # all of them lie before the new tokens
        p.cu = torch.tensor([0, 1 << 30, -5], dtype=torch.int32, device=DEV)
        p.run()
        p.seq = torch.tensor([1 << 30, -9], dtype=torch.int32, device=DEV)
        p.run()


def test_nan_stays_with_its_rows():
    """A NaN in a visible key reaches the rows that see it and no others."""
    for new, lens, Hq in (([1, 1], [500, 700], 8), ([80, 60], [500, 700], 4)):
        p = Problem(new, lens, Hq, 2, 128, 16, torch.bfloat16, seed=41)
        page = int(p.table[0, 5])
        p.kc[page, 1, 3, 7] = NAN               # key 83 of sequence 0, key head 1
        o, lse = p.run()
        hit = torch.zeros(sum(new), Hq, dtype=torch.bool, device=DEV)
        hit[: new[0], Hq // 2:] = True
        assert torch.equal(torch.isnan(o).all(-1), hit) and torch.equal(torch.isnan(o).any(-1), hit)
        assert torch.equal(torch.isnan(lse).t(), hit)


def test_nan_queries_of_sequences_on_many_sms():
    """A query of NaN: its rows are NaN in every piece, and after the join."""
    for new, Hq in (([2], 4), ([40], 4)):
        p = Problem(new, [9000], Hq, 2, 64, 32, torch.float16, seed=43)
        p.q[1, 2] = NAN
        o, lse = p.run()
        hit = torch.zeros(new[0], Hq, dtype=torch.bool, device=DEV)
        hit[1, 2] = True
        assert torch.equal(torch.isnan(o).all(-1), hit) and torch.equal(torch.isnan(o).any(-1), hit)
        assert torch.equal(torch.isnan(lse).t(), hit)


def test_pools_past_32_bits():
    """Pages whose elements lie past 2^31, and bytes past 2^32, from the pool's start:
    append, copy and attention."""
    import exact_attention_67_gb300 as ex
    pages, ps, d = 140000, 128, 128
    pool = torch.empty(2, pages, 1, ps, d, dtype=torch.bfloat16, device=DEV)
    n = 300
    k, v, q = (randn(n, 1, d, seed=s, dtype=torch.bfloat16) for s in (1, 2, 3))
    table = torch.tensor([[pages - 1, 3, pages - 2]], dtype=torch.int32, device=DEV)
    seq = torch.tensor([n], dtype=torch.int32, device=DEV)
    ex.attn_cache_append(k, v, pool[0], pool[1], table, seq)
    ex.attn_cache_copy(pool, [pages - 1, 3], [pages - 7, pages - 9])
    p = Problem([n], [n], 1, 1, d, ps, torch.bfloat16)
    p.q, p.k, p.v = q, [k.double()], [v.double()]
    for first in ([pages - 1, 3, pages - 2], [pages - 7, pages - 9, pages - 2]):
        p.kc, p.vc, p.table = pool[0], pool[1], torch.tensor([first], dtype=torch.int32, device=DEV)
        p.check(*p.run())


@pytest.mark.parametrize("Hq,Hk,d,ps,dtype,window", [(8, 2, 128, 16, torch.bfloat16, 0), (6, 2, 64, 8, torch.float16, 50)])
def test_a_serving_run(Hq, Hk, d, ps, dtype, window):
    """A PagedCache through a life: prompts in chunks, single tokens, forks that write
    on, tokens taken back, sequences freed, the pool compacted -- attention at every
    step and layer against the tokens' own K and V in 64 bits."""
    import random

    import exact_attention_67_gb300 as ex
    from tests.test_rotary_gpu import turned
    r, layers = random.Random(d), 2
    cache = ex.PagedCache(150, ps, layers, Hk, d, dtype)
    cache.pool.fill_(NAN)
    freq, factor = ex.rotary_frequencies(d // 2, yarn=2.0)
    kept = {}                                    # sequence -> per layer, its rounded K and V
    seed = [0]

    def turn(x, pos):                            # [n, H, d], turned and rounded as the cache holds it
        y, _ = turned(x.double().cpu().numpy().transpose(1, 0, 2), pos, freq.cpu().numpy(), factor, False)
        return torch.from_numpy(y.transpose(1, 0, 2))

    def step(seqs, new):
        at = [cache.length(s) for s in seqs]
        new = [new] * len(seqs) if isinstance(new, int) else new
        st = cache.extend(seqs, new if len(set(new)) > 1 else new[0])
        total = sum(new)
        for layer in range(layers):
            seed[0] += 1
            k, v, q = (randn(total, h, d, seed=3 * seed[0] + i, dtype=dtype) for i, h in enumerate((Hk, Hk, Hq)))
            qo = torch.empty_like(q)
            cache.append(layer, st, k, v, q, qo, freq, False, factor)
            o, lse = cache.attend(layer, st, qo, window=window)
            torch.cuda.synchronize()
            t = 0
            for s, n, a in zip(seqs, new, at):
                rows = slice(t, t + n)
                t += n
                if n == 0:
                    continue
                pos = torch.arange(a, a + n).numpy()
                # The cache's own K (checked against the definition to one step of its type).
                pages = cache.pages(s)
                mine = torch.stack([cache.k_cache(layer)[pages[i // ps], :, i % ps] for i in range(a, a + n)])
                want = turn(k[rows], pos).to(DEV)
                assert bool(((mine.double() - want).abs() <= 2 * HALF[dtype] * want.abs() + 2.0 ** -16).all())
                got_k, got_v = kept[s][layer]
                kept[s][layer] = (torch.cat([got_k, mine]), torch.cat([got_v, v[rows]]))
                m = a + n
                p = Problem.__new__(Problem)
                p.new, p.lens, p.Hq, p.Hk, p.d, p.dtype, p.q = [n], [m], Hq, Hk, d, dtype, qo[rows]
                p.k, p.v = [kept[s][layer][0].double()], [kept[s][layer][1].double()]
                p.check(o[rows], lse[:, rows], True, window)
        assert ex.device_error() == 0

    def add():
        s = cache.add()
        kept[s] = [(torch.empty(0, Hk, d, dtype=dtype, device=DEV),) * 2 for _ in range(layers)]
        return s

    a, b, c = add(), add(), add()
    step([a, b], [130, 7])
    step([a, b, c], [1, 40, 1])
    step([a, b, c], 1)
    forks = cache.fork(a, 2)
    for f in forks:
        kept[f] = list(kept[a])
    step([forks[0], b, forks[1], a], 1)          # three writers of one shared page
    step([forks[0], a], 3)
    cache.truncate(a, cache.length(a) - 2)
    kept[a] = [(x[:-2], y[:-2]) for x, y in kept[a]]
    step([a, c], [2, 0])
    cache.free([b, forks[1]])
    moved = cache.compact()
    assert moved > 0
    for _ in range(2):
        step(r.sample([a, c, forks[0]], 3), 1)
    d2 = add()
    step([d2, a], [65, 1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("new,lens,Hq,Hk,d,window,causal", [
    ([1, 1, 1], [200, 777, 90], 8, 2, 128, 70, True),
    ([3, 2], [700, 130], 8, 2, 64, 40, False),
    ([90, 33], [600, 250], 4, 1, 128, 100, True),
    ([150], [500], 2, 2, 64, 33, False)])
def test_rows_before_the_window(new, lens, Hq, Hk, d, window, causal, dtype):
    """Rows that the window has left behind hold NaN, pages that it has left behind
    whole are gone from the table."""
    p = Problem(new, lens, Hq, Hk, d, 16, dtype, seed=47)
    for b, (n, m) in enumerate(zip(new, lens)):
        for r in range(max(0, m - n - window + 1)):
            page = int(p.table[b, r // 16])
            p.kc[page, :, r % 16] = p.vc[page, :, r % 16] = NAN
        gone = max(0, m - n - window + 1) // 16
        p.table[b, : gone // 2] = -1
    p.check(*p.run(causal=causal, window=window), causal=causal, window=window)


def test_helpers_on_a_given_stream():
    """What the helpers allocate and compute belongs to the stream that they are
    given: the current one, held up here, has no part in it."""
    import exact_attention_67_gb300 as ex
    p = Problem([1, 40], [700, 300], 4, 2, 64, 16, torch.bfloat16, seed=53)
    x = p.q[None].transpose(1, 2)                                   # [1, Hq, 41, 64]
    want, turned = p.run(), ex.rotary(x)
    cache = ex.PagedCache(8, 16, 1, 2, 64)
    k, v, q = randn(20, 2, 64, seed=1, dtype=torch.bfloat16), randn(20, 2, 64, seed=2, dtype=torch.bfloat16), p.q[:20]
    seq = cache.add()
    step = cache.extend([seq], 20)
    cache.append(0, step, k, v)
    through = cache.attend(0, step, q)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (other, other.cuda_stream):
        torch.cuda._sleep(400_000_000)
        busy = torch.cuda.Event()
        busy.record()
        got = ex.forward_paged(p.q, p.kc, p.vc, p.table, p.seq, p.cu, max(p.new), max(p.lens), stream=given)
        y = ex.rotary(x, stream=given)
        cache.free(seq)
        seq = cache.add()
        step = cache.extend([seq], 20, stream=given)
        cache.append(0, step, k, v, stream=given)
        again = cache.attend(0, step, q, stream=given)
        other.synchronize()
        assert not busy.query()
        with torch.cuda.stream(other):
            assert all(torch.equal(a, b) for a, b in zip([*got, y, *again], [*want, turned, *through]))
        torch.cuda.synchronize()
    assert ex.device_error() == 0


def test_a_wait_that_gave_up_is_told():
    """The watchdog's self-test, then a call: it raises, and the next one runs."""
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import _lib
    p = Problem([1, 1], [20, 30], 4, 2, 64, 16, torch.bfloat16)
    p.run()
    _lib.watchdog_selftest()
    torch.cuda.synchronize()
    with pytest.raises(ex.ExattnError):
        p.run()
    p.check(*p.run())


def test_cache_steps_in_a_graph():
    """PagedCache's append and attend captured, replayed on other tokens, with eager
    calls before and after."""
    import exact_attention_67_gb300 as ex
    cache = ex.PagedCache(16, 16, 2, 2, 64)
    seqs = [cache.add(), cache.add()]
    freq, factor = ex.rotary_frequencies(64)
    step = cache.extend(seqs, 30)
    new = [randn(60, h, 64, seed=60 + h, dtype=torch.bfloat16) for h in (2, 3, 8)]
    k, v, q = new[0], new[1][:, :2], new[2]

    def run():
        outs = []
        for layer in range(2):
            turned = torch.empty_like(q)
            cache.append(layer, step, k, v, q=q, q_out=turned, inv_freq=freq, factor=factor)
            outs.append(cache.attend(layer, step, turned))
        return outs

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = run()
    for i in range(2):
        for x in (k, v, q):
            x.copy_(randn(*x.shape, seed=70 + i, dtype=torch.bfloat16))
        graph.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in pair] for pair in outs]
        for a, b in zip(got, run()):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert ex.device_error() == 0


def test_attention_refusals():
    import exact_attention_67_gb300 as ex
    p = Problem([1, 1], [20, 30], 4, 2, 64, 16, torch.bfloat16)
    call = ex.forward_paged
    with pytest.raises(TypeError):
        call(p.q, p.kc, p.vc, p.table.long(), p.seq, p.cu)
    with pytest.raises(TypeError):
        call(p.q.float(), p.kc, p.vc, p.table, p.seq, p.cu)
    for bad in (lambda: call(p.q, p.kc.half(), p.vc.half(), p.table, p.seq, p.cu), lambda: call(p.q, p.kc, p.vc[:-1], p.table, p.seq),
                lambda: call(p.q, p.kc, p.vc, p.table, p.seq[:1]), lambda: call(p.q, p.kc, p.vc, p.table, p.seq, p.cu[:2]),
                lambda: call(p.q[:1], p.kc, p.vc, p.table, p.seq), lambda: call(p.q, p.kc, p.vc, p.table.cpu(), p.seq, p.cu),
                lambda: call(p.q, p.kc.transpose(2, 3), p.vc.transpose(2, 3), p.table, p.seq, p.cu)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: call(p.q, p.kc, p.vc, p.table, p.seq, p.cu, window=-1), lambda: call(p.q, p.kc, p.vc, p.table, p.seq, scale=0.0),
                lambda: call(p.q[:, :3], p.kc, p.vc, p.table, p.seq)):
        with pytest.raises(ex.ExattnError):
            bad()
    o, lse = call(p.q[:0], p.kc, p.vc, p.table, p.seq, torch.zeros(3, dtype=torch.int32, device=DEV))
    assert o.shape[0] == 0 and lse.shape[1] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new,G", [(1, 1), (2, 8), (40, 1)])
@pytest.mark.parametrize("at", [0, 70000, 131071])
def test_many_small_weights_beside_a_large_one(new, G, d, dtype, at):
    """One key 17.5 above 131,071 others, whose weights of 2^-25.2 of the largest
    together are 3 in 1,000 of the mass.  Its V is 0, theirs are 1: O is their mass A,
    to the bound of this file's head with the weights' absolute rounding at 2^-32 of
    the largest, in the product and in the sum that normalises it."""
    import exact_attention_67_gb300 as ex
    B, n, ps = 160, 131072, 64
    kc, vc = torch.zeros(2, 1, ps, d, dtype=dtype, device=DEV), torch.ones(2, 1, ps, d, dtype=dtype, device=DEV)
    kc[1, 0, at % ps, 3], vc[1, 0, at % ps] = 17.5, 0.0              # exact in both types
    table = torch.zeros(B, n // ps, dtype=torch.int32, device=DEV)   # page 0, again and again
    table[:, at // ps] = 1
    q = torch.zeros(B * new, G, d, dtype=dtype, device=DEV)
    q[..., 3] = 1.0
    o, lse = ex.forward_paged(q, kc, vc, table, torch.full((B,), n, dtype=torch.int32, device=DEV), None, new, n, causal=False,
                              scale=1.0)
    torch.cuda.synchronize()
    assert ex.device_error() == 0
    mass = (n - 1) * np.exp(-17.5)
    A = mass / (1 + mass)
    bound = HALF[dtype] * A + (2.0 ** -10 + 2.0 ** -12) * A + 2 * 2.0 ** -32 * n
    assert float((o.double() - A).abs().max()) <= bound
    L = 17.5 + np.log1p(mass)
    assert float((lse.double() - L).abs().max()) <= 2.0 ** -12 * (1 + L * 2.0 ** -10)


@pytest.mark.parametrize("new,G,n", [(1, 8, 1300), (1, 1, 3000), (4, 2, 2500), (3, 8, 1500), (40, 1, 5000), (130, 2, 3000)])
@pytest.mark.parametrize("d,dtype", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("base", [4096, 5120, 6144, 7168])
def test_pieces_joined_at_large_scores(new, G, n, d, dtype, base):
    """A sequence on many SMs whose scores all lie near 64 base: exact in 32 bits, and
    with scale = ln 2 their weights are powers of 2, exact too, so that nothing but the
    roundings of this file's head is left -- as where no sequence is cut."""
    import exact_attention_67_gb300 as ex
    g = torch.Generator().manual_seed(n + base)
    small = torch.randint(-3, 4, (n,), generator=g)
    ps, Hk = 32, 2
    pages = -(-n // ps)
    kc, vc = (torch.zeros(pages, Hk, ps, d, dtype=dtype, device=DEV) for _ in range(2))
    sign = torch.where(torch.arange(n) < n // 2, 1.0, -1.0)
    for j0 in range(0, n, ps):
        m = min(ps, n - j0)
        kc[j0 // ps, :, :m, 0], kc[j0 // ps, :, :m, 1] = float(base), small[j0: j0 + m].to(dtype).to(DEV)
        vc[j0 // ps, :, :m] = sign[j0: j0 + m, None].to(dtype).to(DEV)
    q = torch.zeros(new, Hk * G, d, dtype=dtype, device=DEV)
    q[..., 0], q[..., 1] = 64.0, 1.0
    table, lens = torch.arange(pages, dtype=torch.int32, device=DEV)[None], torch.tensor([n], dtype=torch.int32, device=DEV)
    scale = float(torch.tensor(np.log(2.0), dtype=torch.float32))
    o, lse = ex.forward_paged(q, kc, vc, table, lens, None, new, n, causal=False, scale=scale)
    torch.cuda.synchronize()
    assert ex.device_error() == 0
    w = 2.0 ** small.double()
    want = float((w * sign).sum() / w.sum())
    bound = HALF[dtype] * abs(want) + 2.0 ** -10 + 2.0 ** -12 + 2.0 ** -32 * n
    assert float((o.double() - want).abs().max()) <= bound
    L = (64.0 * base + np.log2(float(w.sum()))) * np.log(2.0)
    assert float((lse.double() - L).abs().max()) <= 2.0 ** -23 * L + 2.0 ** -20


@pytest.mark.parametrize("streams", [1, 2])
def test_a_wait_that_gave_up_behind_an_earlier_call_is_told(streams):
    """The stream held up, a call, then a wait that gives up and another call, on the
    same stream or on one that is not held up: once these are done the explicit check
    raises, whatever polls were in flight."""
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import _lib
    p = Problem([1, 1], [20, 30], 4, 2, 64, 16, torch.bfloat16)
    p.run()

    def call():
        return ex.forward_paged(p.q, p.kc, p.vc, p.table, p.seq, p.cu, 1, 30)

    second = torch.cuda.Stream() if streams == 2 else torch.cuda.current_stream()
    torch.cuda._sleep(400_000_000)
    call()
    with torch.cuda.stream(second):
        assert _lib.load().exattn_watchdog_selftest(2000, second.cuda_stream) == 0
        call()
        call()
    second.synchronize()
    with pytest.raises(ex.ExattnError):
        ex.watchdog_check(DEV)
    ex.watchdog_check(DEV)
    assert ex.device_error() == 0
    p.check(*p.run())


def test_a_wait_that_gave_up_in_a_graph_is_told():
    """A captured call takes no poll; the explicit check tells of a replay's wait."""
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import _lib
    p = Problem([1, 1], [20, 30], 4, 2, 64, 16, torch.bfloat16)
    p.run()
    ex.watchdog_check(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ex.forward_paged(p.q, p.kc, p.vc, p.table, p.seq, p.cu, 1, 30)
        assert _lib.load().exattn_watchdog_selftest(2000, torch.cuda.current_stream().cuda_stream) == 0
    ex.watchdog_check(DEV)
    graph.replay()
    torch.cuda.synchronize()
    with pytest.raises(ex.ExattnError):
        ex.watchdog_check(DEV)
    p.check(*p.run())
