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
