"""Attention behind shared rows against the definition in 64 bits: the bounds, and the
NaN in everything that no query may see, are those of test_paged_gpu.  (Joining pieces
in fp32, by differences of references that are exact, adds less than 2^-20 of A.)

Calls whose sizes say that sharing cannot pay run as attn_fwd_paged.  The sizes here are
small, so max_seqlen_k, a bound, is given as 2^20, which lets them share; that they do
shows in their workspace."""
import numpy as np
import pytest
import torch

from .test_paged_gpu import DEV, HALF, NAN, Problem, randn  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from exact_attention_67_gb300 import build
    build.build()


class Family(Problem):
    """families: (shared rows, whole pages, [(new tokens, own rows before them), ...])."""

    def __init__(self, families, Hq, Hk, d, ps, dtype, seed=0, pad=0, sigma=1.0, alone_shares=False):
        self.Hq, self.Hk, self.d, self.ps, self.dtype, self.pad = Hq, Hk, d, ps, dtype, pad
        members = [(p, n, o) for p, ms in families for n, o in ms]
        self.new, self.lens = [n for _, n, _ in members], [p + o + n for p, n, o in members]
        assert all(p % ps == 0 for p, _ in families)
        need = [-(-m // ps) for m in self.lens]
        pages = sum(p // ps for p, _ in families) + sum(need) + 3
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
        table = torch.full((len(members), max(max(need), 1) + 2), 1 << 30, dtype=torch.int32)
        self.kc, self.vc = (torch.full((pages, Hk, ps, d), NAN, dtype=dtype, device=DEV) for _ in range(2))
        self.k, self.v, b = [], [], 0
        for f, (p, ms) in enumerate(families):
            common = [order.pop() for _ in range(p // ps)]
            ks, vs = randn(p, Hk, d, seed=seed + 7000 + 2 * f, dtype=dtype, scale=sigma), randn(p, Hk, d, seed=seed + 7001 + 2 * f, dtype=dtype)
            for n, o in ms:
                m = o + n
                k = torch.cat((ks, randn(m, Hk, d, seed=seed + 10 * b + 1, dtype=dtype, scale=sigma)))
                v = torch.cat((vs, randn(m, Hk, d, seed=seed + 10 * b + 2, dtype=dtype)))
                own = common + [order.pop() for _ in range(need[b] - len(common))]
                table[b, : len(own)] = torch.tensor(own, dtype=torch.int32)
                for i, page in enumerate(own):
                    rows = slice(i * ps, min(p + m, (i + 1) * ps))
                    self.kc[page, :, : rows.stop - rows.start] = k[rows].transpose(0, 1)
                    self.vc[page, :, : rows.stop - rows.start] = v[rows].transpose(0, 1)
                self.k.append(k.double())
                self.v.append(v.double())
                b += 1
        ends = np.cumsum([0] + [len(ms) for _, ms in families])
        self.groups = torch.tensor(ends, dtype=torch.int32, device=DEV)
        self.prefix = torch.tensor([p if len(ms) > 1 or alone_shares else 0 for p, ms in families for _ in ms], dtype=torch.int32, device=DEV)
        self.max_group = max(1, *(sum(self.new[i:j]) for i, j in zip(ends, ends[1:])))
        self.table = table.to(DEV)
        self.q = randn(sum(self.new) + pad, Hq, d, seed=seed + 5, dtype=dtype, scale=sigma)
        self.cu = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32, device=DEV)
        self.seq = torch.tensor(self.lens, dtype=torch.int32, device=DEV)

    def sizes(self, **kw):
        return {"max_seqlen_q": max(1, *self.new), "max_seqlen_k": 1 << 20, "max_group_q": self.max_group} | kw

    def shares(self, **kw):
        """Whether a call of these sizes streams shared rows once."""
        import exact_attention_67_gb300 as ex
        q, k, g = self.sizes(**kw).values()
        B, total = len(self.new), self.q.shape[0]
        return (ex.attn_fwd_paged_shared_workspace_size(B, self.groups.numel() - 1, self.Hq, self.Hk, total, q, k, g, self.d)
                != ex.attn_fwd_paged_workspace_size(B, self.Hq, self.Hk, total, q, k, self.d))

    def run(self, causal=True, scale=None, cu=True, window=0, **kw):
        import exact_attention_67_gb300 as ex
        assert window == 0
        out = ex.forward_paged_shared(self.q, self.kc, self.vc, self.table, self.seq, self.groups, self.prefix, self.cu if cu else None,
                                      causal=causal, scale=scale, **self.sizes(**kw))
        torch.cuda.synchronize()
        assert ex.device_error() == 0
        return out

    def into(self, fill, o=None, lse=None, **kw):
        """The raw call, on a workspace that holds `fill` in every byte."""
        import exact_attention_67_gb300 as ex
        s = self.sizes(**kw)
        total = self.q.shape[0]
        o = torch.full_like(self.q, 5.0) if o is None else o
        lse = torch.full((self.Hq, total), 5.0, device=DEV) if lse is None else lse
        n = ex.attn_fwd_paged_shared_workspace_size(len(self.new), self.groups.numel() - 1, self.Hq, self.Hk, total, *s.values(), self.d)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        ex.attn_fwd_paged_shared(self.q, self.kc, self.vc, o, lse, self.table, self.seq, self.cu, self.groups, self.prefix, *s.values(), True,
                                 self.d ** -0.5, ws)
        torch.cuda.synchronize()
        assert ex.device_error() == 0
        return o, lse


bf, hf = torch.bfloat16, torch.float16
CASES = {
    # name: (families, Hq, Hk, d, page, dtype, causal)
    "two answers": ([(512, [(1, 40), (1, 40)])], 32, 8, 128, 16, bf, True),
    "nothing of their own": ([(256, [(1, 0), (1, 0), (1, 0)])], 8, 2, 64, 16, hf, True),
    "nothing shared": ([(0, [(1, 300), (1, 5)]), (0, [(1, 1)])], 4, 4, 128, 8, bf, True),
    "less than a tile shared": ([(96, [(1, 300), (1, 5)])], 4, 2, 64, 32, bf, True),
    "a tile and a part": ([(128 + 24, [(1, 3), (1, 200), (1, 0)])], 10, 2, 128, 8, hf, True),
    "many pieces": ([(40000, [(1, 4000), (1, 4), (1, 1000)])], 4, 1, 128, 64, bf, True),
    "alone and together": ([(640, [(1, 9)]), (1280, [(1, 700), (1, 3)]), (0, [(1, 50)])], 16, 4, 128, 128, bf, True),
    "forward behind decode": ([(1500 // 16 * 16, [(1, 100 + 13 * i) for i in range(16)])], 24, 8, 64, 16, bf, True),
    "two query tiles": ([(2048, [(1, 10 * i) for i in range(40)])], 64, 8, 128, 64, bf, True),
    "several units a group": ([(1024, [(1, i) for i in range(90)]), (256, [(1, 3)] * 50)], 16, 2, 128, 32, hf, True),
    "drafts": ([(5000 // 32 * 32, [(5, 70), (5, 900)]), (640, [(3, 11), (5, 0), (1, 129)])], 24, 8, 64, 32, hf, True),
    "no new tokens": ([(256, [(0, 40), (1, 3), (0, 0)]), (128, [(0, 0), (0, 2)]), (384, [(2, 2), (1, 1)])], 8, 4, 64, 64, bf, True),
    "chunks": ([(2048, [(100, 0), (257, 5), (31, 700)])], 8, 2, 128, 64, bf, True),
    "chunks, d 64": ([(640, [(300, 0), (17, 100), (9, 3)]), (256, [(130, 1), (200, 0)])], 6, 2, 64, 16, hf, True),
    "not causal": ([(1024, [(4, 60), (2, 9)]), (256, [(1, 0), (1, 300)])], 8, 8, 128, 32, bf, False),
    "chunks, not causal": ([(512, [(90, 60), (70, 0), (14, 5)])], 12, 4, 64, 32, bf, False),
    "forty groups": ([(128 * (i % 4), [(1, 20 * i), (1, 7)]) for i in range(40)], 8, 1, 64, 64, hf, True),
    "sixteen rows": ([(512, [(1, 40)] * 4), (1024, [(1, 3), (1, 200), (1, 77)]), (0, [(1, 9)])], 16, 4, 128, 16, bf, True),
    "sixteen rows of drafts": ([(640, [(2, 40), (2, 0)]), (384, [(1, 300), (2, 1)])], 16, 4, 64, 32, hf, True),
    "odd heads": ([(768, [(1, 5), (1, 250), (3, 0)])], 21, 3, 128, 16, bf, True),
    "a hundred heads a key head": ([(256, [(1, 5), (2, 130)])], 100, 1, 64, 16, hf, True),
    "pages of 1024": ([(1024, [(1, 1100), (1, 3)])], 4, 2, 128, 1024, bf, True),
}


@pytest.mark.parametrize("name", CASES)
def test_shared_rows(name):
    families, Hq, Hk, d, ps, dtype, causal = CASES[name]
    p = Family(families, Hq, Hk, d, ps, dtype, seed=len(name), alone_shares=len(name) % 2 == 0)
    assert p.shares()
    o, lse = p.run(causal)
    p.check(o, lse, causal)
    # The same sizes as they are: some of these calls do not share.
    p.check(*p.run(causal, max_seqlen_k=max(p.lens)), causal)
    again = p.run(causal)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("name", ["two answers", "drafts", "chunks", "sixteen rows of drafts"])
def test_wide_scores_and_wrong_hints(name):
    families, Hq, Hk, d, ps, dtype, causal = CASES[name]
    p = Family(families, Hq, Hk, d, ps, dtype, sigma=3.0)
    p.check(*p.run(causal, scale=0.02), causal, scale=0.02)
    # The hint only chooses a kernel.
    p = Family(families, Hq, Hk, d, ps, dtype)
    for hint in (1, 4, 1 << 20):
        p.check(*p.run(causal, max_group_q=hint), causal)


def test_even_steps_without_offsets():
    p = Family([(512, [(2, 40), (2, 300)]), (128, [(2, 0)]), (256, [(2, 7), (2, 8), (2, 9)])], 16, 4, 64, 32, bf)
    o, lse = p.run(cu=False)
    p.check(o, lse)
    with_cu = p.run()
    assert torch.equal(o, with_cu[0]) and torch.equal(lse, with_cu[1])


@pytest.mark.parametrize("name", ["two answers", "alone and together", "no new tokens", "chunks", "drafts", "sixteen rows"])
@pytest.mark.parametrize("fill", [0xFF, 0x7F, 0x00, 0x05])
def test_whatever_the_workspace_holds(name, fill):
    families, Hq, Hk, d, ps, dtype, _ = CASES[name]
    p = Family(families, Hq, Hk, d, ps, dtype, pad=3)
    o, lse = p.into(fill)
    p.check(o, lse)
    assert (o[sum(p.new):] == 5.0).all() and (lse[:, sum(p.new):] == 5.0).all()  # rows of no sequence


def test_cut_off_and_strided():
    families = [(512, [(4, 40), (2, 300)]), (256, [(1, 7), (3, 8)])]
    p = Family(families, 8, 2, 64, 32, bf)
    o, lse = p.into(0xFF, max_seqlen_q=2)
    kept = torch.tensor([i < 2 for n in p.new for i in range(n)], device=DEV)
    assert (o[~kept] == 5.0).all() and (lse[:, ~kept] == 5.0).all()
    full = p.run()
    # Both within 2^-8 |O| + (2^-10 + 2^-12) A of the same values, |O| and A below 6.
    assert (o[kept].double() - full[0][kept].double()).abs().max() <= 2.0 ** -4
    # O and Q in a wider buffer.
    wide = torch.full((10, 8, 3, 64), 5.0, dtype=bf, device=DEV)
    q, out = wide[:, :, 0], wide[:, :, 2]
    q.copy_(p.q)
    p.q = q
    o, lse = p.into(0xFF, o=out)
    assert torch.equal(out, full[0]) and torch.equal(lse, full[1]) and (wide[:, :, 1] == 5.0).all()


def test_keys_past_the_longest_are_not_seen():
    """max_seqlen_k below the lengths, and below the shared rows of one group: like
    sequences that end there (not causal)."""
    families = [(512, [(1, 40 * i) for i in range(10)]), (768, [(1, 7), (1, 8), (1, 300), (1, 0)])]
    p = Family(families, 32, 32, 128, 64, bf)
    assert p.shares(max_seqlen_k=600)
    cut = p.run(causal=False, max_seqlen_k=600)
    p.lens = [min(m, 600) for m in p.lens]
    p.k, p.v = [x[:600] for x in p.k], [x[:600] for x in p.v]
    p.check(*cut, causal=False)


def test_calls_that_cannot_pay_run_unshared():
    import exact_attention_67_gb300 as ex
    for name in ("two answers", "drafts", "chunks", "nothing shared"):
        families, Hq, Hk, d, ps, dtype, causal = CASES[name]
        p = Family(families, Hq, Hk, d, ps, dtype)
        k = max(p.lens)
        assert not p.shares(max_seqlen_k=k)
        o, lse = p.run(causal, max_seqlen_k=k)
        want = ex.forward_paged(p.q, p.kc, p.vc, p.table, p.seq, p.cu, max(p.new), k, causal=causal)
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_tables_that_break_the_rules_stay_in_bounds():
    """Results are wrong, accesses are not (read in paged_sched.cuh and paged_join.cu:
    sequences, rows, shared rows and slots are clamped or checked)."""
    import exact_attention_67_gb300 as ex
    p = Family([(512, [(1, 40), (2, 300)]), (256, [(1, 7), (3, 8)])], 8, 2, 64, 32, bf)
    for groups in ([0, 9, 4], [5, 2, 4], [-3, 1, 100], [0, 0, 0], [0, 4, 1]):
        p.groups = torch.tensor(groups, dtype=torch.int32, device=DEV)
        for fill in (0xFF, 0x05):
            p.into(fill)
    p.groups = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for prefix in ([1 << 30] * 4, [-(1 << 31)] * 4, [2 ** 31 - 1, 0, 5000, 128]):
        p.prefix = torch.tensor(prefix, dtype=torch.int32, device=DEV)
        p.into(0xFF)
    assert ex.device_error() == 0


@pytest.mark.parametrize("shared", [True, False])
def test_offsets_that_name_tokens_again_and_again(shared):
    """Offsets that go back and forth: their units would weigh past 31 bits (3,000 groups,
    every other one of 4,096 tokens, 514 a token; 2,048 times 16,384 tokens, 514 every
    eight).  Such a line is empty, and the next call is right."""
    import exact_attention_67_gb300 as ex
    B, ps, k, d, Hq = 4096, 1024, 65536, 64, 32
    total = B if shared else 16384
    kc, vc = (torch.randn(64, 1, ps, d, device=DEV).to(bf) for _ in range(2))
    q = torch.randn(total, Hq, d, device=DEV).to(bf)
    table = torch.arange(64, dtype=torch.int32, device=DEV).repeat(B, 1)
    seq = torch.full((B,), k, dtype=torch.int32, device=DEV)
    back = torch.tensor([0, total], dtype=torch.int32, device=DEV).repeat(B)
    if shared:
        prefix = torch.full((B,), k - 128, dtype=torch.int32, device=DEV)
        args = (q, kc, vc, table, seq, back[:3001].contiguous(), prefix, None, 1, k, 1)
        assert ex.attn_fwd_paged_shared_workspace_size(B, 3000, Hq, 1, total, 1, k, 1, d) > ex.attn_fwd_paged_workspace_size(
            B, Hq, 1, total, 1, k, d)
        ex.forward_paged_shared(*args)
    else:
        ex.forward_paged(q, kc, vc, table, seq, back[:B + 1].contiguous(), total, k)
    torch.cuda.synchronize()
    assert ex.device_error() == 0
    p = Family([(256, [(1, 40), (1, 300), (1, 3)])], 8, 2, 64, 32, bf)
    p.check(*p.run())


def test_nan_of_one_sequence_stays_there():
    p = Family([(256, [(1, 40), (1, 300), (1, 3)])], 8, 2, 64, 32, bf)
    want = p.run()
    p.kc[int(p.table[1, 9])] = NAN  # rows of its own
    o, lse = p.run()
    assert o[1].isnan().all() and lse[:, 1].isnan().all()
    for i in (0, 2):
        assert torch.equal(o[i], want[0][i]) and torch.equal(lse[:, i], want[1][:, i])
    p.q[0] = NAN
    o, lse = p.run()
    assert o[0].isnan().all() and torch.equal(o[2], want[0][2]) and torch.equal(lse[:, 2], want[1][:, 2])


def test_captured_on_other_streams_and_replayed():
    import exact_attention_67_gb300 as ex
    a = Family([(512, [(1, 40), (1, 300)]), (256, [(1, 7), (1, 8)])], 8, 2, 64, 32, bf, seed=1)
    b = Family([(128, [(1, 500), (1, 20)]), (768, [(1, 1), (1, 200)])], 8, 2, 64, 32, bf, seed=2)
    want = [p.run(cu=False, max_seqlen_k=1 << 20, max_group_q=2) for p in (a, b)]
    # Two streams at once, each with a workspace of its own.
    torch.cuda.synchronize()
    got = []
    for p in (a, b):
        side = torch.cuda.Stream()
        got.append([ex.forward_paged_shared(p.q, p.kc, p.vc, p.table, p.seq, p.groups, p.prefix, None, 1, 1 << 20, 2, stream=side)
                    for _ in range(3)][-1])
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])
    # A captured call follows its tables: other lengths, pages and groups at replay.
    width, pages = max(a.table.shape[1], b.table.shape[1]), max(a.kc.shape[0], b.kc.shape[0])
    hold = dict(q=torch.zeros_like(a.q), kc=torch.zeros((pages, *a.kc.shape[1:]), dtype=bf, device=DEV), vc=None,
                table=torch.zeros((4, width), dtype=torch.int32, device=DEV), seq=torch.ones_like(a.seq), groups=a.groups.clone(),
                prefix=torch.zeros_like(a.prefix))
    hold["vc"] = torch.zeros_like(hold["kc"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ex.forward_paged_shared(hold["q"], hold["kc"], hold["vc"], hold["table"], hold["seq"], hold["groups"], hold["prefix"], None, 1,
                                      1 << 20, 2)
    for p, w in zip((a, b, a), (*want, want[0])):
        for n in ("q", "seq", "groups", "prefix"):
            hold[n].copy_(getattr(p, n))
        hold["table"][:, : p.table.shape[1]].copy_(p.table)
        hold["kc"][: p.kc.shape[0]].copy_(p.kc)
        hold["vc"][: p.vc.shape[0]].copy_(p.vc)
        graph.replay()
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    assert ex.device_error() == 0


def test_many_calls_in_a_row_and_among_others():
    """The own line's launch begins beside the shared one's: inputs written just before a
    call, and a workspace that the call before has just used, are seen in order."""
    import exact_attention_67_gb300 as ex
    p = Family([(2048, [(1, 100 * i) for i in range(8)])], 32, 8, 128, 16, bf)
    n = ex.attn_fwd_paged_shared_workspace_size(8, 1, 32, 8, 8, *p.sizes().values(), 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    qs = [randn(8, 32, 128, seed=i, dtype=bf) for i in range(6)]
    held, outs = torch.empty_like(p.q), []

    def call(q):
        o, lse = torch.empty_like(p.q), torch.empty(32, 8, device=DEV)
        ex.attn_fwd_paged_shared(q, p.kc, p.vc, o, lse, p.table, p.seq, None, p.groups, p.prefix, *p.sizes().values(), True, 128 ** -0.5, ws)
        return o, lse

    want = []
    for q in qs:
        want.append(call(q))
        torch.cuda.synchronize()
    for q in qs * 3:
        held.copy_(q)
        outs.append(call(held))
    torch.cuda.synchronize()
    for i, (o, lse) in enumerate(outs):
        assert torch.equal(o, want[i % 6][0]) and torch.equal(lse, want[i % 6][1])


def test_among_other_dependent_launches_on_one_workspace():
    """Every kernel may be launched before the stream's last one has ended, and waits for it before it reads or
    writes: this call's lines behind the join of the call before, on the same records and rows; attn_fwd_paged and the
    norms' gradient on the same workspace; the norms into the cache whose rows are read next."""
    import exact_attention_67_gb300 as ex
    p = Family([(2048, [(1, 100 * i) for i in range(8)])], 32, 8, 128, 16, bf)
    plain_sizes = (8, 32, 8, 8, 1, max(p.lens), 128)
    n = max(ex.attn_fwd_paged_shared_workspace_size(8, 1, 32, 8, 8, *p.sizes().values(), 128),
            ex.attn_fwd_paged_workspace_size(*plain_sizes), ex.attn_norm_rotary_backward_workspace_size(1, 8, 128))
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    freq = ex.rotary_frequencies(128)[0]
    pos = torch.tensor(p.lens, dtype=torch.int32, device=DEV) - 1
    gain = 1 + 0.2 * randn(128, seed=1, dtype=torch.float32)
    q, k, v = (torch.empty(8, H, 128, dtype=bf, device=DEV) for H in (32, 8, 8))

    def step(seed):
        q.copy_(randn(8, 32, 128, seed=seed, dtype=bf))
        k.copy_(randn(8, 8, 128, seed=seed + 1, dtype=bf))
        v.copy_(randn(8, 8, 128, seed=seed + 2, dtype=bf))
        q_out, o, plain = (torch.empty_like(q) for _ in range(3))
        lse, plain_lse = (torch.empty(32, 8, device=DEV) for _ in range(2))
        dq, dg = torch.empty_like(q), torch.empty_like(gain)
        ex.attn_cache_append(k, v, p.kc, p.vc, p.table, p.seq, None, q=q, q_out=q_out, inv_freq=freq, q_gain=gain, k_gain=gain)
        for _ in range(2):
            ex.attn_fwd_paged_shared(q_out, p.kc, p.vc, o, lse, p.table, p.seq, None, p.groups, p.prefix, *p.sizes().values(), True,
                                     128 ** -0.5, ws)
        ex.attn_norm_rotary_backward(o, q, dq, None, None, None, pos, freq, gain, None, dg, None, False, 1.0, 1e-6, ws)
        ex.attn_fwd_paged(q_out, p.kc, p.vc, plain, plain_lse, p.table, p.seq, None, 1, max(p.lens), True, 128 ** -0.5, ws)
        ex.attn_fwd_paged_shared(dq, p.kc, p.vc, q_out, lse, p.table, p.seq, None, p.groups, p.prefix, *p.sizes().values(), True,
                                 128 ** -0.5, ws)
        return q_out, o, lse, plain, plain_lse, dq, dg

    want = []
    for i in range(4):
        want.append(step(10 * i))
        torch.cuda.synchronize()
    got = [step(10 * (i % 4)) for i in range(16)]
    torch.cuda.synchronize()
    assert ex.device_error() == 0
    for i, outs in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(outs, want[i % 4]))
    # Behind shared rows and not: within 2^-8 |O| + (2^-10 + 2^-12) A of the same values, |O| and A below 6.
    assert all((w[1].double() - w[3].double()).abs().max() <= 2.0 ** -4 for w in want)


# ---------------------------------------------------------------- together, as a server runs them
@pytest.mark.parametrize("d,Hq,Hk,ps,dtype", [(128, 8, 2, 16, bf), (64, 6, 2, 32, hf)])
def test_prompt_forks_and_next_tokens(d, Hq, Hk, ps, dtype, monkeypatch):
    """A prompt, forks of it, next tokens with norms, rotation, the cache and attention
    behind the shared prompt, in two layers: against attention in 64 bits over what the
    cache holds."""
    import exact_attention_67_gb300 as ex
    from exact_attention_67_gb300 import cache as cache_module
    plain_call = cache_module.forward_paged_shared
    monkeypatch.setattr(cache_module, "forward_paged_shared",
                        lambda *a: plain_call(*a[:9], 1 << 20, *a[10:]))  # max_seqlen_k, so that these sizes share
    layers, prompt = 2, 300
    cache = ex.PagedCache(200, ps, layers, Hk, d, dtype=dtype, share_from=0)
    freq, factor = ex.rotary_frequencies(d)
    qg, kg = (1 + 0.2 * randn(d, seed=i, dtype=torch.float32) for i in (1, 2))
    root = cache.add()
    seed = [10]

    def step_of(seqs, new):
        step = cache.extend(seqs, new, shared=True)
        for layer in range(layers):
            seed[0] += 3
            q, k, v = (randn(step.tokens, H, d, seed=seed[0] + i, dtype=dtype) for i, H in enumerate((Hq, Hk, Hk)))
            plain = ex.norm_rotary(q, None, qg, None, positions(step), freq, factor=factor)
            cache.append(layer, step, k, v, q=q, q_out=q, inv_freq=freq, factor=factor, q_gain=qg, k_gain=kg)
            assert torch.equal(q, plain)
            check(layer, step, q, *cache.attend(layer, step, q))
        return step

    def positions(step):
        at = [p for s, n in zip(step.ids, step.new) for p in range(cache.length(s) - n, cache.length(s))]
        return torch.tensor(at, dtype=torch.int32, device=DEV)

    def check(layer, step, q, o, lse):
        p = Problem.__new__(Problem)
        p.new, p.lens, p.Hq, p.Hk, p.d, p.dtype, p.q = list(step.new), [cache.length(s) for s in step.ids], Hq, Hk, d, dtype, q
        for name, whole in (("k", cache.k_cache(layer)), ("v", cache.v_cache(layer))):
            setattr(p, name, [whole[list(cache.pages(s))].transpose(1, 2).reshape(-1, Hk, d)[:cache.length(s)].double() for s in step.ids])
        p.check(o, lse)

    assert step_of([root], prompt).cu_groups is None
    forks = cache.fork(root, 5)
    other = cache.add()
    step_of([other], 40)
    for i in range(3):
        step = step_of(forks + [other], 1)
        assert step.cu_groups.tolist() == [0, 5, 6] and step.prefix_lens.tolist() == [256] * 5 + [0] and step.max_group_q == 5
    step_of([forks[0], forks[3], other], [4, 1, 2])  # drafts
    cache.truncate(forks[0], prompt + 4)
    more = cache.fork(forks[0], 2)
    cache.free([forks[1], root])
    cache.compact()
    step_of([forks[0], *more, *forks[2:], other], 1)
    # Under a window the step's groups are left aside.
    step = cache.extend([forks[0], *more], 1, shared=True)
    q, k, v = (randn(3, H, d, seed=i, dtype=dtype) for i, H in enumerate((Hq, Hk, Hk)))
    cache.append(0, step, k, v)
    o, lse = cache.attend(0, step, q, window=100)
    want = ex.forward_paged(q, cache.k_cache(0), cache.v_cache(0), step.page_table, step.seqlens, None, 1, step.max_seqlen_k, window=100)
    assert step.cu_groups is not None and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert ex.device_error() == 0
