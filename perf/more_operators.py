"""Cases of the operators on both sides of a paged key/value cache: the norm of each head of queries and keys with the
rotary turn in one pass, its gradient, and the same on the way into the cache; and attention over a cache for a batch
whose sequences share their first pages, which are streamed once for all of them.  `run` computes them either with
elementary torch operations in 32 bits (`own` false) or through the framework's calls (`own` true)."""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # A training step's Q and K of one long sequence.
        {"name": "norm_train", "op": "norm", "grad": False, "B": 1, "N": 8192, "Hq": 32, "Hk": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "start": 0, "layout": "bhnd", "gain": "bf16", "dtype": "bf16"},
        # A short prompt, token-major, a part of each head turned in pairs, an odd length: latency.
        {"name": "norm_short", "op": "norm", "grad": False, "B": 1, "N": 77, "Hq": 24, "Hk": 8, "d": 64, "rot": 20,
         "interleaved": True, "scaling": "linear", "start": 4000, "layout": "bnhd", "gain": "f32", "dtype": "f16"},
        # Gradients of the training step.
        {"name": "norm_grad_train", "op": "norm", "grad": True, "B": 1, "N": 8192, "Hq": 32, "Hk": 8, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "start": 0, "layout": "bhnd", "gain": "bf16", "dtype": "bf16"},
        # Gradients of a batch of odd length, token-major, half of each head turned in pairs, gains kept in 32 bits.
        {"name": "norm_grad_partial", "op": "norm", "grad": True, "B": 3, "N": 1001, "Hq": 16, "Hk": 16, "d": 64, "rot": 32,
         "interleaved": True, "scaling": "yarn", "start": 70000, "layout": "bnhd", "gain": "f32", "dtype": "f16"},
        # One new token of each running sequence, between projection and attention.
        {"name": "append_norm_tokens", "op": "append", "B": 64, "new": 1, "ctx": 8192, "ragged": True, "mix": 1, "Hq": 32, "Hk": 8,
         "d": 128, "page": 16, "rot": 128, "interleaved": False, "scaling": "none", "gain": "bf16", "dtype": "bf16"},
        # Ragged prompts written in one call, beyond the trained length.
        {"name": "append_norm_prompts", "op": "append", "B": 5, "new": 4096, "ctx": 40000, "ragged": True, "mix": 2, "Hq": 32, "Hk": 4,
         "d": 64, "page": 64, "rot": 64, "interleaved": False, "scaling": "yarn", "gain": "f32", "dtype": "bf16"},
        # Two answers to one short prompt, next tokens: latency.
        {"name": "shared_pair", "op": "shared", "groups": 1, "each": 2, "new": 1, "prefix": 512, "own": 40, "ragged": False, "mix": 3,
         "Hq": 32, "Hk": 8, "d": 128, "page": 16, "causal": True, "dtype": "bf16"},
        # Sixteen samples of one prompt, next tokens.
        {"name": "shared_samples", "op": "shared", "groups": 1, "each": 16, "new": 1, "prefix": 8192, "own": 500, "ragged": True, "mix": 4,
         "Hq": 32, "Hk": 8, "d": 128, "page": 16, "causal": True, "dtype": "bf16"},
        # A serving batch: chats behind a few long system prompts, of ragged lengths, eight query heads to a key head.
        {"name": "shared_system", "op": "shared", "groups": 4, "each": 32, "new": 1, "prefix": 16384, "own": 4000, "ragged": True,
         "mix": 5, "Hq": 32, "Hk": 4, "d": 128, "page": 64, "causal": True, "dtype": "bf16"},
        # Drafted tokens of samples checked at once, small heads in a group of three.
        {"name": "shared_verify", "op": "shared", "groups": 3, "each": 12, "new": 5, "prefix": 5000, "own": 900, "ragged": True, "mix": 6,
         "Hq": 24, "Hk": 8, "d": 64, "page": 32, "causal": True, "dtype": "f16"},
        # Questions behind one document, prefilled together.
        {"name": "shared_chunks", "op": "shared", "groups": 1, "each": 6, "new": 400, "prefix": 16384, "own": 0, "ragged": True, "mix": 7,
         "Hq": 32, "Hk": 8, "d": 128, "page": 64, "causal": True, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "shared", "shared", "shared"])
    dtype, d = rng.choice(["bf16", "bf16", "f16"]), rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 2, 3, 4, 5, 7, 8] if Hk < 8 else [1, 2, 4])
    rope = {"rot": rng.choice([d, d, d // 2, 20, 6]), "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "yarn"]),
            "gain": rng.choice([dtype, "f32"])}
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        B = rng.choice([1, 2, 3, 4])
        N = _log(rng, 1, max(2, (1 << 25) // (B * (Hq + Hk) * d)))
        return {"op": op, "grad": rng.random() < 0.5, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, **rope, "start": _log(rng, 1, 1000000),
                "layout": rng.choice(["bhnd", "bnhd"]), "dtype": dtype}
    if op == "append":
        B = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, 16384 // B))
        ctx = max(new, _log(rng, 16, min(100000, (1 << 20) // B)))
        return {"op": op, "B": B, "new": new, "ctx": ctx, "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 20), "Hq": Hq, "Hk": Hk, "d": d,
                "page": page, **rope, "dtype": dtype}
    while True:
        groups = _log(rng, 1, 8)
        if rng.random() < 0.7:
            each, new = _log(rng, 1, 32), rng.choice([1, 1, 1, 2, 5])
        else:
            each, new = _log(rng, 1, 6), _log(rng, 5, 400)
        c = {"op": op, "groups": groups, "each": each, "new": new, "prefix": _log(rng, 1, 16384), "own": _log(rng, 1, 4000) - 1,
             "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 20), "Hq": Hq, "Hk": Hk, "d": d, "page": page,
             "causal": rng.random() < 0.85, "dtype": dtype}
        B, L = groups * each, c["prefix"] + c["own"] + new
        if B * L * Hk * d <= 1 << 30 and B * new * L * Hq * d <= 8e10 and work(c)["bytes"] <= 4e8:
            return c


def _lengths(case):
    """New tokens and lengths (the new tokens included) of the sequences, from the case alone."""
    r, B, new, ctx = random.Random(case["mix"]), case["B"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [new] * B, [ctx] * B
    fresh = [new if new == 1 else r.randint(max(1, new // 4), new) for _ in range(B)]
    lens = [max(n, r.randint(max(1, ctx // 8), ctx)) for n in fresh]
    at = r.randrange(B)
    fresh[at], lens[at] = new, ctx
    return fresh, lens


def _families(case):
    """For each group of sequences its shared rows (whole pages), and for each member (new tokens, rows of its own before them)."""
    r, page = random.Random(case["mix"]), case["page"]
    out = []
    for g in range(case["groups"]):
        if not case["ragged"]:
            out.append((case["prefix"] // page * page, [(case["new"], case["own"])] * case["each"]))
            continue
        first = g == 0  # the largest of everything, the others spread below
        shared = case["prefix"] if first else r.randint(case["prefix"] // 8, case["prefix"])
        count = case["each"] if first else r.randint(1, case["each"])
        members = [(case["new"] if case["new"] == 1 else r.randint(max(1, case["new"] // 4), case["new"]), r.randint(case["own"] // 8, case["own"]))
                   for _ in range(count)]
        if first:
            members[r.randrange(count)] = (case["new"], case["own"])
        out.append((shared // page * page, members))
    return out


def _frequencies(rot, scaling):
    """Radians a token of each pair, and the factor of cos and sin: base 10000, plain; positions divided by 4; or, for 8 times the trained
    length of 8192, slow pairs divided by 8, fast ones kept and those between blended (by the turns that they make over that length)."""
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    f = 10000.0 ** (-i / rot)
    if scaling == "linear":
        return f / 4, 1.0
    if scaling == "yarn":
        turns = 8192 * f / (2 * math.pi)
        keep = ((turns - 1) / (32 - 1)).clamp(0, 1)
        return f / 8 * (1 - keep) + f * keep, 0.1 * math.log(8) + 1
    return f, 1.0


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t, op, d = TYPES[case["dtype"]], case["op"], case["d"]

    def normal(*shape, dtype=t):
        x = torch.empty(shape, dtype=dtype, device=DEV)
        return x.normal_(generator=g)

    def heads(*shape):
        """Projections: rows of one head differ in size."""
        x = normal(*shape)
        return x.mul_(normal(*shape[:-1], 1).mul_(0.7).exp_())

    s = {"case": case}
    if op != "shared":
        f, s["factor"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = f.to(DEV)
        for name in ("q_gain", "k_gain"):
            s[name] = normal(d, dtype=TYPES[case["gain"]]).mul_(0.2).add_(1)
    if op == "norm":
        B, N = case["B"], case["N"]
        for name, H in (("q", case["Hq"]), ("k", case["Hk"])):
            for part, make in (("", heads), ("d", normal)):
                if case["grad"] or not part:
                    s[part + name] = make(B, H, N, d) if case["layout"] == "bhnd" else make(B, N, H, d).transpose(1, 2)
        first = torch.randint(0, case["start"] + 1, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        s["positions"] = first + torch.arange(N, device=DEV, dtype=torch.int32)
        torch.cuda.synchronize()
        return s
    Hk, ps = case["Hk"], case["page"]
    if op == "append":
        fresh, lens = _lengths(case)
        need = [-(-n // ps) for n in lens]
        shared = [0] * len(lens)
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at : at + n]
            at += n
    else:
        families = _families(case)
        fresh = [n for _, members in families for n, _ in members]
        lens = [p + o + n for p, members in families for n, o in members]
        shared = [p if len(members) > 1 else 0 for p, members in families for _ in members]  # one alone shares with none
        need = [-(-n // ps) for n in lens]
        pages = sum(p // ps for p, _ in families) + sum(need) - sum(p // ps * len(m) for p, m in families) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(len(lens), max(need), dtype=torch.int32, device=DEV)
        at = b = 0
        for p, members in families:
            first, at = order[at : at + p // ps], at + p // ps
            for _ in members:
                table[b, : p // ps] = first
                rest = need[b] - p // ps
                table[b, p // ps : need[b]] = order[at : at + rest]
                at, b = at + rest, b + 1
        ends = [0]
        for _, members in families:
            ends.append(ends[-1] + len(members))
        s["cu_groups"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        s["prefix"] = torch.tensor(shared, dtype=torch.int32, device=DEV)
        s["max_group"] = max(sum(fresh[i:j]) for i, j in zip(ends, ends[1:]))
    s["k_cache"], s["v_cache"] = normal(pages, Hk, ps, d), normal(pages, Hk, ps, d)
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
    s["cu"] = torch.tensor([sum(fresh[:b]) for b in range(len(fresh) + 1)], dtype=torch.int32, device=DEV)
    s["max_new"], s["max_len"] = max(fresh), max(lens)
    total = sum(fresh)
    s["q"] = heads(total, case["Hq"], d) if op == "append" else normal(total, case["Hq"], d)
    s["q_out"] = torch.empty_like(s["q"])
    if op == "append":
        s["k"], s["v"] = heads(total, Hk, d), normal(total, Hk, d)
    else:
        s["lse"] = torch.empty(case["Hq"], total, dtype=torch.float32, device=DEV)
        if own:
            import exact_attention_67_gb300 as ex

            n = ex.attn_fwd_paged_shared_workspace_size(len(lens), case["groups"], case["Hq"], Hk, total, s["max_new"], s["max_len"],
                                                        s["max_group"], d)
            s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    return s


# ------------------------------------------------------------------ one pass
def _rotate(x, angle, factor, interleaved, sign=1.0):
    """x [..., d] in 32 bits with its first pairs turned by `angle` [..., rot / 2] (64 bits)."""
    c, s = (angle.cos() * factor).float(), (angle.sin() * (factor * sign)).float()
    rot = 2 * angle.shape[-1]
    a, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack((x1 * c - x2 * s, x2 * c + x1 * s), -1).flatten(-2)
    else:
        x1, x2 = a[..., : rot // 2], a[..., rot // 2 :]
        y = torch.cat((x1 * c - x2 * s, x2 * c + x1 * s), -1)
    return torch.cat((y, rest), -1)


def _inverse_size(x):
    """1 / sqrt(mean of squares + eps) of each row, x in 32 bits."""
    return ((x * x).mean(-1, keepdim=True) + EPS).rsqrt()


def _tokens(s):
    """Sequence, place among its new tokens, and position of every new token."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.bucketize(t, cu[1:], right=True)
    i = t - cu[b]
    return b, i, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _norm(s):
    case = s["case"]
    if own:
        import exact_attention_67_gb300 as ex

        how = dict(positions=s["positions"], inv_freq=s["freq"], interleaved=case["interleaved"], factor=s["factor"], eps=EPS)
        if case["grad"]:
            return ex.norm_rotary_backward(s["dq"], s["dk"], s["q"], s["k"], s["q_gain"], s["k_gain"], **how)
        return ex.norm_rotary(s["q"], s["k"], s["q_gain"], s["k_gain"], **how)
    angle = (s["positions"].double()[..., None] * s["freq"])[:, None]
    if not case["grad"]:
        out = []
        for n in ("q", "k"):
            x = s[n].float()
            x = x * _inverse_size(x) * s[n + "_gain"].float()
            out.append(_rotate(x, angle, s["factor"], case["interleaved"]).to(s[n].dtype))
        return tuple(out)
    grads, gains = [], []
    for n in ("q", "k"):
        x, w = s[n].float(), s[n + "_gain"].float()
        r = _inverse_size(x)
        y = _rotate(s["d" + n].float(), angle, s["factor"], case["interleaved"], -1.0)
        u = x * r
        gains.append((y * u).sum((0, 1, 2), dtype=torch.float64).to(s[n + "_gain"].dtype))
        y = y * w
        grads.append((r * (y - u * (y * u).mean(-1, keepdim=True))).to(s[n].dtype))
    return (*grads, *gains)


def _append(s):
    case = s["case"]
    if own:
        import exact_attention_67_gb300 as ex

        ex.attn_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], None if case["new"] == 1 else s["cu"], q=s["q"],
                             q_out=s["q_out"], inv_freq=s["freq"], interleaved=case["interleaved"], factor=s["factor"], q_gain=s["q_gain"],
                             k_gain=s["k_gain"], eps=EPS)
        return s["q_out"], s["k_cache"], s["v_cache"]
    b, _, p = _tokens(s)
    page = s["table"].long()[b, p // case["page"]]
    angle = (p.double()[:, None] * s["freq"])[:, None]
    turned = []
    for n in ("q", "k"):
        x = s[n].float()
        x = x * _inverse_size(x) * s[n + "_gain"].float()
        turned.append(_rotate(x, angle, s["factor"], case["interleaved"]).to(s[n].dtype))
    s["k_cache"][page, :, p % case["page"]] = turned[1]
    s["v_cache"][page, :, p % case["page"]] = s["v"]
    return turned[0], s["k_cache"], s["v_cache"]


def _shared(s):
    case, scale = s["case"], s["case"]["d"] ** -0.5
    if own:
        import exact_attention_67_gb300 as ex

        even = case["new"] == 1 or not case["ragged"]
        ex.attn_fwd_paged_shared(s["q"], s["k_cache"], s["v_cache"], s["q_out"], s["lse"], s["table"], s["lens"], None if even else s["cu"],
                                 s["cu_groups"], s["prefix"], s["max_new"], s["max_len"], s["max_group"], case["causal"], scale, s["workspace"])
        return s["q_out"], s["lse"]
    # Every sequence's keys gathered from its pages, the shared ones too.
    B, Hq, Hk, d = s["lens"].shape[0], case["Hq"], case["Hk"], case["d"]
    b, i, p = _tokens(s)
    L = s["table"].shape[1] * case["page"]
    at = s["table"].long()
    k = s["k_cache"][at].float().transpose(2, 3).reshape(B, L, Hk, d)
    v = s["v_cache"][at].float().transpose(2, 3).reshape(B, L, Hk, d)
    q = torch.zeros(B, s["max_new"], Hk, Hq // Hk, d, device=DEV)
    q[b, i] = s["q"].float().view(-1, Hk, Hq // Hk, d)
    pos = torch.zeros(B, s["max_new"], dtype=torch.long, device=DEV)
    pos[b, i] = p
    x = torch.einsum("bihgd,blhd->bhgil", q, k) * scale
    j = torch.arange(L, device=DEV)
    seen = (j < s["lens"].long()[:, None, None]).expand(B, s["max_new"], L)
    if case["causal"]:
        seen = seen & (j <= pos[..., None])
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = x.sub_(top.clamp(min=-1e30)).exp_()
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgil,blhd->bihgd", e, v)
    z = z[..., 0].permute(0, 3, 1, 2)  # [B, new, Hk, G]
    o = torch.where(z[..., None] > 0, o / z[..., None], 0.0)
    lse = top[..., 0].permute(0, 3, 1, 2) + z.log()
    return o[b, i].reshape(-1, Hq, d).to(s["q"].dtype), lse[b, i].reshape(-1, Hq).t().contiguous()


def run(state):
    return {"norm": _norm, "append": _append, "shared": _shared}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d, Hq, Hk = case["op"], case["d"], case["Hq"], case["Hk"]
    if op == "norm":
        rows = case["B"] * case["N"] * (Hq + Hk)
        if case["grad"]:  # x and the gradient read, the gradient written
            return {"bytes": 6 * rows * d + 4 * case["B"] * case["N"], "flops": rows * (12 * d + 3 * case["rot"])}
        return {"bytes": 4 * rows * d + 4 * case["B"] * case["N"], "flops": rows * (4 * d + 3 * case["rot"])}
    if op == "append":
        n = sum(_lengths(case)[0])
        return {"bytes": 4 * n * (Hq + 2 * Hk) * d, "flops": n * (Hq + Hk) * (4 * d + 3 * case["rot"])}
    n = keys = pairs = 0
    for p, members in _families(case):
        keys += p
        for f, o in members:
            n += f
            keys += o + f
            pairs += f * (p + o) + (f * (f + 1) // 2 if case["causal"] else f * f)
    return {"bytes": 4 * n * Hq * d + 4 * keys * Hk * d + 4 * n * Hq, "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def _turn(x, pos, freq, factor, interleaved, sign):
    """As a product of complex numbers: (x1 + i x2) * factor * exp(i angle)."""
    n = freq.numel()
    a = sign * pos.double()[..., None] * freq
    w = torch.polar(torch.full_like(a, factor), a)
    y = x.double().clone()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous()) * w
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _unit(x):
    """Rows divided by the root of their mean square (and eps)."""
    x = x.double()
    return x / torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / x.shape[-1] + EPS)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        where = (s["positions"][:, None], s["freq"], s["factor"], case["interleaved"])
        if not case["grad"]:
            return tuple(_turn(_unit(s[n]) * s[n + "_gain"].double(), *where, 1) for n in ("q", "k"))
        # e = x / size with size^2 = |x|^2 / d + eps: the gradient of y.e is y / size - x (y.x) / (d size^3).
        grads, gains = [], []
        for n in ("q", "k"):
            e, x = _unit(s[n]), s[n].double()
            size = torch.sqrt(x.pow(2).mean(-1, keepdim=True) + EPS)
            y = _turn(s["d" + n], *where, -1)
            gains.append(torch.einsum("bhnd,bhnd->d", y, e))
            y = y * s[n + "_gain"].double()
            grads.append(y / size - x * (torch.linalg.vecdot(y, x)[..., None] / (x.shape[-1] * size**3)))
        return (*grads, *gains)
    ps, cu, table = case["page"], s["cu"].tolist(), s["table"].long()
    if op == "append":
        fresh, lens = _lengths(case)
        q, kc, vc = torch.empty_like(s["q"], dtype=torch.float64), s["k_cache"].double(), s["v_cache"].double()
        for b, (f, m) in enumerate(zip(fresh, lens)):
            rows = slice(cu[b], cu[b + 1])
            p = torch.arange(m - f, m, device=DEV)
            page, off = table[b][p // ps], p % ps
            where = (p[:, None], s["freq"], s["factor"], case["interleaved"], 1)
            q[rows] = _turn(_unit(s["q"][rows]) * s["q_gain"].double(), *where)
            kc[page, :, off] = _turn(_unit(s["k"][rows]) * s["k_gain"].double(), *where)
            vc[page, :, off] = s["v"][rows].double()
        return q, kc, vc
    Hq, Hk, d = case["Hq"], case["Hk"], case["d"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full((Hq, o.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    for b, m in enumerate(s["lens"].tolist()):
        rows, f = slice(cu[b], cu[b + 1]), cu[b + 1] - cu[b]
        hidden = torch.arange(m, device=DEV)[None] > torch.arange(m - f, m, device=DEV)[:, None]
        pages = table[b, : -(-m // ps)]
        for h in range(Hk):
            k = s["k_cache"][pages, h].reshape(-1, d)[:m].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:m].double()
            for n in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                x = s["q"][rows, n].double() @ k.T / math.sqrt(d)
                if case["causal"]:
                    x = x.masked_fill(hidden, -math.inf)
                lse[n, rows] = torch.logsumexp(x, -1)
                o[rows, n] = torch.softmax(x, -1) @ v
    return o, lse
