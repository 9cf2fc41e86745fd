"""Cases of the operators around a paged key/value cache: rotary positions and their gradient, appending new tokens to
the cache, attention over it, and copying its pages.  `run` computes them either with elementary torch operations in
32 bits (`own` false) or through the framework's calls (`own` true)."""
import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # A training step's Q and K of one long sequence, every element rotated.
        {"name": "rotary_train", "op": "rotary", "grad": False, "B": 1, "N": 8192, "Hq": 16, "Hk": 16, "d": 128, "rot": 128,
         "interleaved": False, "scaling": "none", "start": 0, "layout": "bhnd", "dtype": "bf16"},
        # Gradients of a batch with shared key heads, half of each head rotated in pairs, an odd length, token-major tensors.
        {"name": "rotary_grad_partial", "op": "rotary", "grad": True, "B": 4, "N": 4095, "Hq": 32, "Hk": 8, "d": 64, "rot": 32,
         "interleaved": True, "scaling": "yarn", "start": 70000, "layout": "bnhd", "dtype": "f16"},
        # One new token of each running sequence, the step between projection and attention when serving.
        {"name": "append_tokens", "op": "append", "B": 64, "new": 1, "ctx": 8192, "ragged": True, "mix": 1, "Hq": 32, "Hk": 8, "d": 128,
         "page": 16, "rot": 128, "interleaved": False, "scaling": "none", "dtype": "bf16"},
        # Prompts written in one call: ragged chunks, positions beyond the trained length.
        {"name": "append_prompts", "op": "append", "B": 5, "new": 4096, "ctx": 40000, "ragged": True, "mix": 2, "Hq": 32, "Hk": 8, "d": 128,
         "page": 64, "rot": 64, "interleaved": True, "scaling": "yarn", "dtype": "bf16"},
        # One user's next token after a short prompt: latency.
        {"name": "decode_one", "op": "attend", "B": 1, "new": 1, "ctx": 777, "ragged": False, "mix": 3, "Hq": 32, "Hk": 8, "d": 128,
         "page": 16, "window": 0, "causal": True, "dtype": "bf16"},
        # A batch of next tokens over long contexts, a key head for each query head.
        {"name": "decode_long", "op": "attend", "B": 4, "new": 1, "ctx": 32768, "ragged": False, "mix": 4, "Hq": 32, "Hk": 32, "d": 128,
         "page": 64, "window": 0, "causal": True, "dtype": "bf16"},
        # A serving batch of mixed lengths, eight query heads to a key head.
        {"name": "decode_ragged", "op": "attend", "B": 48, "new": 1, "ctx": 16384, "ragged": True, "mix": 5, "Hq": 32, "Hk": 4, "d": 128,
         "page": 16, "window": 0, "causal": True, "dtype": "bf16"},
        # Checking a few drafted tokens of each sequence at once, small heads in a group of three.
        {"name": "verify_d64", "op": "attend", "B": 16, "new": 5, "ctx": 5000, "ragged": True, "mix": 6, "Hq": 24, "Hk": 8, "d": 64,
         "page": 32, "window": 0, "causal": True, "dtype": "f16"},
        # Ragged chunks of prompts under a sliding window, an odd group.
        {"name": "chunk_window", "op": "attend", "B": 6, "new": 600, "ctx": 5000, "ragged": True, "mix": 7, "Hq": 20, "Hk": 4, "d": 64,
         "page": 16, "window": 1024, "causal": True, "dtype": "bf16"},
        # A long prompt's chunk near its end.
        {"name": "chunk_long", "op": "attend", "B": 1, "new": 2048, "ctx": 32768, "ragged": False, "mix": 8, "Hq": 32, "Hk": 8, "d": 128,
         "page": 64, "window": 0, "causal": True, "dtype": "bf16"},
        # Last pages of forked sequences, copied in every layer before they are written to.
        {"name": "copy_fork", "op": "copy", "slabs": 64, "pages": 256, "copies": 7, "Hk": 8, "d": 128, "page": 16, "dtype": "bf16"},
        # A fragmented cache moved together.
        {"name": "copy_compact", "op": "copy", "slabs": 32, "pages": 4096, "copies": 1500, "Hk": 8, "d": 128, "page": 16, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rotary", "append", "attend", "attend", "copy"])
    dtype, d = rng.choice(["bf16", "bf16", "f16"]), rng.choice([64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    Hq = Hk * rng.choice([1, 2, 3, 4, 5, 7, 8] if Hk < 8 else [1, 2, 4])
    rope = {"rot": rng.choice([d, d, d // 2, 20, 6]), "interleaved": rng.random() < 0.5, "scaling": rng.choice(["none", "linear", "yarn"])}
    if op == "rotary":
        B = rng.choice([1, 2, 3, 4])
        N = _log(rng, 1, max(2, (1 << 25) // (B * (Hq + Hk) * d)))
        return {"op": op, "grad": rng.random() < 0.5, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, **rope, "start": _log(rng, 1, 1000000),
                "layout": rng.choice(["bhnd", "bnhd"]), "dtype": dtype}
    page = rng.choice([16, 32, 64, 128])
    if op == "copy":
        slabs, pages = rng.choice([2, 8, 24, 64]), _log(rng, 64, 2048)
        page = rng.choice([16, 32])
        most = max(2, min(pages // 2 - 1, (1 << 30) // (slabs * Hk * page * d * 2)))
        return {"op": op, "slabs": slabs, "pages": pages, "copies": _log(rng, 1, most), "Hk": Hk, "d": d, "page": page, "dtype": dtype}
    if op == "append":
        B = _log(rng, 1, 128)
        new = 1 if rng.random() < 0.4 else _log(rng, 1, max(2, 16384 // B))
        ctx = max(new, _log(rng, 16, min(100000, (1 << 20) // B)))
        return {"op": op, "B": B, "new": new, "ctx": ctx, "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 20), "Hq": Hq, "Hk": Hk, "d": d,
                "page": page, **rope, "dtype": dtype}
    while True:
        if rng.random() < 0.5:
            B, new = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 4])
        else:
            B, new = _log(rng, 1, 8), _log(rng, 5, 2048)
        c = {"op": op, "B": B, "new": new, "ctx": max(new, _log(rng, 1, 32768)), "ragged": rng.random() < 0.7, "mix": rng.randrange(1 << 20),
             "Hq": Hq, "Hk": Hk, "d": d, "page": page, "window": rng.choice([0, 0, 0, 127, 1000]), "causal": rng.random() < 0.85, "dtype": dtype}
        if c["B"] * c["ctx"] * Hk * d * 4 <= 1 << 31 and c["B"] * c["new"] * c["ctx"] * Hq * d * 4 <= 1e12:
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
    t, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape):
        x = torch.empty(shape, dtype=t, device=DEV)
        return x.normal_(generator=g)

    s = {"case": case}
    if op == "rotary":
        B, N, d = case["B"], case["N"], case["d"]
        for name, H in (("q", case["Hq"]), ("k", case["Hk"])):
            s[name] = normal(B, H, N, d) if case["layout"] == "bhnd" else normal(B, N, H, d).transpose(1, 2)
        first = torch.randint(0, case["start"] + 1, (B, 1), generator=g, device=DEV, dtype=torch.int32)
        s["positions"] = first + torch.arange(N, device=DEV, dtype=torch.int32)
    elif op == "copy":
        r = random.Random(seed)
        s["pool"] = normal(case["slabs"], case["pages"], case["Hk"], case["page"], case["d"])
        picked = r.sample(range(case["pages"]), 2 * case["copies"])
        s["src"] = torch.tensor(picked[: case["copies"]], dtype=torch.int32)  # page lists are kept on the host
        s["dst"] = torch.tensor(picked[case["copies"] :], dtype=torch.int32)
        return s
    else:
        fresh, lens = _lengths(case)
        B, Hk, d, ps = case["B"], case["Hk"], case["d"], case["page"]
        need = [-(-n // ps) for n in lens]
        pages = sum(need) + 3
        order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.zeros(B, max(need), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at : at + n]
            at += n
        s["k_cache"], s["v_cache"] = normal(pages, Hk, ps, d), normal(pages, Hk, ps, d)
        s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["cu"] = torch.tensor([0] + [sum(fresh[: b + 1]) for b in range(B)], dtype=torch.int32, device=DEV)
        s["max_new"], s["max_len"] = max(fresh), max(lens)
        total = sum(fresh)
        s["q"] = normal(total, case["Hq"], d)
        s["q_out"] = torch.empty_like(s["q"])
        if op == "append":
            s["k"], s["v"] = normal(total, Hk, d), normal(total, Hk, d)
        else:
            s["lse"] = torch.empty(case["Hq"], total, dtype=torch.float32, device=DEV)
            if own:
                import exact_attention_67_gb300 as ex

                n = ex.attn_fwd_paged_workspace_size(B, case["Hq"], Hk, total, s["max_new"], s["max_len"], d)
                s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    if op != "attend":
        f, s["factor"] = _frequencies(case["rot"], case["scaling"])
        s["freq"] = f.to(DEV)
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


def _tokens(s):
    """Sequence, place among its new tokens, and position of every new token."""
    cu = s["cu"].long()
    t = torch.arange(s["q"].shape[0], device=DEV)
    b = torch.bucketize(t, cu[1:], right=True)
    i = t - cu[b]
    return b, i, s["lens"].long()[b] - (cu[b + 1] - cu[b]) + i


def _rotary(s):
    case = s["case"]
    if own:
        import exact_attention_67_gb300 as ex

        f = ex.rotary_backward if case["grad"] else ex.rotary
        return f(s["q"], s["k"], s["positions"], s["freq"], interleaved=case["interleaved"], factor=s["factor"])
    angle = (s["positions"].double()[..., None] * s["freq"])[:, None]
    sign = -1.0 if case["grad"] else 1.0
    q, k = (_rotate(x.float(), angle, s["factor"], case["interleaved"], sign).to(x.dtype) for x in (s["q"], s["k"]))
    return q, k


def _append(s):
    case = s["case"]
    if own:
        import exact_attention_67_gb300 as ex

        ex.attn_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], None if case["new"] == 1 else s["cu"], q=s["q"],
                             q_out=s["q_out"], inv_freq=s["freq"], interleaved=case["interleaved"], factor=s["factor"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    b, _, p = _tokens(s)
    page = s["table"].long()[b, p // case["page"]]
    angle = (p.double()[:, None] * s["freq"])[:, None]
    q = _rotate(s["q"].float(), angle, s["factor"], case["interleaved"]).to(s["q"].dtype)
    s["k_cache"][page, :, p % case["page"]] = _rotate(s["k"].float(), angle, s["factor"], case["interleaved"]).to(q.dtype)
    s["v_cache"][page, :, p % case["page"]] = s["v"]
    return q, s["k_cache"], s["v_cache"]


def _attend(s):
    case, scale = s["case"], s["case"]["d"] ** -0.5
    if own:
        import exact_attention_67_gb300 as ex

        ex.attn_fwd_paged(s["q"], s["k_cache"], s["v_cache"], s["q_out"], s["lse"], s["table"], s["lens"], s["cu"], s["max_new"], s["max_len"],
                          case["causal"], scale, s["workspace"], window=case["window"])
        return s["q_out"], s["lse"]
    B, Hq, Hk, d, W = case["B"], case["Hq"], case["Hk"], case["d"], case["window"]
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
    if W:
        seen = seen & (pos[..., None] - j < W) & (j - pos[..., None] < W)
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    e = x.sub_(top.clamp(min=-1e30)).exp_()
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgil,blhd->bihgd", e, v)
    z = z[..., 0].permute(0, 3, 1, 2)  # [B, new, Hk, G]
    o = torch.where(z[..., None] > 0, o / z[..., None], 0.0)
    lse = top[..., 0].permute(0, 3, 1, 2) + z.log()
    return o[b, i].reshape(-1, Hq, d).to(s["q"].dtype), lse[b, i].reshape(-1, Hq).t().contiguous()


def _copy(s):
    if own:
        import exact_attention_67_gb300 as ex

        ex.attn_cache_copy(s["pool"], s["src"], s["dst"])
        return s["pool"]
    src, dst = s["src"].to(DEV), s["dst"].to(DEV)
    s["pool"][:, dst.long()] = s["pool"][:, src.long()]
    return s["pool"]


def run(state):
    return {"rotary": _rotary, "append": _append, "attend": _attend, "copy": _copy}[state["case"]["op"]](state)


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    op, d = case["op"], case["d"]
    if op == "rotary":
        n = case["B"] * case["N"]
        return {"bytes": 4 * n * (case["Hq"] + case["Hk"]) * d + 4 * n, "flops": 3 * n * (case["Hq"] + case["Hk"]) * case["rot"]}
    if op == "copy":
        return {"bytes": 4 * case["copies"] * case["slabs"] * case["Hk"] * case["page"] * d, "flops": 0}
    fresh, lens = _lengths(case)
    Hq, Hk, n = case["Hq"], case["Hk"], sum(fresh)
    if op == "append":
        return {"bytes": 4 * n * (Hq + 2 * Hk) * d, "flops": 3 * n * (Hq + Hk) * case["rot"]}
    W, pairs, keys = case["window"], 0, 0
    for f, m in zip(fresh, lens):
        lo = max(0, m - f - W + 1) if W else 0
        keys += m - lo
        for p in range(m - f, m):
            end = p + 1 if case["causal"] else min(m, p + W) if W else m
            pairs += end - (max(0, p - W + 1) if W else 0)
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


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rotary":
        sign = -1 if case["grad"] else 1
        return tuple(_turn(s[n], s["positions"][:, None], s["freq"], s["factor"], case["interleaved"], sign) for n in ("q", "k"))
    if op == "copy":
        pool = s["pool"].double()
        pool[:, s["dst"].to(DEV).long()] = s["pool"][:, s["src"].to(DEV).long()].double()
        return pool
    fresh, lens = _lengths(case)
    ps, cu, table = case["page"], s["cu"].tolist(), s["table"].long()
    if op == "append":
        q, kc, vc = torch.empty_like(s["q"], dtype=torch.float64), s["k_cache"].double(), s["v_cache"].double()
        for b, (f, m) in enumerate(zip(fresh, lens)):
            rows = slice(cu[b], cu[b + 1])
            p = torch.arange(m - f, m, device=DEV)
            page, off = table[b][p // ps], p % ps
            q[rows] = _turn(s["q"][rows], p[:, None], s["freq"], s["factor"], case["interleaved"], 1)
            kc[page, :, off] = _turn(s["k"][rows], p[:, None], s["freq"], s["factor"], case["interleaved"], 1)
            vc[page, :, off] = s["v"][rows].double()
        return q, kc, vc
    Hq, Hk, d, W = case["Hq"], case["Hk"], case["d"], case["window"]
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.full((Hq, o.shape[0]), -math.inf, dtype=torch.float64, device=DEV)
    for b, (f, m) in enumerate(zip(fresh, lens)):
        rows = slice(cu[b], cu[b + 1])
        pos, j = torch.arange(m - f, m, device=DEV)[:, None], torch.arange(m, device=DEV)[None]
        hidden = torch.zeros(f, m, dtype=torch.bool, device=DEV)
        if case["causal"]:
            hidden |= j > pos
        if W:
            hidden |= (j - pos).abs() >= W
        pages = table[b, : -(-m // ps)]
        for h in range(Hk):
            k = s["k_cache"][pages, h].reshape(-1, d)[:m].double()
            v = s["v_cache"][pages, h].reshape(-1, d)[:m].double()
            for n in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                x = (s["q"][rows, n].double() @ k.T / math.sqrt(d)).masked_fill(hidden, -math.inf)
                lse[n, rows] = torch.logsumexp(x, -1)
                o[rows, n] = torch.softmax(x, -1).nan_to_num(0.0) @ v
    return o, lse
