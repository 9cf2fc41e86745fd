"""Throughput of the library's wider entry points on one GPU:

    python -m exact_attention_67_gb300.bench_rows [--iters 20]

One JSON line per case: f16 inputs, the [B, N, H, d] layout, a sliding
window, a packed variable-length batch, decode-shaped forwards, rotary
positions, head norms with them, and the paged cache (append, attention, attention
behind shared rows, page copies).  Inputs are
seeded synthetic bf16/f16 N(0, 1), resident on the device; each figure is the
mean device time of ``iters`` back-to-back calls between two CUDA events after
three warm-up calls (the square cases move far more than L2 per call and are
compute-bound); the decode, rotary and paged cases run the C ABI call on preallocated buffers,
``iters`` calls captured once as a CUDA graph and replayed, so that the
host's per-call work does not show in calls of a few microseconds.  FLOPs count
only visible (query, key) pairs: 4 d per pair forward, 2.5x that backward.
"""
from __future__ import annotations

import argparse
import json
import os

import torch

from . import (attn_cache_append, attn_cache_copy, attn_fwd_decode, attn_fwd_decode_workspace_size, attn_fwd_paged,
               attn_fwd_paged_shared, attn_fwd_paged_shared_workspace_size, attn_fwd_paged_workspace_size, attn_norm_rotary,
               attn_norm_rotary_backward, attn_norm_rotary_backward_workspace_size, attn_rotary, backward,
               backward_varlen, forward, forward_varlen, rotary_frequencies)
from .synth import seeded_bf16

DEV = torch.device("cuda:0")


def _peaks():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "MEASURED_PEAKS.json")
    try:
        with open(path) as f:
            p = json.load(f)
        return float(p["bf16_tflops"]), float(p["hbm_gbs"]), "measured"
    except (OSError, KeyError, ValueError):
        return 1900.0, 6800.0, "fallback"


def _time_ms(fn, iters: int) -> float:
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(iters):
        fn()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / iters


def _pairs(nq: int, nk: int, causal: bool, window: int) -> int:
    """Visible (query, key) pairs of one head, queries at the last nq of nk positions."""
    total = 0
    off = nk - nq
    for i in range(nq):
        p = i + off
        lo = max(0, p - window + 1) if window > 0 else 0
        hi = p if causal else (min(nk - 1, p + window - 1) if window > 0 else nk - 1)
        total += max(0, hi - lo + 1)
    return total


def _square(name, B, H, N, d, causal, dtype, layout="bhnd", window=0, iters=20, peak=1.0):
    x = [seeded_bf16((B, H, N, d), 11 + t, 1.0, dtype) for t in range(4)]
    if layout == "bnhd":
        q, k, v, do = (t.transpose(1, 2).contiguous().to(DEV).transpose(1, 2) for t in x)
    else:
        q, k, v, do = (t.to(DEV) for t in x)
    scale = d ** -0.5
    o, lse = forward(q, k, v, causal, scale, window=window)
    t_f = _time_ms(lambda: forward(q, k, v, causal, scale, window=window), iters)
    t_b = _time_ms(lambda: backward(q, k, v, o, lse, do, causal, scale, window=window), iters)
    f = 4.0 * d * _pairs(N, N, causal, window) * B * H
    return {"case": name, "B": B, "H": H, "N": N, "d": d, "causal": causal, "window": window,
            "dtype": str(dtype).replace("torch.", ""), "layout": layout, "fwd_ms": t_f, "bwd_ms": t_b,
            "fwd_tflops": f / t_f / 1e9, "bwd_tflops": 2.5 * f / t_b / 1e9,
            "fwd_bwd_tflops": 3.5 * f / (t_f + t_b) / 1e9, "fwd_pct_peak": f / t_f / 1e9 / peak * 100}


def _varlen(name, lens, H, d, causal, dtype, iters, peak):
    total = sum(lens)
    q, k, v, do = (seeded_bf16((total, H, d), 21 + t, 1.0, dtype).to(DEV) for t in range(4))
    cu = torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32, device=DEV)
    scale = d ** -0.5
    mx = max(lens)
    o, lse = forward_varlen(q, k, v, cu, mx, causal, scale)
    t_f = _time_ms(lambda: forward_varlen(q, k, v, cu, mx, causal, scale), iters)
    t_b = _time_ms(lambda: backward_varlen(q, k, v, o, lse, do, cu, mx, causal, scale), iters)
    f = 4.0 * d * H * sum(_pairs(n, n, causal, 0) for n in lens)
    return {"case": name, "lens": lens, "H": H, "d": d, "causal": causal, "dtype": str(dtype).replace("torch.", ""),
            "fwd_ms": t_f, "bwd_ms": t_b, "fwd_tflops": f / t_f / 1e9, "bwd_tflops": 2.5 * f / t_b / 1e9,
            "fwd_bwd_tflops": 3.5 * f / (t_f + t_b) / 1e9, "fwd_pct_peak": f / t_f / 1e9 / peak * 100}


def _time_graph_ms(fn, iters: int) -> float:
    """Mean device time of ``iters`` calls captured once as a CUDA graph and
    replayed: back-to-back launches with no host work between them, for
    calls too short to hide the host's per-call overhead."""
    for _ in range(3):
        fn()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(iters):
            fn()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    g.replay()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) / iters


def _decode(name, B, H, Nq, Nk, d, iters, hbm):
    q = seeded_bf16((B, H, Nq, d), 31, 1.0).to(DEV)
    k = seeded_bf16((B, H, Nk, d), 32, 1.0).to(DEV)
    v = seeded_bf16((B, H, Nk, d), 33, 1.0).to(DEV)
    o = torch.empty_like(q)
    lse = torch.empty((B, H, Nq), dtype=torch.float32, device=DEV)
    nws = attn_fwd_decode_workspace_size(B, H, Nq, Nk, d)
    ws = torch.empty(nws, dtype=torch.uint8, device=DEV) if nws else None
    # The C ABI call on preallocated buffers (what forward_decode runs, minus
    # its allocations and watchdog poll), replayed from a CUDA graph.
    t = _time_graph_ms(lambda: attn_fwd_decode(q, k, v, o, lse, True, d ** -0.5, ws), iters)
    nbytes = 2.0 * B * H * Nk * d * 2 + 2.0 * B * H * Nq * d * 2  # K, V read; Q read, O written
    return {"case": name, "B": B, "H": H, "Nq": Nq, "Nk": Nk, "d": d, "causal": True, "ms": t,
            "gbs": nbytes / t / 1e6, "pct_hbm": nbytes / t / 1e6 / hbm * 100,
            "workspace_bytes": attn_fwd_decode_workspace_size(B, H, Nq, Nk, d)}


def _rotary(name, B, N, Hq, Hk, d, iters, hbm):
    q, k = (seeded_bf16((B, h, N, d), 41 + h, 1.0).to(DEV) for h in (Hq, Hk))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freq, _ = rotary_frequencies(d)
    t = _time_graph_ms(lambda: attn_rotary(q, qo, k, ko, pos, freq), iters)
    nbytes = 4.0 * B * N * (Hq + Hk) * d  # read and written
    return {"case": name, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, "ms": t, "gbs": nbytes / t / 1e6,
            "pct_hbm": nbytes / t / 1e6 / hbm * 100}


def _norm_rotary(name, B, N, Hq, Hk, d, iters, hbm):
    """The norms with the turn, and their gradient."""
    q, k, dq, dk = (seeded_bf16((B, h, N, d), 61 + i, 1.0).to(DEV) for i, h in enumerate((Hq, Hk, Hq, Hk)))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    gains = [torch.ones(d, dtype=torch.bfloat16, device=DEV) for _ in range(4)]
    pos = torch.arange(N, dtype=torch.int32, device=DEV)
    freq, _ = rotary_frequencies(d)
    ws = torch.empty(attn_norm_rotary_backward_workspace_size(B, N, d), dtype=torch.uint8, device=DEV)
    t_f = _time_graph_ms(lambda: attn_norm_rotary(q, qo, k, ko, pos, freq, *gains[:2]), iters)
    t_b = _time_graph_ms(lambda: attn_norm_rotary_backward(dq, q, qo, dk, k, ko, pos, freq, *gains, False, 1.0, 1e-6, ws), iters)
    nbytes = 4.0 * B * N * (Hq + Hk) * d  # read and written; the gradient reads twice that
    return {"case": name, "B": B, "N": N, "Hq": Hq, "Hk": Hk, "d": d, "ms": t_f, "bwd_ms": t_b, "gbs": nbytes / t_f / 1e6,
            "pct_hbm": nbytes / t_f / 1e6 / hbm * 100, "bwd_gbs": 1.5 * nbytes / t_b / 1e6,
            "bwd_pct_hbm": 1.5 * nbytes / t_b / 1e6 / hbm * 100}


def _shared(name, prefix, own, Hq, Hk, d, ps, iters, hbm):
    """Next tokens of sequences whose first ``prefix`` rows are on the same pages, with
    ``own`` rows each behind them; and the same without sharing the reads."""
    B, lens = len(own), [prefix + n for n in own]
    first, width = prefix // ps, max(-(-n // ps) for n in lens)
    pages = first + B * (width - first)
    kc, vc = (seeded_bf16((pages, Hk, ps, d), 71 + t, 1.0).to(DEV) for t in range(2))
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32)
    table = torch.cat((order[:first].expand(B, first), order[first:].view(B, width - first)), 1).contiguous().to(DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    groups = torch.tensor([0, B], dtype=torch.int32, device=DEV)
    shared = torch.full((B,), prefix, dtype=torch.int32, device=DEV)
    q = seeded_bf16((B, Hq, d), 73, 1.0).to(DEV)
    o, lse = torch.empty_like(q), torch.empty((Hq, B), dtype=torch.float32, device=DEV)
    ws = torch.empty(attn_fwd_paged_shared_workspace_size(B, 1, Hq, Hk, B, 1, max(lens), B, d), dtype=torch.uint8, device=DEV)
    t = _time_graph_ms(lambda: attn_fwd_paged_shared(q, kc, vc, o, lse, table, seq, None, groups, shared, 1, max(lens), B, True,
                                                     d ** -0.5, ws), iters)
    plain = torch.empty(attn_fwd_paged_workspace_size(B, Hq, Hk, B, 1, max(lens), d), dtype=torch.uint8, device=DEV)
    t_p = _time_graph_ms(lambda: attn_fwd_paged(q, kc, vc, o, lse, table, seq, None, 1, max(lens), True, d ** -0.5, plain), iters)
    nbytes = 4.0 * (prefix + sum(own)) * Hk * d + 4.0 * B * Hq * d
    return {"case": name, "B": B, "prefix": prefix, "keys": prefix + sum(own), "Hq": Hq, "Hk": Hk, "d": d, "page_size": ps, "ms": t,
            "unshared_ms": t_p, "gbs": nbytes / t / 1e6, "pct_hbm": nbytes / t / 1e6 / hbm * 100}


def _paged(name, lens, new, Hq, Hk, d, ps, iters, peak, hbm):
    """Append and attention of ``new`` tokens of sequences of the given lengths."""
    B, width = len(lens), max(-(-n // ps) for n in lens)
    pages = B * width
    kc, vc = (seeded_bf16((pages, Hk, ps, d), 51 + t, 1.0).to(DEV) for t in range(2))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(5)).to(torch.int32).view(B, width).to(DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)
    total = B * new
    q, k, v = (seeded_bf16((total, h, d), 53 + i, 1.0).to(DEV) for i, h in enumerate((Hq, Hk, Hk)))
    qo, o, lse = torch.empty_like(q), torch.empty_like(q), torch.empty((Hq, total), dtype=torch.float32, device=DEV)
    freq, _ = rotary_frequencies(d)
    ws = torch.empty(attn_fwd_paged_workspace_size(B, Hq, Hk, total, new, max(lens), d), dtype=torch.uint8, device=DEV)
    t_a = _time_graph_ms(lambda: attn_cache_append(k, v, kc, vc, table, seq, None, q, qo, freq), iters)
    t = _time_graph_ms(lambda: attn_fwd_paged(qo, kc, vc, o, lse, table, seq, None, new, max(lens), True, d ** -0.5, ws), iters)
    nbytes = 4.0 * sum(lens) * Hk * d + 4.0 * total * Hq * d
    f = 4.0 * d * Hq * sum(_pairs(new, n, True, 0) for n in lens)
    return {"case": name, "B": B, "new": new, "keys": sum(lens), "Hq": Hq, "Hk": Hk, "d": d, "page_size": ps, "append_ms": t_a,
            "ms": t, "gbs": nbytes / t / 1e6, "pct_hbm": nbytes / t / 1e6 / hbm * 100, "tflops": f / t / 1e9,
            "pct_peak": f / t / 1e9 / peak * 100}


def _copy(name, slabs, pages, copies, page_bytes, iters, hbm):
    pool = torch.zeros((slabs, pages, page_bytes), dtype=torch.uint8, device=DEV)
    order = torch.randperm(pages, generator=torch.Generator().manual_seed(6)).to(torch.int32)
    src, dst = order[:copies].clone(), order[copies: 2 * copies].clone()
    t = _time_graph_ms(lambda: attn_cache_copy(pool, src, dst), iters)
    nbytes = 2.0 * slabs * copies * page_bytes
    return {"case": name, "slabs": slabs, "pages": pages, "copies": copies, "page_bytes": page_bytes, "ms": t,
            "gbs": nbytes / t / 1e6, "pct_hbm": nbytes / t / 1e6 / hbm * 100}


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--iters", type=int, default=20)
    a = ap.parse_args(argv)
    peak, hbm, src = _peaks()
    rows = [
        _square("bf16 [B,H,N,d] (reference point)", 1, 16, 8192, 128, True, torch.bfloat16, iters=a.iters, peak=peak),
        _square("f16 [B,H,N,d]", 1, 16, 8192, 128, True, torch.float16, iters=a.iters, peak=peak),
        _square("bf16 [B,N,H,d]", 1, 16, 8192, 128, True, torch.bfloat16, layout="bnhd", iters=a.iters, peak=peak),
        _square("bf16 sliding window 1024", 1, 16, 8192, 128, True, torch.bfloat16, window=1024, iters=a.iters,
                peak=peak),
        _varlen("bf16 packed varlen", [8192, 4096, 4096, 2048, 1024, 512, 256, 128] * 2, 16, 128, True,
                torch.bfloat16, a.iters, peak),
        _decode("decode Nq=1", 4, 32, 1, 32768, 128, a.iters, hbm),
        _decode("decode Nq=1, one head", 1, 1, 1, 131072, 128, a.iters, hbm),
        _decode("decode Nq=16", 8, 16, 16, 16384, 128, a.iters, hbm),
        _rotary("rotary", 1, 32768, 16, 16, 128, a.iters, hbm),
        _norm_rotary("head norms with rotary", 1, 32768, 16, 16, 128, a.iters, hbm),
        _shared("paged decode behind shared rows", 16384, [64 * (i + 1) for i in range(32)], 32, 8, 128, 16, a.iters, hbm),
        _paged("paged decode", [32768] * 4, 1, 32, 32, 128, 64, a.iters, peak, hbm),
        _paged("paged decode, shared key heads, mixed lengths", [512 * (i + 1) for i in range(32)], 1, 32, 4, 128, 16,
               a.iters, peak, hbm),
        _paged("paged chunk", [32768], 2048, 32, 8, 128, 64, a.iters, peak, hbm),
        _copy("page copies", 32, 4096, 1500, 32768, a.iters, hbm),
    ]
    for r in rows:
        r["peak_source"] = src
        print(json.dumps(r))


if __name__ == "__main__":
    main()
