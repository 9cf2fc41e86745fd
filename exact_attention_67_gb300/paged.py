"""Operators around a paged key/value cache: ctypes binding of the C ABI's
rotary, cache and paged-attention calls (include/exattn.h; the same names,
argument marshalling only), and the helpers on top of them.

A cache is a pair of [num_pages, Hkv, page_size, d] views (d contiguous; a
token-major [num_pages, page_size, Hkv, d] tensor passes as
``x.transpose(1, 2)``), a page table int32 [B, max_pages] and lengths int32 [B]
on the device.  New tokens are packed [total, H, d] tensors with offsets
``cu_seqlens`` int32 [B + 1], or ``cu_seqlens=None`` when every sequence has
total / B of them.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _lib
from ._lib import _DTYPES, _check, Strides, load, watchdog_check, watchdog_poll

_NO_STRIDES = Strides(0, 0, 0)
_raw_stream = torch._C._cuda_getCurrentRawStream


# The calls here are made once a layer and token when serving, on kernels of a
# few microseconds, so the marshalling is kept short: each tensor's type, shape,
# strides and device are read once (a call took 27 us on the host with the
# library's other helpers, of which the C call is 4 to 7).
def _operand(t, name: str, dims: int):
    """Shape and strides of a bf16/f16 view with `dims` axes, d contiguous."""
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    shape, st = t.shape, t.stride()
    if len(shape) != dims:
        raise ValueError(f"{name} must have {dims} axes, got {tuple(shape)}")
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: the d axis must be contiguous (stride 1), got stride {st[-1]}")
    return shape, st


def _like(t, name: str, shape, dtype):
    """Strides of a view that has to have this shape and type."""
    sh, st = _operand(t, name, len(shape))
    if sh != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {list(shape)} of {dtype}, got {list(sh)} of {t.dtype}")
    return st


def _on(first, *others) -> int:
    """The CUDA device of all the given tensors (None entries skipped)."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("all device operands must be CUDA tensors")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"operands are on different devices ({first.device} and {t.device})")
    return dev


def _call(fn, dev: int, stream, *args) -> None:
    """One C call on device ``dev``, made current if it is not, the stream last."""
    if stream is None:
        stream = _raw_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if dev == torch.cuda.current_device():
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        _check(status)


def _int32(t, name: str, shape):
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if shape and shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis must be contiguous")


def _frequencies(inv_freq):
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous float64 tensor [rot_dim / 2] (rotary_frequencies)")
    return 2 * inv_freq.numel()


# ---------------------------------------------------------------- rotary positions
def rotary_frequencies(rot_dim: int, base: float = 10000.0, *, linear: float = 1.0, yarn: float = 1.0,
                       trained_length: int = 8192, slow_turns: float = 1.0, fast_turns: float = 32.0, device="cuda"):
    """Frequencies float64 [rot_dim / 2] (radians a token) and the factor of cos
    and sin, for ``rotary``: f_i = base^(-2 i / rot_dim), and for contexts
    beyond the trained length
      * ``linear`` = s > 1: positions divided by s (every f_i / s);
      * ``yarn`` = s > 1: pairs that make fewer than ``slow_turns`` turns over
        ``trained_length`` tokens are divided by s, those that make more than
        ``fast_turns`` are kept, those between are blended linearly in their
        turns; the factor is 0.1 ln s + 1.
    A changed ``base`` is the remaining common scaling."""
    if rot_dim < 2 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and at least 2, got {rot_dim}")
    if not (base > 0 and linear > 0 and yarn > 0) or (linear != 1.0 and yarn != 1.0):
        raise ValueError("base, linear and yarn must be positive, and only one of linear and yarn given")
    if not fast_turns > slow_turns:
        raise ValueError("fast_turns must exceed slow_turns")
    f = torch.tensor(float(base), dtype=torch.float64) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64) / rot_dim)
    factor = 1.0
    if linear != 1.0:
        f = f / linear
    if yarn != 1.0:
        turns = trained_length * f / (2 * math.pi)
        keep = ((turns - slow_turns) / (fast_turns - slow_turns)).clamp(0, 1)
        f = f / yarn * (1 - keep) + f * keep
        factor = 0.1 * math.log(yarn) + 1.0 if yarn > 1.0 else 1.0
    return f.to(device), factor


def attn_rotary(q, q_out, k, k_out, positions, inv_freq, interleaved: bool = False, inverse: bool = False,
                factor: float = 1.0, stream=None) -> None:
    """C ``attn_rotary``: q, q_out [B, Hq, N, d] and k, k_out [B, Hk, N, d] views of
    one 16-bit type (k, k_out may be None); positions int32 [N] or [B, N];
    inv_freq float64 [rot_dim / 2].  An output may be its own input."""
    shape, sq = _operand(q, "q", 4)
    B, Hq, N, d = shape
    dtype = q.dtype
    so = _like(q_out, "q_out", shape, dtype)
    if (k is None) != (k_out is None):
        raise ValueError("k and k_out go together")
    Hk, kp, kop, sk, sko = 0, None, None, _NO_STRIDES, _NO_STRIDES
    if k is not None:
        kshape, ks = _operand(k, "k", 4)
        Hk = kshape[1]
        if kshape != (B, Hk, N, d) or k.dtype != dtype:
            raise ValueError("k must be [B, Hk, N, d] like q, of one dtype")
        ko = _like(k_out, "k_out", kshape, dtype)
        kp, kop, sk, sko = k.data_ptr(), k_out.data_ptr(), Strides(ks[0], ks[1], ks[2]), Strides(ko[0], ko[1], ko[2])
    if positions.dim() == 1:
        _int32(positions, "positions", (N,))
        ps = 0
    else:
        _int32(positions, "positions", (B, N))
        ps = positions.stride(0) if B > 1 else 0
    rot = _frequencies(inv_freq)
    _call((_lib._lib or load()).attn_rotary, _on(q, q_out, k, k_out, positions, inv_freq), stream, _DTYPES[dtype],
          q.data_ptr(), Strides(sq[0], sq[1], sq[2]), q_out.data_ptr(), Strides(so[0], so[1], so[2]), Hq, kp, sk, kop, sko,
          Hk, positions.data_ptr(), ps, inv_freq.data_ptr(), rot, 1 if interleaved else 0, 1 if inverse else 0, factor, B,
          N, d)


def _rotary(q, k, positions, inv_freq, interleaved, inverse, factor, stream):
    def four(x):  # packed [total, H, d] as one batch
        return x.transpose(0, 1).unsqueeze(0) if x is not None and x.dim() == 3 else x

    if k is not None and k.dim() != q.dim():
        raise ValueError("q and k must both be [B, H, N, d], or both packed [total, H, d]")
    qo, ko = torch.empty_like(q), None if k is None else torch.empty_like(k)
    if q.numel():
        if positions is None:
            positions = torch.arange(q.shape[2] if q.dim() == 4 else q.shape[0], dtype=torch.int32, device=q.device)
        attn_rotary(four(q), four(qo), four(k), four(ko), positions, inv_freq, interleaved, inverse, factor, stream)
    return qo if k is None else (qo, ko)


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, factor):
        ctx.save_for_backward(positions, inv_freq)
        ctx.how = (interleaved, factor)
        return _rotary(q, k, positions, inv_freq, interleaved, False, factor, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dq, dk=None):
        positions, inv_freq = ctx.saved_tensors
        # As for attention: gradients the library cannot read in place (expanded,
        # oddly strided, misaligned) are made contiguous first.
        dq, dk = (g if g is None or _readable(g) else g.contiguous() for g in (dq, dk))
        got = _rotary(dq, dk, positions, inv_freq, ctx.how[0], True, ctx.how[1], None)
        dq, dk = (got, None) if dk is None else got
        return dq, dk, None, None, None, None


def _readable(g) -> bool:
    return g.stride(-1) == 1 and all(s and s % 8 == 0 for s in g.stride()[:-1]) and g.data_ptr() % 16 == 0


def rotary(q, k=None, positions=None, inv_freq=None, interleaved: bool = False, factor: float = 1.0, stream=None):
    """Q and K (or Q alone) with rotary positions applied, differentiable in
    both: q [B, Hq, N, d] and k [B, Hk, N, d] bf16/f16 views (any layout with d
    contiguous), or both packed [total, H, d].  ``positions``: int32 [N] or
    [B, N] ([total] when packed), by default 0..N-1; ``inv_freq`` and ``factor``
    from ``rotary_frequencies`` (its defaults if not given).  The first
    2 * len(inv_freq) elements of a head are turned, the others copied."""
    if inv_freq is None:
        inv_freq, _ = rotary_frequencies(q.shape[-1], device=q.device)
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if stream is not None:
            raise ValueError("rotary under autograd runs on the current stream: use torch.cuda.stream(...)")
        return _Rotary.apply(q, k, positions, inv_freq, bool(interleaved), float(factor))
    return _rotary(q, k, positions, inv_freq, interleaved, False, factor, stream)


def rotary_backward(dq, dk=None, positions=None, inv_freq=None, interleaved: bool = False, factor: float = 1.0,
                    stream=None):
    """The gradient of ``rotary`` with the same arguments: from the gradients of
    its outputs those of q and k."""
    if inv_freq is None:
        inv_freq, _ = rotary_frequencies(dq.shape[-1], device=dq.device)
    return _rotary(dq, dk, positions, inv_freq, interleaved, True, factor, stream)


# ---------------------------------------------------------------- the cache
def _cache(k_cache, v_cache, dtype, d):
    """Pages, heads, page size and C strides of a cache."""
    shape, sk = _operand(k_cache, "k_cache", 4)
    if k_cache.dtype != dtype or shape[3] != d:
        raise ValueError("k_cache and v_cache must be [num_pages, Hkv, page_size, d] of the tokens' type and d")
    sv = _like(v_cache, "v_cache", shape, dtype)
    return shape[0], shape[1], shape[2], Strides(sk[0], sk[1], sk[2]), Strides(sv[0], sv[1], sv[2])


def _tables(page_table, seqlens, cu_seqlens, total):
    """B, pages a row, and row stride of the table, and the offsets' address."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError(f"page_table must be [B, max_pages], got {tuple(shape)}")
    B, pages = shape
    _int32(page_table, "page_table", shape)
    _int32(seqlens, "seqlens", (B,))
    if cu_seqlens is None:
        if B == 0 or total % B:
            raise ValueError(f"without cu_seqlens the {total} new tokens must divide evenly over {B} sequences")
        return B, pages, page_table.stride(0) if B > 1 else pages, None
    _int32(cu_seqlens, "cu_seqlens", (B + 1,))
    return B, pages, page_table.stride(0) if B > 1 else pages, cu_seqlens.data_ptr()


def attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens=None, q=None, q_out=None, inv_freq=None,
                      interleaved: bool = False, factor: float = 1.0, stream=None) -> None:
    """C ``attn_cache_append``: k, v packed [total, Hkv, d] into the pages of their
    sequences; with ``inv_freq`` K is turned to its position, and q into q_out
    ([total, Hq, d], which may be q) if given."""
    shape, sk = _operand(k, "k", 3)
    total, Hk, d = shape
    dtype = k.dtype
    sv = _like(v, "v", shape, dtype)
    P, Hc, ps, skc, svc = _cache(k_cache, v_cache, dtype, d)
    if Hc != Hk:
        raise ValueError(f"k and v have {Hk} heads, the cache {Hc}")
    B, pages, row, cu = _tables(page_table, seqlens, cu_seqlens, total)
    if (q is None) != (q_out is None) or (q is not None and inv_freq is None):
        raise ValueError("q, q_out and inv_freq go together")
    Hq, qp, qop, sq, sqo, fp, rot = 0, None, None, _NO_STRIDES, _NO_STRIDES, None, 0
    if q is not None:
        qs, st = _operand(q, "q", 3)
        Hq = qs[1]
        if qs != (total, Hq, d) or q.dtype != dtype:
            raise ValueError("q must be [total, Hq, d] of k's type")
        so = _like(q_out, "q_out", qs, dtype)
        qp, qop, sq, sqo = q.data_ptr(), q_out.data_ptr(), Strides(0, st[1], st[0]), Strides(0, so[1], so[0])
    if inv_freq is not None:
        fp, rot = inv_freq.data_ptr(), _frequencies(inv_freq)
    dev = _on(k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens, q, q_out, inv_freq)
    if total == 0:
        return
    _call((_lib._lib or load()).attn_cache_append, dev, stream, _DTYPES[dtype], qp, sq, qop, sqo, Hq, k.data_ptr(),
          Strides(0, sk[1], sk[0]), v.data_ptr(), Strides(0, sv[1], sv[0]), k_cache.data_ptr(), skc, v_cache.data_ptr(), svc,
          Hk, P, ps, page_table.data_ptr(), row, pages, seqlens.data_ptr(), cu, B, total, d, fp, rot,
          1 if interleaved else 0, factor)


def attn_fwd_paged_workspace_size(B: int, Hq: int, Hkv: int, total: int, max_seqlen_q: int, max_seqlen_k: int,
                                  d: int) -> int:
    """C ``attn_fwd_paged_workspace_size`` (bytes; 0 for invalid sizes)."""
    return int(load().attn_fwd_paged_workspace_size(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d))


def attn_fwd_paged(q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q: int, max_seqlen_k: int,
                   causal: bool, scale: float, workspace, stream=None, window: int = 0) -> None:
    """C ``attn_fwd_paged``: q, o packed [total, Hq, d], lse fp32 [Hq, total]; the new
    tokens are the last positions of their sequences in the cache."""
    shape, sq = _operand(q, "q", 3)
    total, Hq, d = shape
    dtype = q.dtype
    P, Hkv, ps, skc, svc = _cache(k_cache, v_cache, dtype, d)
    so = _like(o, "o", shape, dtype)
    if lse.dtype != torch.float32 or lse.shape != (Hq, total) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous float32 [Hq, total]")
    B, pages, row, cu = _tables(page_table, seqlens, cu_seqlens, total)
    dev = _on(q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, workspace)
    if total == 0:
        return
    ws, ws_bytes = (None, 0) if workspace is None else (workspace.data_ptr(), workspace.nbytes)
    _call((_lib._lib or load()).attn_fwd_paged, dev, stream, _DTYPES[dtype], q.data_ptr(), Strides(0, sq[1], sq[0]),
          k_cache.data_ptr(), skc, v_cache.data_ptr(), svc, o.data_ptr(), Strides(0, so[1], so[0]), lse.data_ptr(), P, ps,
          page_table.data_ptr(), row, pages, seqlens.data_ptr(), cu, B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d,
          1 if causal else 0, window, scale, ws, ws_bytes)


def forward_paged(q, k_cache, v_cache, page_table, seqlens, cu_seqlens=None, max_seqlen_q: int | None = None,
                  max_seqlen_k: int | None = None, causal: bool = True, scale: float | None = None, stream=None,
                  window: int = 0):
    """Attention of new tokens over a paged cache: q packed [total, Hq, d], the
    cache and tables as in the module's head; returns O (like q) and lse fp32
    [Hq, total].  ``max_seqlen_q`` defaults to total / B without ``cu_seqlens`` and
    to total with them, ``max_seqlen_k`` to the table's capacity: give them where
    they are known, they size the work's split."""
    total, Hq, d = q.shape
    B = page_table.shape[0]
    if max_seqlen_q is None:
        max_seqlen_q = total if cu_seqlens is not None else total // max(B, 1)
    if max_seqlen_k is None:
        max_seqlen_k = page_table.shape[1] * k_cache.shape[2]
    watchdog_check(q.device)
    o = torch.empty_like(q)
    lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
    nbytes = attn_fwd_paged_workspace_size(B, Hq, k_cache.shape[1], total, max_seqlen_q, max_seqlen_k, d)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
    attn_fwd_paged(q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q, max_seqlen_k, causal,
                   d ** -0.5 if scale is None else scale, ws, stream, window)
    watchdog_poll(q.device, stream)
    return o, lse


def _pages(x, name: str):
    """Host int32 page numbers, contiguous."""
    if not isinstance(x, torch.Tensor):
        x = torch.tensor(list(x), dtype=torch.int32)
    if x.is_cuda:
        raise ValueError(f"{name}: page numbers are host data (page tables are kept on the host)")
    if x.dim() != 1 or x.dtype != torch.int32:
        raise ValueError(f"{name} must be 1-D int32 page numbers")
    return x.contiguous()


def attn_cache_copy(pool, src, dst, stream=None) -> None:
    """C ``attn_cache_copy``: pool [slabs, num_pages, ...] (each page dense; slabs are
    layers' K and V; a single cache passes as ``x.unsqueeze(0)``), src and dst
    host page numbers (int32 tensors or sequences): page dst[i] of every slab
    becomes a copy of page src[i]."""
    if pool.dim() < 3 or not pool.is_cuda:
        raise ValueError("pool must be a CUDA tensor [slabs, num_pages, ...]")
    shape, st = pool.shape, pool.stride()
    each = 1
    for step, n in sorted((step, n) for step, n in zip(st[2:], shape[2:]) if n > 1):
        if step != each:
            raise ValueError("each page of the pool must be one dense block")
        each *= n
    src, dst = _pages(src, "src"), _pages(dst, "dst")
    n = src.numel()
    if n != dst.numel():
        raise ValueError("src and dst must be of one length")
    if n == 0:
        return
    size = pool.element_size()
    _call((_lib._lib or load()).attn_cache_copy, pool.get_device(), stream, pool.data_ptr(), st[0] * size, st[1] * size,
          each * size, shape[0], shape[1], src.data_ptr(), dst.data_ptr(), n)
