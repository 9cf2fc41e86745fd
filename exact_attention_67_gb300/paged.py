"""Operators around a paged key/value cache: the C ABI's rotary, cache and
paged-attention calls on torch tensors (include/exattn.h; the same names, checks
and argument marshalling only, in csrc/binding.cpp), and the helpers on top of
them.

A cache is a pair of [num_pages, Hkv, page_size, d] views (d contiguous; a
token-major [num_pages, page_size, Hkv, d] tensor passes as
``x.transpose(1, 2)``), a page table int32 [B, max_pages] and lengths int32 [B]
on the device.  New tokens are packed [total, H, d] tensors with offsets
``cu_seqlens`` int32 [B + 1], or ``cu_seqlens=None`` when every sequence has
total / B of them.
"""
from __future__ import annotations

import contextlib
import importlib.machinery
import importlib.util
import math
import os

import torch

from . import build as _build
from ._lib import _check, load, watchdog_step

_binding = None


def _native():
    """The module that checks the tensors and calls the C ABI (csrc/binding.cpp);
    like the library, it has to have been built."""
    global _binding
    if _binding is None:
        load()
        if not os.path.exists(_build.BINDING):
            raise ImportError(f"{_build.BINDING} is missing: build it with `python -m exact_attention_67_gb300.build`")
        if not _build.binding_fits():
            raise ImportError(f"{_build.BINDING} was built for another Python or PyTorch: build it again with "
                              "`python -m exact_attention_67_gb300.build`")
        loader = importlib.machinery.ExtensionFileLoader("_exattn_binding", _build.BINDING)
        spec = importlib.util.spec_from_file_location("_exattn_binding", _build.BINDING, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        _binding = module
    return _binding


def on_stream(stream, device):
    """What a helper allocates and computes for a call on ``stream`` belongs to it:
    made on the current stream, it would not be ordered with the call, and its
    memory could be given away while the call runs."""
    if stream is None or device.type != "cuda":
        return contextlib.nullcontext()
    if isinstance(stream, int):
        # The default stream's handle is 0, which ExternalStream takes for none.
        stream = torch.cuda.ExternalStream(stream, device=device) if stream else torch.cuda.default_stream(device)
    return torch.cuda.stream(stream)


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
    one 16-bit type (k, k_out may be None), positions int32 [N] or [B, N]; or
    packed [total, H, d] ones, positions [total].  inv_freq float64
    [rot_dim / 2].  An output may be its own input."""
    status = _native().rotary(q, q_out, k, k_out, positions, inv_freq, interleaved, inverse, factor, stream)
    if status:
        _check(status)


def _rotary(q, k, positions, inv_freq, interleaved, inverse, factor, stream):
    if stream is not None:
        with on_stream(stream, q.device):
            return _rotary(q, k, positions, inv_freq, interleaved, inverse, factor, None)
    if positions is None:
        positions = torch.arange(q.shape[2] if q.dim() == 4 else q.shape[0], dtype=torch.int32, device=q.device)
    status, qo, ko = _native().rotary_new(q, k, positions, inv_freq, interleaved, inverse, factor, None)
    if status:
        _check(status)
    return qo if k is None else (qo, ko)


class _Rotary(torch.autograd.Function):
    """The rotation, and with ``inverse`` its gradient.  It is linear, so forward
    mode is the same call on the tangents, reverse mode the other one on the
    gradients, to any order."""

    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, interleaved, inverse, factor):
        ctx.save_for_backward(positions, inv_freq)
        ctx.save_for_forward(positions, inv_freq)
        ctx.how = (interleaved, inverse, factor)
        return _rotary(q, k, positions, inv_freq, interleaved, inverse, factor, None)

    @staticmethod
    def jvp(ctx, tq, tk, *_):
        positions, inv_freq = ctx.saved_tensors
        interleaved, inverse, factor = ctx.how
        return _turn(_read(tq), _read(tk), positions, inv_freq, interleaved, inverse, factor, None)

    @staticmethod
    def backward(ctx, dq, dk=None):
        positions, inv_freq = ctx.saved_tensors
        interleaved, inverse, factor = ctx.how
        got = _turn(_read(dq), _read(dk), positions, inv_freq, interleaved, not inverse, factor, None)
        dq, dk = (got, None) if dk is None else got
        return dq, dk, None, None, None, None, None


def _read(g):
    """As for attention: gradients the library cannot read in place (expanded,
    oddly strided, misaligned) are copied first.  (``contiguous()`` would give back
    a contiguous tensor at a misaligned address, or with an odd stride along an axis
    of one.)"""
    return g if g is None or _readable(g) else g.clone(memory_format=torch.contiguous_format)


def _readable(g) -> bool:
    return g.stride(-1) == 1 and all(s and s % 8 == 0 for s in g.stride()[:-1]) and g.data_ptr() % 16 == 0


def _differentiated(*tensors) -> bool:
    """Whether automatic differentiation, in either mode, follows one of them."""
    return any(t is not None and (t.requires_grad and torch.is_grad_enabled()
                                  or torch.autograd.forward_ad.unpack_dual(t).tangent is not None) for t in tensors)


def _turn(q, k, positions, inv_freq, interleaved, inverse, factor, stream):
    if inv_freq is None:
        with on_stream(stream, q.device):
            inv_freq, _ = rotary_frequencies(q.shape[-1], device=q.device)
    if _differentiated(q, k):
        if stream is not None:
            raise ValueError("rotary under autograd runs on the current stream: use torch.cuda.stream(...)")
        return _Rotary.apply(q, k, positions, inv_freq, bool(interleaved), inverse, float(factor))
    return _rotary(q, k, positions, inv_freq, interleaved, inverse, factor, stream)


def rotary(q, k=None, positions=None, inv_freq=None, interleaved: bool = False, factor: float = 1.0, stream=None):
    """Q and K (or Q alone) with rotary positions applied, differentiable in
    both (in reverse and forward mode, to any order): q [B, Hq, N, d] and k [B, Hk, N, d]
    bf16/f16 views (any layout with d contiguous), or both packed [total, H, d].
    ``positions``: int32 [N] or [B, N] ([total] when packed), by default 0..N-1;
    ``inv_freq`` and ``factor`` from ``rotary_frequencies`` (its defaults if not
    given: they come from the host, so give them to a captured call).  The first 2 * len(inv_freq) elements of a head are turned, the
    others copied."""
    return _turn(q, k, positions, inv_freq, interleaved, False, factor, stream)


def rotary_backward(dq, dk=None, positions=None, inv_freq=None, interleaved: bool = False, factor: float = 1.0,
                    stream=None):
    """The gradient of ``rotary`` with the same arguments: from the gradients of
    its outputs those of q and k.  Differentiable like ``rotary``."""
    return _turn(dq, dk, positions, inv_freq, interleaved, True, factor, stream)


# ---------------------------------------------------------------- the cache
def attn_cache_append(k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens=None, q=None, q_out=None, inv_freq=None,
                      interleaved: bool = False, factor: float = 1.0, stream=None) -> None:
    """C ``attn_cache_append``: k, v packed [total, Hkv, d] into the pages of their
    sequences; with ``inv_freq`` K is turned to its position, and q into q_out
    ([total, Hq, d], which may be q) if given."""
    status = _native().cache_append(k, v, k_cache, v_cache, page_table, seqlens, cu_seqlens, q, q_out, inv_freq, interleaved,
                                    factor, stream)
    if status:
        _check(status)


def attn_fwd_paged_workspace_size(B: int, Hq: int, Hkv: int, total: int, max_seqlen_q: int, max_seqlen_k: int,
                                  d: int) -> int:
    """C ``attn_fwd_paged_workspace_size`` (bytes; 0 for invalid sizes)."""
    return int(load().attn_fwd_paged_workspace_size(B, Hq, Hkv, total, max_seqlen_q, max_seqlen_k, d))


def attn_fwd_paged(q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q: int, max_seqlen_k: int,
                   causal: bool, scale: float, workspace, stream=None, window: int = 0) -> None:
    """C ``attn_fwd_paged``: q, o packed [total, Hq, d], lse fp32 [Hq, total]; the new
    tokens are the last positions of their sequences in the cache."""
    status = _native().fwd_paged(q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q, max_seqlen_k,
                                 causal, scale, workspace, stream, window)
    if status:
        _check(status)


def forward_paged(q, k_cache, v_cache, page_table, seqlens, cu_seqlens=None, max_seqlen_q: int | None = None,
                  max_seqlen_k: int | None = None, causal: bool = True, scale: float | None = None, stream=None,
                  window: int = 0):
    """Attention of new tokens over a paged cache: q packed [total, Hq, d], the
    cache and tables as in the module's head; returns O (like q) and lse fp32
    [Hq, total].  ``max_seqlen_q`` defaults to total / B without ``cu_seqlens`` and
    to total with them, ``max_seqlen_k`` to the table's capacity: give them where
    they are known, they size the work's split.  Rows of no sequence, and new
    tokens past ``max_seqlen_q``, are not written.  Not differentiable."""
    if not q.is_cuda:
        raise ValueError("all device operands must be CUDA tensors")
    total, Hq, d = q.shape
    B = page_table.shape[0]
    if max_seqlen_q is None:
        max_seqlen_q = total if cu_seqlens is not None else total // max(B, 1)
    if max_seqlen_k is None:
        max_seqlen_k = page_table.shape[1] * k_cache.shape[2]
    nbytes = attn_fwd_paged_workspace_size(B, Hq, k_cache.shape[1], total, max_seqlen_q, max_seqlen_k, d)
    with on_stream(stream, q.device):
        o = torch.empty_like(q)
        lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        watchdog_step(q.device, lambda: attn_fwd_paged(
            q, k_cache, v_cache, o, lse, page_table, seqlens, cu_seqlens, max_seqlen_q, max_seqlen_k, causal,
            d ** -0.5 if scale is None else scale, ws, None, window))
    return o, lse


def attn_cache_copy(pool, src, dst, stream=None) -> None:
    """C ``attn_cache_copy``: pool [slabs, num_pages, ...] (each page dense; slabs are
    layers' K and V; a single cache passes as ``x.unsqueeze(0)``), src and dst
    host page numbers (int32 tensors or sequences): page dst[i] of every slab
    becomes a copy of page src[i]."""
    status = _native().cache_copy(pool, src, dst, stream)
    if status:
        _check(status)
