"""A paged key/value cache for serving: the pages of all layers in one pool, and
on the host the page tables, lengths and reference counts of the sequences.

    cache = PagedCache(num_pages=4096, page_size=16, layers=32, kv_heads=8, head_dim=128)
    seq = cache.add()
    step = cache.extend([seq], 300)                      # a prompt of 300 tokens
    for layer in ...:
        cache.append(layer, step, k, v, q=q, q_out=q, inv_freq=freq, factor=factor)
        o, lse = cache.attend(layer, step, q)
    drafts = cache.fork(seq, 4)                          # share the prompt's pages
    step = cache.extend(drafts, 1)                       # each gets its own last page
    cache.free(drafts[1:])
    cache.compact()

Everything that moves or computes on the device runs in the library's kernels
(attn_cache_append, attn_fwd_paged, attn_cache_copy)."""
from __future__ import annotations

import heapq
from dataclasses import dataclass
from functools import cached_property

import torch

from .paged import attn_cache_append, attn_cache_copy, forward_paged, on_stream


class OutOfPages(RuntimeError):
    """The pool has too few free pages; the cache is as it was before the call."""


@dataclass(frozen=True)
class Step:
    """New tokens of some sequences, as the cache calls take them: the tokens are
    packed in the order of ``ids``, ``new[i]`` of sequence ``ids[i]``."""
    ids: tuple
    new: tuple
    page_table: torch.Tensor            # int32 [B, max_pages]
    seqlens: torch.Tensor               # int32 [B], the new tokens included
    cu_seqlens: torch.Tensor | None     # int32 [B + 1]; None where all have as many
    max_seqlen_q: int
    max_seqlen_k: int

    @cached_property
    def tokens(self) -> int:
        """Rows of the packed tensors."""
        return sum(self.new)


class PagedCache:
    """Pages of ``layers`` layers' K and V, [2 layers, num_pages, kv_heads, page_size,
    head_dim], and the sequences that hold them.  Not thread-safe; the device work
    of a call runs on the current stream (or ``stream``), so calls on several
    streams are for the caller to order.  Contents start uninitialised: rows that
    no sequence has written reach no output."""

    def __init__(self, num_pages: int, page_size: int, layers: int, kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda"):
        if num_pages < 1 or layers < 1 or kv_heads < 1:
            raise ValueError("num_pages, layers and kv_heads must be positive")
        if page_size < 8 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two, 8 to 1024, got {page_size}")
        if head_dim not in (64, 128) or dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("head_dim must be 64 or 128, dtype bfloat16 or float16")
        self.page_size, self.num_pages, self.layers = page_size, num_pages, layers
        self.pool = torch.empty((2 * layers, num_pages, kv_heads, page_size, head_dim), dtype=dtype, device=device)
        self._free = list(range(num_pages))  # a heap: the lowest first
        self._refs = [0] * num_pages
        self._pages: dict[int, list[int]] = {}
        self._length: dict[int, int] = {}
        self._next = 0

    # ------------------------------------------------------------ what is there
    @property
    def free_pages(self) -> int:
        return len(self._free)

    def length(self, seq: int) -> int:
        return self._length[seq]

    def pages(self, seq: int) -> tuple:
        return tuple(self._pages[seq])

    def k_cache(self, layer: int) -> torch.Tensor:
        """[num_pages, kv_heads, page_size, head_dim] of one layer."""
        return self.pool[2 * self._layer(layer)]

    def v_cache(self, layer: int) -> torch.Tensor:
        return self.pool[2 * self._layer(layer) + 1]

    def _layer(self, layer: int) -> int:
        if not 0 <= layer < self.layers:
            raise IndexError(f"layer {layer} of {self.layers}")
        return layer

    # ------------------------------------------------------------ sequences
    def add(self) -> int:
        """A new, empty sequence."""
        seq, self._next = self._next, self._next + 1
        self._pages[seq], self._length[seq] = [], 0
        return seq

    def fork(self, seq: int, count: int = 1) -> list[int]:
        """``count`` sequences that begin as ``seq`` and share its pages; nothing is
        copied until one of them writes to a shared page (``extend``)."""
        pages, length = self._pages[seq], self._length[seq]
        out = []
        for _ in range(count):
            new = self.add()
            self._pages[new], self._length[new] = list(pages), length
            for p in pages:
                self._refs[p] += 1
            out.append(new)
        return out

    def free(self, seqs) -> None:
        """Forget sequences; pages that no other sequence holds are free again."""
        seqs = [seqs] if isinstance(seqs, int) else list(seqs)
        if len(set(seqs)) != len(seqs) or any(s not in self._pages for s in seqs):
            raise KeyError(f"not all of {seqs} are distinct sequences of this cache")
        for s in seqs:
            self._release(self._pages.pop(s))
            del self._length[s]

    def truncate(self, seq: int, length: int) -> None:
        """Drop the tokens from ``length`` on (rejected drafts, for instance)."""
        if not 0 <= length <= self._length[seq]:
            raise ValueError(f"length {length} of {self._length[seq]}")
        keep = -(-length // self.page_size)
        self._release(self._pages[seq][keep:])
        del self._pages[seq][keep:]
        self._length[seq] = length

    def _release(self, pages) -> None:
        for p in pages:
            self._refs[p] -= 1
            if self._refs[p] == 0:
                heapq.heappush(self._free, p)

    # ------------------------------------------------------------ a step
    def extend(self, seqs, new, stream=None) -> Step:
        """Room for ``new`` tokens (a number, or one a sequence) at the end of each
        sequence.  A last page that is shared and will be written to is copied
        first, for all sequences and layers in one launch.  Raises OutOfPages,
        changing nothing, if the pool is too small."""
        seqs = list(seqs)
        new = [new] * len(seqs) if isinstance(new, int) else list(new)
        if not seqs or len(new) != len(seqs) or any(n < 0 for n in new):
            raise ValueError("give at least one sequence, and a count of new tokens for each")
        if len(set(seqs)) != len(seqs) or any(s not in self._pages for s in seqs):
            raise KeyError(f"not all of {seqs} are distinct sequences of this cache")
        ps = self.page_size
        # Who copies: of the holders of a shared page, the last one to write keeps it.
        held, copies, grow = {}, [], []
        for s, n in zip(seqs, new):
            pages, length = self._pages[s], self._length[s]
            if n and length % ps:
                last = pages[-1]
                holders = held.get(last, self._refs[last])
                if holders > 1:
                    copies.append(s)
                    held[last] = holders - 1
            grow.append(-(-(length + n) // ps) - len(pages))
        need = len(copies) + sum(grow)
        if need > len(self._free):
            raise OutOfPages(f"{need} pages needed, {len(self._free)} free")
        taken = [heapq.heappop(self._free) for _ in range(need)]
        src, dst = [self._pages[s][-1] for s in copies], taken[: len(copies)]
        try:
            # Tables first, then the copy: whatever fails, nothing has changed.
            tables, fresh = [], iter(taken[len(copies):])
            own = dict(zip(copies, dst))
            for s, g in zip(seqs, grow):
                pages = list(self._pages[s])
                if s in own:
                    pages[-1] = own[s]
                pages.extend(next(fresh) for _ in range(g))
                tables.append(pages)
            step = self._step(seqs, new, tables, stream)
            if src:
                self._copy(src, dst, stream)
        except BaseException:
            for p in taken:
                heapq.heappush(self._free, p)
            raise
        for p in src:
            self._refs[p] -= 1
        for p in taken:
            self._refs[p] = 1
        for s, n, pages in zip(seqs, new, tables):
            self._pages[s] = pages
            self._length[s] += n
        return step

    def _step(self, seqs, new, tables, stream) -> Step:
        B = len(seqs)
        lens = [self._length[s] + n for s, n in zip(seqs, new)]
        width = max(max(len(pages) for pages in tables), 1)
        even = len(set(new)) == 1 and new[0] > 0
        # One copy to the device: the table, the lengths, the offsets.
        rows = [p for pages in tables for p in pages + [0] * (width - len(pages))]
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        host = torch.tensor(rows + lens + offsets, dtype=torch.int32)
        if self.pool.is_cuda:
            host = host.pin_memory()
        with on_stream(stream, self.pool.device):
            dev = host.to(self.pool.device, non_blocking=True)
        return Step(tuple(seqs), tuple(new), dev[: B * width].view(B, width), dev[B * width: B * width + B],
                    None if even else dev[B * width + B:], max(max(new), 1), max(max(lens), 1))

    def append(self, layer: int, step: Step, k, v, q=None, q_out=None, inv_freq=None, interleaved: bool = False,
               factor: float = 1.0, stream=None) -> None:
        """Store the step's K and V of one layer, [tokens, kv_heads, head_dim], K and Q
        turned to their positions with ``inv_freq`` (``attn_cache_append``).  A step
        with offsets may be followed by rows of no sequence (padding)."""
        self._rows(step, k)
        attn_cache_append(k, v, self.k_cache(layer), self.v_cache(layer), step.page_table, step.seqlens, step.cu_seqlens,
                          q, q_out, inv_freq, interleaved, factor, stream)

    def attend(self, layer: int, step: Step, q, causal: bool = True, scale: float | None = None, window: int = 0,
               stream=None):
        """Attention of the step's Q, [tokens, Hq, head_dim], over one layer of the
        cache: O like q and the logsumexp [Hq, tokens] (``forward_paged``), padding's
        rows as they happen to be."""
        self._rows(step, q)
        return forward_paged(q, self.k_cache(layer), self.v_cache(layer), step.page_table, step.seqlens, step.cu_seqlens,
                             step.max_seqlen_q, step.max_seqlen_k, causal, scale, stream, window)

    @staticmethod
    def _rows(step, x) -> None:
        # Without offsets the kernels take the rows to be divided evenly: twice the
        # tokens would be taken for two a sequence, over the one before.  Rows behind
        # the last offset are of no sequence.
        if x.dim() != 3 or x.shape[0] < step.tokens or (x.shape[0] > step.tokens and step.cu_seqlens is None):
            raise ValueError(f"the step has {step.tokens} new tokens, got {tuple(x.shape)}")

    # ------------------------------------------------------------ the pool
    def compact(self, stream=None) -> int:
        """Move pages so that those in use are the pool's first; returns how many
        moved.  Steps made before hold the old page numbers: make new ones
        (``extend`` by 0 tokens gives the tables of sequences as they are)."""
        used = self.num_pages - len(self._free)
        holes = sorted(p for p in self._free if p < used)
        movers = [p for p in range(used, self.num_pages) if self._refs[p]]
        if not movers:
            return 0
        self._copy(movers, holes, stream)
        to = dict(zip(movers, holes))
        for pages in self._pages.values():
            pages[:] = [to.get(p, p) for p in pages]
        for a, b in to.items():
            self._refs[b], self._refs[a] = self._refs[a], 0
        self._free = list(range(used, self.num_pages))
        return len(movers)

    def _copy(self, src, dst, stream) -> None:
        attn_cache_copy(self.pool, src, dst, stream)
