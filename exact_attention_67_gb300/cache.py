"""A paged key/value cache for serving: the pages of all layers in one pool, and
on the host the page tables, lengths and reference counts of the sequences.

    cache = PagedCache(num_pages=4096, page_size=16, layers=32, kv_heads=8, head_dim=128)
    seq = cache.add()
    step = cache.extend([seq], 300)                      # a prompt of 300 tokens
    for layer in ...:
        cache.append(layer, step, k, v, q=q, q_out=q, inv_freq=freq, factor=factor)
        o, lse = cache.attend(layer, step, q)
    drafts = cache.fork(seq, 4)                          # share the prompt's pages
    step = cache.extend(drafts, 1, shared=True)          # each gets its own last page; attend reads the prompt once
    cache.free(drafts[1:])
    cache.compact()

Everything that moves or computes on the device runs in the library's kernels
(attn_cache_append, attn_fwd_paged, attn_fwd_paged_shared, attn_cache_copy)."""
from __future__ import annotations

import heapq
from dataclasses import dataclass, replace
from functools import cached_property

import torch

from .paged import attn_cache_append, attn_cache_copy, forward_paged, forward_paged_shared, on_stream


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
    cu_groups: torch.Tensor | None = None    # int32 [groups + 1]: neighbours that share rows; None: no groups
    prefix_lens: torch.Tensor | None = None  # int32 [B]: rows that a sequence shares with its group
    max_group_q: int = 0

    @cached_property
    def tokens(self) -> int:
        """Rows of the packed tensors."""
        return sum(self.new)


def _shared_rows(a, b, page_size: int) -> int:
    """Rows of the leading pages that two page lists have in common."""
    lo, hi = 0, min(len(a), len(b))
    while lo < hi:
        mid = (lo + hi + 1) // 2
        if a[lo:mid] == b[lo:mid]:
            lo = mid
        else:
            hi = mid - 1
    return lo * page_size


def _groups(tables, before, page_size: int):
    """Offsets of the groups of neighbours that share rows before their new tokens, and
    each sequence's shared rows: the split that saves the most reads, where m sequences that
    share c rows save (m - 1) c.  (Taken as they come, a short one in front would pull a deep
    group down to its own few rows.)  The kernels share whole tiles of 128 rows.

    A group shares the least that two neighbours in it have in common, so the best split of
    the first sequences follows from those of fewer.  Where neighbours have as many rows in
    common as the next ones, a cut between moves to an end of that run without a loss: cuts
    are tried there only, and forks of one prompt cost no more than a pair.  (64 forks on 2,048
    pages 2.2 ms, nearly all for the pages in common; 600 prompts that all branch at other rows
    40 to 60, of which their tables take as much again in ``extend``.)"""
    B = len(tables)
    edge = [min(before[i], before[i + 1], _shared_rows(tables[i], tables[i + 1], page_size)) // 128 * 128 for i in range(B - 1)]
    inner = {i + 1 for i in range(B - 1)
             if not edge[i] or i in (0, B - 2) or edge[i] != edge[i - 1] or edge[i] != edge[i + 1]}
    cuts = [0, *sorted(inner), B]
    best, last = [0], [0]  # of the sequences before a cut: reads saved, the cut that their last group begins at
    for j in range(1, len(cuts)):
        rows, top, start = 1 << 62, -1, 0
        for i in range(j - 1, -1, -1):
            if i + 1 < j:
                rows = min(rows, edge[cuts[i + 1] - 1])
            if cuts[i + 1] - cuts[i] > 1:
                rows = min(rows, edge[cuts[i]])
            if not rows:
                break
            saved = best[i] + (cuts[j] - cuts[i] - 1) * rows
            if saved >= top:
                top, start = saved, i
            if best[i] + (cuts[j] - 1) * rows < top:  # what is left for groups that begin before
                break
        best.append(top)
        last.append(start)
    offsets, shared, j = [B], [0] * B, len(cuts) - 1
    while j > 0:
        begin, end = cuts[last[j]], cuts[j]
        if end - begin > 1:
            shared[begin:end] = [min(edge[begin:end - 1])] * (end - begin)
        offsets.append(begin)
        j = last[j]
    return offsets[::-1], shared


class PagedCache:
    """Pages of ``layers`` layers' K and V, [2 layers, num_pages, kv_heads, page_size,
    head_dim], and the sequences that hold them.  Not thread-safe; the device work
    of a call runs on the current stream (or ``stream``), so calls on several
    streams are for the caller to order.  Contents start uninitialised: rows that
    no sequence has written reach no output.

    ``share_from``: bytes of K and V of a layer whose repeated reads a step has to save
    before ``extend(shared=True)`` makes it one of groups; None: 96 MiB where each sequence
    takes one new token, 256 MB where some take more.  Reading shared pages again, mostly from
    L2, costs less than a second line of units and a join: next tokens are even at 60 to 130 MB
    (of 16 sequences behind 4,096 rows, 8 key heads of 64, 126 MB: 19.4 us with groups, 25.4
    without; behind 1,024, 31 MB, 17.9 and 12.6), five at some 250 (126 MB 38.2 and 34.9, 252 MB
    53.5 and 57.5).  (``attn_fwd_paged_shared`` decides by its call's sizes once more, as if all
    of the longest sequence were shared.)  A call over groups has a workspace of 8 bytes an
    element of O, for the join, beside what it has without."""

    def __init__(self, num_pages: int, page_size: int, layers: int, kv_heads: int, head_dim: int,
                 dtype=torch.bfloat16, device="cuda", share_from: int | None = None):
        if num_pages < 1 or layers < 1 or kv_heads < 1:
            raise ValueError("num_pages, layers and kv_heads must be positive")
        if page_size < 8 or page_size > 1024 or page_size & (page_size - 1):
            raise ValueError(f"page_size must be a power of two, 8 to 1024, got {page_size}")
        if head_dim not in (64, 128) or dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("head_dim must be 64 or 128, dtype bfloat16 or float16")
        self.page_size, self.num_pages, self.layers, self.share_from = page_size, num_pages, layers, share_from
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
    def extend(self, seqs, new, stream=None, shared: bool = False) -> Step:
        """Room for ``new`` tokens (a number, or one a sequence) at the end of each
        sequence.  With ``shared`` neighbours in ``seqs`` that have their first pages in
        common (``fork``) are taken as groups, whose shared rows ``attend`` streams once,
        where that pays (``share_from``): put such sequences side by side.  A last page
        that is shared and will be written to is copied first, for all sequences and
        layers in one launch.  Raises OutOfPages, changing nothing, if the pool is too
        small."""
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
            step = self._step(seqs, new, tables, stream, shared)
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

    def _step(self, seqs, new, tables, stream, shared) -> Step:
        B = len(seqs)
        lens = [self._length[s] + n for s, n in zip(seqs, new)]
        width = max(max(len(pages) for pages in tables), 1)
        even = len(set(new)) == 1 and new[0] > 0
        # One copy to the device: the table, the lengths, the offsets.
        rows = [p for pages in tables for p in pages + [0] * (width - len(pages))]
        offsets = [0]
        for n in new:
            offsets.append(offsets[-1] + n)
        groups, prefix = _groups(tables, [self._length[s] for s in seqs], self.page_size) if shared else ([], [])
        # What the first of a group reads, the others need not.
        saved = sum(prefix) - sum(prefix[i] for i in groups[:-1])
        least = self.share_from if self.share_from is not None else 96 << 20 if max(new) <= 1 else 256_000_000
        if saved * self.pool.shape[2] * self.pool.shape[4] * 4 < max(1, least):
            groups, prefix = [], []
        host = torch.tensor(rows + lens + offsets + prefix + groups, dtype=torch.int32)
        if self.pool.is_cuda:
            host = host.pin_memory()
        with on_stream(stream, self.pool.device):
            dev = host.to(self.pool.device, non_blocking=True)
        table, lens_d, offsets_d, prefix_d, groups_d = dev.split([B * width, B, B + 1, len(prefix), len(groups)])
        step = Step(tuple(seqs), tuple(new), table.view(B, width), lens_d, None if even else offsets_d, max(max(new), 1),
                    max(max(lens), 1))
        if groups:
            step = replace(step, cu_groups=groups_d, prefix_lens=prefix_d,
                           max_group_q=max(1, *(offsets[j] - offsets[i] for i, j in zip(groups, groups[1:]))))
        return step

    def append(self, layer: int, step: Step, k, v, q=None, q_out=None, inv_freq=None, interleaved: bool = False,
               factor: float = 1.0, stream=None, q_gain=None, k_gain=None, eps: float = 1e-6) -> None:
        """Store the step's K and V of one layer, [tokens, kv_heads, head_dim], K and Q
        turned to their positions with ``inv_freq``, and before it normalised by head
        with gains (``attn_cache_append``).  A step with offsets may be followed by rows
        of no sequence (padding)."""
        self._rows(step, k)
        attn_cache_append(k, v, self.k_cache(layer), self.v_cache(layer), step.page_table, step.seqlens, step.cu_seqlens,
                          q, q_out, inv_freq, interleaved, factor, stream, q_gain, k_gain, eps)

    def attend(self, layer: int, step: Step, q, causal: bool = True, scale: float | None = None, window: int = 0,
               stream=None):
        """Attention of the step's Q, [tokens, Hq, head_dim], over one layer of the
        cache: O like q and the logsumexp [Hq, tokens] (``forward_paged``; over a step
        made with ``shared`` and without a window ``forward_paged_shared``), padding's
        rows as they happen to be."""
        self._rows(step, q)
        if step.cu_groups is not None and window == 0:
            return forward_paged_shared(q, self.k_cache(layer), self.v_cache(layer), step.page_table, step.seqlens,
                                        step.cu_groups, step.prefix_lens, step.cu_seqlens, step.max_seqlen_q,
                                        step.max_seqlen_k, step.max_group_q, causal, scale, stream)
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
