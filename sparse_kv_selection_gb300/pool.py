"""Sequences that share the pages of one cache.

``PagePool`` keeps the bookkeeping of a paged cache's pages on the device: which
are free, how many each sequence holds and how many sequences hold each. Rows of
the batch become copies of other rows (samples of one prompt, beams that trade
places), end, or keep a part of their positions; the rows that have to move are
copied in the cache of every layer. Nothing synchronises with the host, so the
calls can be captured into a graph, and ``TokenBatch(kv, rope, ...,
share_prefixes=True, **pool.pages)`` feeds tokens to the same sequences.

A ``SparseDecoder`` on one of the caches loses its anchors of the rows that change (a
captured call: those decoders that were there when it was captured, which the pool then
keeps). Decoders on other ``KVCache`` objects of the same table need ``reset(rows)``.
"""
from __future__ import annotations

import torch

from . import binding as _b
from .tokens import _own_stream


class PagePool:
    def __init__(self, kv: _b.KVCache, *, free_pages, n_pages, free_head=None, page_shares=None, layers=(), stream=None):
        """free_pages (int32): the pages that no sequence holds from free_head[0]
        on (int32 [1], 0 when left out); those in front of it are room for pages that come
        back, so a list of all the pool's pages with free_head at the number in use always
        has enough. n_pages (int32 [B]): the pages that each row of the block table holds.
        page_shares (int32 [num_blocks], zeros when left out): the rows that hold each page,
        less one. layers: caches of further layers on the same block table and lengths."""
        if kv.block_table is None:
            raise ValueError("PagePool needs a paged cache")
        for x in layers:
            if x.block_table is None or x.block_table.data_ptr() != kv.block_table.data_ptr() or x.desc.block_size != kv.desc.block_size:
                raise ValueError("the layers' caches must use the same block table and page size")
            if x.seq_lens.data_ptr() != kv.seq_lens.data_ptr():
                raise ValueError("the layers' caches must use the same seq_lens")
            if x.block_table.shape != kv.block_table.shape or x.desc.num_blocks < kv.desc.num_blocks:
                raise ValueError("the layers' caches must have the same rows and columns, and no fewer pages")
        self.kv, self.layers, self.stream = kv, (kv, *layers), stream
        i32 = dict(device=kv.device, dtype=torch.int32)
        with torch.cuda.stream(_own_stream(stream, kv.device)):
            self.pages = dict(free_pages=free_pages, n_pages=n_pages,
                              free_head=torch.zeros(1, **i32) if free_head is None else free_head)
            self.page_shares = torch.zeros(kv.desc.num_blocks, **i32) if page_shares is None else page_shares
            self.ws = _b.make_pages_workspace(kv)
            self._rows = torch.arange(kv.B, **i32)
        self._moves, self._captured = [], []

    def _lists(self, cap):
        """The lists of a call's row copies: the front of two buffers, which double when a call
        needs more (the older ones stay, for the graphs that hold them)."""
        n = _b._int32(self.kv.B * cap, "the number of rows to copy")
        if not self._moves or self._moves[-1][0].numel() < n:
            most = max(n, 2 * self._moves[-1][0].numel()) if self._moves else n
            with torch.cuda.stream(_own_stream(self.stream, self.kv.device)):
                self._moves.append([torch.empty(most, device=self.kv.device, dtype=torch.int32) for _ in range(2)])
        return [x[:n].view(self.kv.B, cap) for x in self._moves[-1]]

    def _copy(self, lists):
        for kv in self.layers:
            _b.copy_rows(kv, *lists, stream=self.stream)

    def _forget(self, changed):
        """No anchors of rows that are not what they were: changed() flags them. Those of
        a refused call's rows too, which then retrieve once more."""
        decoders = [x for kv in self.layers for x in kv.decoders]
        if not decoders:
            return
        with torch.cuda.device(self.kv.index), torch.cuda.stream(_own_stream(self.stream, self.kv.device)):
            rows = changed()
            for x in decoders:
                x.reset(rows)
            if torch.cuda.is_current_stream_capturing():  # the graph writes to them
                self._captured += [x for x in decoders if x not in self._captured]

    def fork(self, parent: torch.Tensor) -> None:
        """Row b becomes what row parent[b] (int32 [B]) is: b itself, another row, or -1:
        the sequence ends."""
        lists = self._lists(self.kv.desc.block_size)
        _b.fork_seqs(self.kv, parent, *lists, self.ws, page_shares=self.page_shares, stream=self.stream, **self.pages)
        self._copy(lists)
        self._forget(lambda: parent != self._rows)

    def free(self, done: torch.Tensor) -> None:
        """The rows flagged in done (bool [B]) end."""
        _b._flags(done, "done", self.kv)
        with torch.cuda.stream(_own_stream(self.stream, self.kv.device)):
            parent = torch.where(done, -1, self._rows)
        self.fork(parent)

    def compact(self, keep: torch.Tensor, keep_n: torch.Tensor) -> None:
        """Row b keeps the positions keep[b][:keep_n[b]] (int32, ascending; keep_n[b] < 0:
        all). Keys keep the rotation they were cached with."""
        lists = self._lists(keep.shape[-1])
        _b.compact_seqs(self.kv, keep, keep_n, *lists, self.ws, page_shares=self.page_shares, stream=self.stream,
                        **self.pages)
        self._copy(lists)
        self._forget(lambda: keep_n >= 0)
