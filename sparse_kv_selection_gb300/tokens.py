"""Steps that feed several new tokens per sequence through one KV cache.

``TokenBatch`` holds the device buffers of such a step and calls the four
operators in order: ``plan`` (pages, slots, positions, tree masks), ``rotate``
(rotary positions; k and v into the cache or kept packed), ``attend`` (over
the cache and the new tokens) and ``commit`` (accepted tokens join the cache).
It serves prompt chunks (``rotate(..., append=True)``, then ``commit`` of all
tokens), the verification of drafted trees, and plain decode with one token a
sequence. Nothing synchronises with the host, so a step can be captured into a
graph; the same cache can be decoded by ``SparseDecoder`` between steps. Where
neighbouring sequences share pages (``PagePool.fork``), ``share_prefixes`` reads
what they share once.

Layers of a model whose caches have one block table and one ``seq_lens`` take a batch each,
TokenBatch(kv_i, ..., **first.pages). Every layer plans (the pages that the first one took
are there for the others, so all get the same slots) before any commits, and the lengths move
once: chunks are appended by ``rotate`` in every layer and committed in the last; accepted
tokens of trees are committed in the others by ``commit_tokens`` with a ``new_lens`` that
nobody reads.
"""
from __future__ import annotations

import torch

from . import binding as _b


def _own_stream(stream, device):
    """The stream object of a handle (None: the current stream)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return stream
    handle = int(getattr(stream, "cuda_stream", stream))
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


class TokenBatch:
    def __init__(self, kv: _b.KVCache, rope: _b.RopeTable, *, max_tokens: int, max_new: int,
                 free_pages=None, n_pages=None, free_head=None, scale: float | None = None, stream=None,
                 share_prefixes: bool = False, min_shared: int = 256):
        """max_tokens packed tokens at most (padding included), max_new of one
        sequence (the attention's form is chosen by it, so a batch for single tokens
        is faster with 1 than one for chunks is at the same step). A paged cache needs free_pages (int32, the pages that no
        sequence holds), n_pages (int32 [B], the pages each row of its block
        table holds) and free_head (int32 [1], how many of free_pages have been
        taken; zero when left out). plan updates free_head and n_pages in place:
        batches on one cache share all three, TokenBatch(..., **other.pages). A
        sequence that ends gives its p pages back in front of the free ones
        (free_head -= p, then free_pages[free_head : free_head + p] = them) and has
        its n_pages and its length set to 0; PagePool does that, and keeps count of
        pages that several sequences hold.
        share_prefixes: plan also finds the prefixes of at least min_shared keys that
        neighbouring sequences share, and attend reads each once (find_shared,
        shared_attn)."""
        dev, B, d = kv.k.device, kv.B, kv.desc.d
        self.kv, self.rope, self.stream = kv, rope, stream
        self.max_new = int(max_new)
        if share_prefixes and not 0 <= min_shared < 2**31:
            raise ValueError(f"min_shared must be in [0, 2**31), got {min_shared}")
        self.scale = scale if scale is not None else d ** -0.5
        # on the batch's own stream: it may run a step before this one gets to the fills
        with torch.cuda.stream(_own_stream(stream, dev)):
            i32 = dict(device=dev, dtype=torch.int32)
            T = int(max_tokens)
            self.cu_new = torch.zeros(B + 1, **i32)
            self.positions = torch.zeros(T, **i32)
            self.slots = torch.full((T,), -1, **i32)
            self._mask = torch.zeros(T, _b.TREE_WORDS, **i32)
            self.tree_mask = None
            self.pages = {}
            if kv.block_table is not None:
                if free_pages is None or n_pages is None:
                    raise ValueError("a paged cache needs free_pages and n_pages")
                self.pages = dict(free_pages=free_pages, n_pages=n_pages,
                                  free_head=torch.zeros(1, **i32) if free_head is None else free_head)
            self.q = torch.zeros(T, kv.Hq, d, device=dev, dtype=kv.k.dtype)
            self.k = torch.zeros(T, kv.desc.Hkv, d, device=dev, dtype=kv.k.dtype)
            self.v = None
            self.out = torch.zeros(T, kv.Hq, d, device=dev, dtype=kv.k.dtype)
            self.lse = torch.zeros(T, kv.Hq, device=dev, dtype=torch.float32)
            self.min_shared, self.shared = int(min_shared), None
            if share_prefixes:
                self.shared = torch.zeros(B, 4, **i32)
                self.ws = _b.make_shared_workspace(kv, T, self.max_new)
            else:
                self.ws = _b.make_tree_workspace(kv, self.max_new)
        self._in_cache = False

    def plan(self, n_new: torch.Tensor, parents: torch.Tensor | None = None) -> None:
        """Place n_new[b] tokens behind each sequence's cached prefix. parents
        ([max_tokens] int32, packed) makes them trees; without, they are chunks."""
        self.tree_mask = None if parents is None else self._mask
        self.v, self._in_cache = None, False     # rows of an earlier plan are not this one's
        _b.plan_tokens(self.kv, n_new, self.cu_new, self.positions, self.slots, parents=parents,
                       tree_mask=self.tree_mask, stream=self.stream, **self.pages)
        if self.shared is not None:
            _b.find_shared(self.kv, self.cu_new, self.shared, min_keys=self.min_shared, stream=self.stream)

    def rotate(self, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, append: bool = False) -> None:
        """Rotate q [max_tokens][Hq][d] and k [max_tokens][Hkv][d] at the planned
        positions; append writes k and v into the cache at the planned slots
        (chunks whose tokens will all be committed), and leaves out those that
        plan refused, whose attention then has no meaning. v is kept for attend
        and commit: it must not change before them."""
        if append and self.tree_mask is not None:
            raise ValueError("a tree's tokens join the cache when they are committed")
        _b.rope_append(self.kv, self.rope, self.positions, q, k, v, self.q,
                       slots=self.slots if append else None, k_out=self.k, stream=self.stream)
        self.v, self._in_cache = v, append

    def attend(self, out: torch.Tensor | None = None, lse: torch.Tensor | None = None) -> None:
        """Attention of the new tokens into out and lse (the batch's own by default)."""
        tree = self.tree_mask is not None     # (planning refuses trees above TREE_MAX tokens)
        max_new = min(self.max_new, _b.TREE_MAX) if tree else self.max_new
        to = (self.out if out is None else out, self.lse if lse is None else lse, self.ws)
        if self.shared is not None:
            _b.shared_attn(self.kv, self.q, self.k, self.v, self.scale, self.cu_new, max_new, self.shared, *to,
                           tree_mask=self.tree_mask, stream=self.stream)
        else:
            _b.tree_attn(self.kv, self.q, self.k, self.v, self.scale, self.cu_new, max_new, *to,
                         tree_mask=self.tree_mask, stream=self.stream)

    def commit(self, accept_n: torch.Tensor, accept_idx: torch.Tensor | None = None) -> None:
        """Add accept_n[b] tokens (numbers accept_idx[b], or the first ones) to
        each sequence's cache and advance its length. Sequences that plan refused
        stay as they are, flagged, whatever accept_n says of them."""
        rows = {} if self._in_cache and accept_idx is None else dict(k_new=self.k, v_new=self.v)
        _b.commit_tokens(self.kv, self.cu_new, accept_n, slots=self.slots, accept_idx=accept_idx,
                         stream=self.stream, **rows)
