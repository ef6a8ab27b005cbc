"""GB300-native Pre-hoc Sparsity (PrHS) sparse-decode path.

The compute lives in ``libprhs.so`` (hand-written sm_103a CUDA behind a C
ABI, declared in ``include/prhs.h``); ``binding`` marshals torch tensors
into it, ``decoder`` keeps the per-head CIS anchor state of a decode
sequence, ``tokens`` the buffers of a step of several tokens and ``pool`` the
pages that sequences share. Nothing here falls back to host code: without the built library
every call raises.
"""
from .binding import (KVCache, PrhsError, RopeTable, cis_dilate, commit_tokens, compact_seqs, copy_rows,
                      decode_step, dense_attn, find_shared, fork_seqs, last_error, load,
                      make_pages_workspace, make_shared_workspace, make_tree_workspace, make_workspace,
                      num_sms, pages_workspace_size, plan_tokens, retrieve, rope_append, rope_turns,
                      score_select, set_mass, shared_attn, shared_workspace_size, sparse_attn,
                      tree_attn, tree_workspace_size, workspace_init, workspace_size)
from .decoder import SparseDecoder
from .pool import PagePool
from .tokens import TokenBatch

__all__ = ["KVCache", "PagePool", "PrhsError", "RopeTable", "SparseDecoder", "TokenBatch",
           "cis_dilate", "commit_tokens", "compact_seqs", "copy_rows", "decode_step",
           "dense_attn", "find_shared", "fork_seqs", "last_error", "load", "make_pages_workspace",
           "make_shared_workspace", "make_tree_workspace", "make_workspace", "num_sms",
           "pages_workspace_size", "plan_tokens", "retrieve", "rope_append", "rope_turns",
           "score_select", "set_mass", "shared_attn", "shared_workspace_size", "sparse_attn",
           "tree_attn", "tree_workspace_size", "workspace_init", "workspace_size"]
