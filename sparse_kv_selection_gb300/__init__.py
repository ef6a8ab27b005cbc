"""GB300-native Pre-hoc Sparsity (PrHS) sparse-decode path.

The compute lives in ``libprhs.so`` (hand-written sm_103a CUDA behind a C
ABI, declared in ``include/prhs.h``); ``binding`` marshals torch tensors
into it and ``decoder`` keeps the per-head CIS anchor state of a decode
sequence. Nothing here falls back to host code: without the built library
every call raises.
"""
from .binding import (KVCache, PrhsError, RopeTable, cis_dilate, commit_tokens, decode_step,
                      dense_attn, last_error, load, make_tree_workspace, make_workspace, num_sms,
                      plan_tokens, retrieve, rope_append, rope_turns, score_select, set_mass,
                      sparse_attn, tree_attn, tree_workspace_size, workspace_init, workspace_size)
from .decoder import SparseDecoder
from .tokens import TokenBatch

__all__ = ["KVCache", "PrhsError", "RopeTable", "SparseDecoder", "TokenBatch", "cis_dilate",
           "commit_tokens", "decode_step", "dense_attn", "last_error", "load",
           "make_tree_workspace", "make_workspace", "num_sms", "plan_tokens", "retrieve",
           "rope_append", "rope_turns", "score_select", "set_mass", "sparse_attn", "tree_attn",
           "tree_workspace_size", "workspace_init", "workspace_size"]
